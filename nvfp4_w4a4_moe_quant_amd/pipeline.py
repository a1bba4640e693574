"""The rollout hot path as a sequence of C-ABI calls (no arithmetic here).

Dense linear (one GEMM input):
    nvfp4_quantize(X, stats) -> rac_select_residual -> w4a4_grouped_gemm_rac
MoE FFN layer (QUADS rollout: online NVFP4 activations + RAC on every GEMM
input, 4-bit by 4-bit expert GEMMs; arXiv abstract on the mlsanity page and the
blog post's section "Two fixes, on two different sides"):
    moe_route(logits)
    nvfp4_quantize(X, stats) -> rac_select_residual(X)
    w4a4_grouped_gemm_rac(gate/up, gather = routed rows, epilogue SiLU*mul -> H
                          bf16 and max|H|)
    nvfp4_quantize(H, amax_in = max|H|, stats) -> rac_select_residual(H)
    w4a4_grouped_gemm_rac(down) -> Y (FP32, rows in expert order)
    moe_combine(Y, row_of, routing weights) -> token-order output (moe_block)
GraphedMoEBlock captures the whole block once as a HIP graph for fixed
shapes (decode), so a step replays every kernel with no host work per launch.
For up to 64 tokens moe_decode computes the whole layer in two or three
launches with unquantized activations, on the same weights; token_logprobs
gives the log-probabilities and entropies of the tokens that both sides of
the rollout-trainer gap are measured by, with their gradient.
int8_linear and int8_moe_block are the dense layer and the MoE block in 8-bit
integers (per-token and per-channel scales), a rollout to compare with;
moe_balance_loss is the trainer's loss on the router that moe_route follows.
Weights are quantized once, per expert and projection, by the same
nvfp4_quantize (every engine quantizes the synchronized weights the same way:
blog post, section "The failure mode").
"""
from __future__ import annotations

from typing import Dict, Iterable, NamedTuple, Optional, Tuple

import torch
from torch.autograd import forward_ad

from . import _lib as L


class QuantWeights(NamedTuple):
    w: L.NVFP4          # codes [G, N, K/2], scales [G, N, K/16], tscale [G]
    N: int
    K: int


def quantize_weights(mats: Iterable[Tuple[int, torch.Tensor]], G: int, N: int, K: int,
                     device) -> QuantWeights:
    """mats yields (group index, W_g [N, K] on any device); each W_g becomes one
    NVFP4 tensor with its own tensor scale."""
    codes = torch.empty((G, N, K // 2), dtype=torch.uint8, device=device)
    scales = torch.empty((G, N, K // 16), dtype=torch.uint8, device=device)
    ts = torch.empty(G, dtype=torch.float32, device=device)
    for g, wg in mats:
        wg = wg.to(device, non_blocking=True)
        q = L.nvfp4_quantize(wg).q
        codes[g].copy_(q.codes)
        scales[g].copy_(q.scales)
        ts[g:g + 1].copy_(q.tscale)
    return QuantWeights(L.NVFP4(codes, scales, ts), N, K)


class GemmInput(NamedTuple):
    qo: L.QuantOut
    rac: Optional[L.RacOut]
    skip_inactive: bool = False
    per_group: bool = False  # per-expert tensor scales (quantize_input_grouped)


# Below this selected fraction of channels, many 16-blocks are likely to hold
# no selected channel, and the GEMM skips their residual MFMAs; above it the
# branch-free residual pass is faster (an inactive block's residual is zero).
SKIP_BELOW_FRACTION = 1.0 / 8


def quantize_input(x: torch.Tensor, n_select: Optional[int],
                   amax_in: Optional[torch.Tensor] = None) -> GemmInput:
    """Online quantization of a GEMM input; n_select None turns RAC off."""
    qo = L.nvfp4_quantize(x, amax_in=amax_in, stats=n_select is not None, channel_max=False)
    rac = L.rac_select_residual(x, qo, n_select) if n_select is not None else None
    skip = n_select is not None and n_select <= SKIP_BELOW_FRACTION * x.shape[1]
    return GemmInput(qo, rac, skip)


def quantize_input_grouped(x: torch.Tensor, offsets: torch.Tensor, total_rows: int,
                           n_select: Optional[int],
                           gather: Optional[torch.Tensor] = None) -> GemmInput:
    """Per-expert RAC: each expert's rows (gathered from x when gather is
    given) are quantized and compensated as their own tensor; the GEMM then
    runs on grouped rows without a gather."""
    qo = L.nvfp4_quantize_grouped(x, offsets, total_rows, gather_rows=gather,
                                  stats=n_select is not None, channel_max=False)
    rac = (L.rac_select_residual_grouped(x, qo, offsets, total_rows, n_select, gather_rows=gather)
           if n_select is not None else None)
    skip = n_select is not None and n_select <= SKIP_BELOW_FRACTION * x.shape[1]
    return GemmInput(qo, rac, skip, True)


def gemm(inp: GemmInput, wq: QuantWeights, offsets: torch.Tensor, total_rows: int, *,
         gather: Optional[torch.Tensor] = None, epilogue: int = L.NVFP4_EPI_F32,
         out_amax: Optional[torch.Tensor] = None) -> torch.Tensor:
    return L.w4a4_grouped_gemm_rac(
        inp.qo.q, wq.w, offsets, N=wq.N, K=wq.K, total_rows=total_rows, gather_rows=gather,
        r=inp.rac.r if inp.rac else None,
        kblock_active=inp.rac.kblock_active if inp.rac else None,
        epilogue=epilogue, out_amax=out_amax, skip_inactive=inp.skip_inactive,
        per_group_scales=inp.per_group)


def dense_forward(x: torch.Tensor, wq: QuantWeights, n_select: Optional[int],
                  offsets: Optional[torch.Tensor] = None) -> Dict:
    """offsets: the one-group offsets [0, rows] (int32, on the device); made
    here when not given (a host-to-device copy, so a graph capture passes
    its own)."""
    rows = x.shape[0]
    if offsets is None:
        offsets = torch.tensor([0, rows], dtype=torch.int32, device=x.device)
    inp = quantize_input(x, n_select)
    y = gemm(inp, wq, offsets, rows)
    return dict(x_in=inp, y=y, offsets=offsets)


def moe_forward(x: torch.Tensor, logits: torch.Tensor, wgu: QuantWeights, wd: QuantWeights,
                topk: int, n_sel_x: Optional[int], n_sel_h: Optional[int],
                per_expert: bool = False) -> Dict:
    """per_expert: RAC (and the activation tensor scales) per expert group
    instead of per GEMM-input tensor; the gate/up input is then quantized per
    expert from the gathered token rows."""
    T = x.shape[0]
    rt = L.moe_route(logits, topk)
    rows = T * topk
    amax_h = torch.zeros(1, dtype=torch.float32, device=x.device)
    if per_expert:
        x_in = quantize_input_grouped(x, rt.expert_offsets, rows, n_sel_x, gather=rt.gather_rows)
        h = gemm(x_in, wgu, rt.expert_offsets, rows, epilogue=L.NVFP4_EPI_SILU_MUL_BF16,
                 out_amax=amax_h)
        h_in = quantize_input_grouped(h, rt.expert_offsets, rows, n_sel_h)
    else:
        x_in = quantize_input(x, n_sel_x)
        h = gemm(x_in, wgu, rt.expert_offsets, rows, gather=rt.gather_rows,
                 epilogue=L.NVFP4_EPI_SILU_MUL_BF16, out_amax=amax_h)
        h_in = quantize_input(h, n_sel_h, amax_in=amax_h)
    y = gemm(h_in, wd, rt.expert_offsets, rows)
    return dict(route=rt, x_in=x_in, h=h, amax_h=amax_h, h_in=h_in, y=y)


def moe_block(x: torch.Tensor, logits: torch.Tensor, wgu: QuantWeights, wd: QuantWeights,
              topk: int, n_sel_x: Optional[int], n_sel_h: Optional[int],
              out_dtype: torch.dtype = torch.bfloat16) -> Dict:
    """The full MoE FFN block: moe_forward, then the weighted combine."""
    d = moe_forward(x, logits, wgu, wd, topk, n_sel_x, n_sel_h)
    d["out"] = L.moe_combine(d["y"], d["route"].row_of, d["route"].topk_weights,
                             out_dtype=out_dtype)
    return d


def _is_dual(t: torch.Tensor) -> bool:
    """Whether t carries a tangent of forward-mode differentiation; its
    requires_grad does not say so, and no_grad does not end it."""
    return forward_ad._current_level >= 0 and forward_ad.unpack_dual(t).tangent is not None


def _no_gradient(x: Optional[torch.Tensor], logits: Optional[torch.Tensor]):
    if torch.is_grad_enabled() and ((x is not None and x.requires_grad) or
                                    (logits is not None and logits.requires_grad)):
        raise RuntimeError("the decode-step layer has no gradient: detach its inputs or call it "
                           "under torch.no_grad()")
    if (x is not None and _is_dual(x)) or (logits is not None and _is_dual(logits)):
        raise RuntimeError("the decode-step layer has no forward-mode derivative: detach its inputs")


def moe_decode(x: torch.Tensor, logits: torch.Tensor, wgu: QuantWeights, wd: QuantWeights,
               topk: int, out: Optional[torch.Tensor] = None) -> L.MoEDecodeOut:
    """The MoE FFN layer for up to 64 tokens, in token order, on the same
    quantized weights as moe_block but with unquantized activations (the values
    of the trainer's fake-quantized forward).  There is no backward pass: with
    gradients enabled, x or logits that require one are refused, and dual tensors
    of forward-mode differentiation always."""
    _no_gradient(x, logits)
    return L.nvfp4_moe_decode(x, logits, wgu.w, wd.w, topk, out=out)


class GraphedMoEBlock:
    """moe_block captured once as a HIP graph (torch.cuda.CUDAGraph) for fixed
    T, H, E.  The graph reads its inputs from two static buffers: its own, or
    the caller's x [T, H] and logits [T, E] when given (a producer that writes
    the next step's inputs there lets a call replay with no copy).  A call
    copies inputs that live elsewhere into those buffers and replays; the
    returned tensor is the graph's static output, overwritten by the next
    call.  Every kernel of the block only reads device memory the graph owns,
    the static inputs or the weights, which the object keeps, and nothing in
    it is a memset node."""

    def __init__(self, wgu: QuantWeights, wd: QuantWeights, topk: int, n_sel_x: Optional[int],
                 n_sel_h: Optional[int], T: int, E: int, x_dtype: torch.dtype, device,
                 out_dtype: torch.dtype = torch.bfloat16, warmup: int = 2,
                 x: Optional[torch.Tensor] = None, logits: Optional[torch.Tensor] = None):
        if x is not None:
            assert x.shape == (T, wgu.K) and x.dtype == x_dtype and x.is_contiguous()
        if logits is not None:
            assert logits.shape == (T, E) and logits.dtype == torch.float32
            assert logits.is_contiguous()
        self.x = x if x is not None else torch.zeros((T, wgu.K), dtype=x_dtype, device=device)
        self.logits = (logits if logits is not None
                       else torch.zeros((T, E), dtype=torch.float32, device=device))
        args = (wgu, wd, topk, n_sel_x, n_sel_h, out_dtype)
        self.weights = (wgu, wd)
        side = torch.cuda.Stream(device)
        side.wait_stream(torch.cuda.current_stream(device))
        with torch.cuda.stream(side):
            for _ in range(warmup):
                moe_block(self.x, self.logits, *args)
        torch.cuda.current_stream(device).wait_stream(side)
        self.graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(self.graph):
            self.out = moe_block(self.x, self.logits, *args)["out"]

    def __call__(self, x: Optional[torch.Tensor] = None,
                 logits: Optional[torch.Tensor] = None) -> torch.Tensor:
        if x is not None and x.data_ptr() != self.x.data_ptr():
            self.x.copy_(x)
        if logits is not None and logits.data_ptr() != self.logits.data_ptr():
            self.logits.copy_(logits)
        self.graph.replay()
        return self.out


class GraphedMoEDecode:
    """moe_decode captured once as a HIP graph for a fixed number of tokens (at
    most 64): a call replays the layer on the static inputs, its own or the
    caller's x [T, H] and logits [T, E] when given, after copying inputs of the
    same shape and type that live elsewhere.  A batch of fewer tokens is written
    into the first rows and the remaining logits rows are filled with -inf: such
    rows cost nothing and give 0.  The returned MoEDecodeOut is
    the graph's own, overwritten by the next call.  The object keeps the weights
    (the graph holds their addresses only); values written into their tensors
    are what the next call computes with."""

    def __init__(self, wgu: QuantWeights, wd: QuantWeights, topk: int, T: int, E: int,
                 x_dtype: torch.dtype, device, warmup: int = 2,
                 x: Optional[torch.Tensor] = None, logits: Optional[torch.Tensor] = None):
        self.x = x if x is not None else torch.zeros((T, wgu.K), dtype=x_dtype, device=device)
        self.logits = (logits if logits is not None
                       else torch.zeros((T, E), dtype=torch.float32, device=device))
        if self.x.shape != (T, wgu.K) or self.x.dtype != x_dtype or self.logits.shape != (T, E):
            raise ValueError("x [T, H] of x_dtype and logits [T, E]")
        dev = torch.device(device)
        if dev.type == "cuda" and dev.index is None:
            dev = torch.device("cuda", torch.cuda.current_device())
        if self.x.device != dev or self.logits.device != dev:
            raise ValueError(f"x and logits on the graph's device, {dev}")
        args = (wgu, wd, topk)
        self.weights = (wgu, wd)
        with torch.cuda.device(device):
            side = torch.cuda.Stream()
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                for _ in range(warmup):
                    moe_decode(self.x, self.logits, *args)
            torch.cuda.current_stream().wait_stream(side)
            self.graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(self.graph):
                self.out = moe_decode(self.x, self.logits, *args)

    @staticmethod
    def _lives_in(static: torch.Tensor, t: torch.Tensor) -> bool:
        """t is the static input itself, element for element."""
        return t.data_ptr() == static.data_ptr() and all(
            n == 1 or a == b for n, a, b in zip(t.shape, t.stride(), static.stride()))

    def __call__(self, x: Optional[torch.Tensor] = None,
                 logits: Optional[torch.Tensor] = None) -> L.MoEDecodeOut:
        _no_gradient(x, logits)
        given = ((self.x, x), (self.logits, logits))
        for static, t in given:
            if t is not None and (t.shape != static.shape or t.dtype != static.dtype):
                raise ValueError(f"{static.dtype} {tuple(static.shape)} instead of "
                                 f"{t.dtype} {tuple(t.shape)}")
        for static, t in given:
            if t is not None and not self._lives_in(static, t):
                static.copy_(t)
        self.graph.replay()
        return self.out


class GraphedDense:
    """dense_forward captured once as a HIP graph for fixed [rows, K] (the
    decode shape): a call copies x into the static input and replays every
    kernel of quantize + RAC + GEMM with no host work per launch.  The object
    keeps the weights."""

    def __init__(self, wq: QuantWeights, n_select: Optional[int], rows: int,
                 x_dtype: torch.dtype, device, warmup: int = 2):
        self.weights = wq
        self.x = torch.zeros((rows, wq.K), dtype=x_dtype, device=device)
        self.offsets = torch.tensor([0, rows], dtype=torch.int32, device=device)
        side = torch.cuda.Stream(device)
        side.wait_stream(torch.cuda.current_stream(device))
        with torch.cuda.stream(side):
            for _ in range(warmup):
                dense_forward(self.x, wq, n_select, self.offsets)
        torch.cuda.current_stream(device).wait_stream(side)
        self.graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(self.graph):
            self.y = dense_forward(self.x, wq, n_select, self.offsets)["y"]

    def __call__(self, x: torch.Tensor) -> torch.Tensor:
        self.x.copy_(x)
        self.graph.replay()
        return self.y


class NVFP4WeightFakeQuant(torch.autograd.Function):
    """Trainer-side Asymmetric QAT for one weight matrix: the forward pass
    uses the rollout's NVFP4 quantize-dequantize of W (nvfp4_qdq, bf16 out),
    the backward pass hands the gradient to W unchanged (straight-through).
    Activations stay unquantized (QUADS blog post, section "Two fixes, on two
    different sides")."""

    @staticmethod
    def forward(ctx, w: torch.Tensor) -> torch.Tensor:
        return L.nvfp4_qdq(w.detach().contiguous(), out_dtype=w.dtype)

    @staticmethod
    def backward(ctx, grad: torch.Tensor) -> torch.Tensor:
        return grad


class _TokenLogprobs(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, targets, inv_temperature):
        r = L.token_logprobs(logits, targets, inv_temperature=inv_temperature)
        ctx.save_for_backward(logits, targets, inv_temperature, r.norm, r.entropy)
        ctx.set_materialize_grads(False)
        return r.logprobs, r.entropy

    @staticmethod
    def backward(ctx, g_logprobs, g_entropy):
        if torch.is_grad_enabled():  # under create_graph
            raise RuntimeError("token_logprobs has no second derivative")
        logits, targets, inv_temperature, norm, entropy = ctx.saved_tensors
        if g_logprobs is None and g_entropy is None:
            return None, None, None
        if g_logprobs is not None and not g_logprobs.is_contiguous():
            g_logprobs = g_logprobs.contiguous()
        if g_entropy is not None and not g_entropy.is_contiguous():
            g_entropy = g_entropy.contiguous()
        return L.token_logprobs_backward(logits, targets, norm, entropy, g_logprobs, g_entropy,
                                         inv_temperature=inv_temperature), None, None


def token_logprobs(logits: torch.Tensor, targets: torch.Tensor,
                   inv_temperature: Optional[torch.Tensor] = None
                   ) -> Tuple[torch.Tensor, torch.Tensor]:
    """(log-probabilities of targets, entropies) of logits [T, V], with the
    gradient of the logits (the trainer's side of the rollout-trainer
    log-prob gap).  Targets and temperatures get no gradient, and there is no
    second derivative.  The gradient is contiguous; logits whose rows are spaced
    otherwise (a view of a padded vocabulary) take a slower backward pass.  Leaf
    logits that require a gradient are refused under graph capture, where
    another living graph of the same leaf ends the process: capture the two
    library calls instead.  Captured logits that an operation gave are fine as
    long as no eager graph of their leaves lives, as for any backward pass."""
    if inv_temperature is not None and inv_temperature.requires_grad:
        raise ValueError("inv_temperature gets no gradient")
    if logits.requires_grad and logits.is_leaf and torch.cuda.is_current_stream_capturing():
        raise RuntimeError("leaf logits under capture: use the library's token_logprobs and "
                           "token_logprobs_backward")
    return _TokenLogprobs.apply(logits, targets, inv_temperature)


# ------------------------------------------------- INT8 W8A8 comparator
def int8_quantize_weights(mats: Iterable[Tuple[int, torch.Tensor]], G: int, N: int, K: int,
                          device) -> L.INT8:
    """mats yields (group index, W_g [N, K] on any device); one scale for every
    output channel."""
    w = L.INT8(torch.empty((G, N, K), dtype=torch.int8, device=device),
               torch.empty((G, N), dtype=torch.float32, device=device))
    for g, wg in mats:
        L.int8_quantize_rows(wg.to(device, non_blocking=True),
                             out=L.INT8(w.codes[g], w.scales[g]))
    return w


def _int8_no_gradient(x: torch.Tensor, logits: Optional[torch.Tensor] = None):
    if (x.requires_grad or (logits is not None and logits.requires_grad)) \
            and torch.is_grad_enabled():
        raise RuntimeError("the INT8 layers have no gradient: detach their inputs or call them "
                           "under torch.no_grad()")
    if _is_dual(x) or (logits is not None and _is_dual(logits)):
        raise RuntimeError("the INT8 layers have no forward-mode derivative: detach their inputs")


def int8_linear(x: torch.Tensor, w: L.INT8,
                out_dtype: torch.dtype = torch.bfloat16) -> torch.Tensor:
    """y = x W^T of x [rows, K] (bf16 or FP32), quantized per row by the call, and
    w (codes [1, N, K], scales [1, N]), as bf16 or FP32 [rows, N]."""
    _int8_no_gradient(x)
    if out_dtype is torch.bfloat16:
        epilogue = L.NVFP4_EPI_BF16
    elif out_dtype is torch.float32:
        epilogue = L.NVFP4_EPI_F32
    else:
        raise TypeError(f"unsupported dtype {out_dtype}")
    _, N, K = w.codes.shape
    return L.int8_grouped_gemm(x, w, N=N, K=K, total_rows=x.shape[0], epilogue=epilogue)


def int8_moe_block(x: torch.Tensor, logits: torch.Tensor, wgu: L.INT8, wd: L.INT8, topk: int,
                   out_dtype: torch.dtype = torch.bfloat16) -> Dict:
    """moe_block in 8-bit integers: routing, gate/up on the rows of x quantized
    per token, SiLU*mul, down on the rows of h quantized per row, combine.  wgu
    holds [E, 2I, H] (gate rows first), wd [E, H, I]."""
    _int8_no_gradient(x, logits)
    rows = x.shape[0] * topk
    rt = L.moe_route(logits, topk)
    h = L.int8_grouped_gemm(x, wgu, rt.expert_offsets, N=wgu.codes.shape[1], K=wgu.codes.shape[2],
                            total_rows=rows, gather_rows=rt.gather_rows,
                            epilogue=L.NVFP4_EPI_SILU_MUL_BF16)
    y = L.int8_grouped_gemm(h, wd, rt.expert_offsets, N=wd.codes.shape[1], K=wd.codes.shape[2],
                            total_rows=rows)
    out = L.moe_combine(y, rt.row_of, rt.topk_weights, out_dtype=out_dtype)
    return dict(route=rt, h=h, y=y, out=out)


# ------------------------------------------------- the router's balance loss
class _BalanceLoss(torch.autograd.Function):
    """The losses; what else the call gives goes into the list `rest`."""

    @staticmethod
    def forward(ctx, logits, topk_ids, mask, rest):
        r = L.moe_balance_loss(logits, topk_ids, mask=mask)
        ctx.save_for_backward(logits, r.counts, r.tokens, mask)
        ctx.k = topk_ids.shape[1]
        ctx.set_materialize_grads(False)
        rest.append(r)
        return r.losses

    @staticmethod
    def backward(ctx, g_losses):
        if torch.is_grad_enabled():  # under create_graph
            raise RuntimeError("moe_balance_loss has no second derivative")
        if g_losses is None:
            return None, None, None, None
        logits, counts, tokens, mask = ctx.saved_tensors
        return L.moe_balance_loss_backward(logits, ctx.k, counts, tokens, g_losses.contiguous(),
                                           mask=mask), None, None, None


def moe_balance_loss(logits: torch.Tensor, topk_ids: torch.Tensor,
                     mask: Optional[torch.Tensor] = None) -> L.BalanceOut:
    """The router's balance loss and z-loss (losses [2]) with the gradient of
    logits [T, E], and the counts and mean probabilities, which get none.
    topk_ids [T, k] is moe_route's choice.  There is no second derivative and no
    forward-mode one (a dual tensor is refused), and a backward pass fails if the
    counts were written to before it.  Leaf logits that require a gradient are
    refused under graph capture, where another living graph of the same leaf ends
    the process: capture the two library calls instead.  Captured logits that an
    operation gave are fine as long as no eager graph of their leaves lives, as for
    any backward pass."""
    if _is_dual(logits):
        raise RuntimeError("moe_balance_loss has no forward-mode derivative: detach the logits")
    if not (logits.requires_grad and torch.is_grad_enabled()):
        return L.moe_balance_loss(logits, topk_ids, mask=mask)
    if logits.is_leaf and torch.cuda.is_current_stream_capturing():
        raise RuntimeError("leaf logits under capture: use the library's moe_balance_loss and "
                           "moe_balance_loss_backward")
    rest = []
    losses = _BalanceLoss.apply(logits, topk_ids, mask, rest)
    return rest[0]._replace(losses=losses)
