"""Cases of the INT8 (W8A8) expert products and of the router's balance loss.

* `linear`: a dense layer, y = x W^T, with x quantized per token to 8-bit
  integers when it is called and W quantized per output channel beforehand;
* `experts`: one of the two products of an MoE FFN layer on the same scheme,
  grouped by expert: gate/up with the routed rows gathered and SiLU*mul, or
  down on rows in expert order;
* `balance`: what a router's statistics are per batch: the slots that each
  expert got, its mean probability, the balance loss and the z-loss;
* `balance_step`: the same with the gradient of the router's logits.

With `own` false, run() computes them from elementary torch operations in 32
bits; with `own` true it calls this package's operators.
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------- cases
def _linear(name, rows, K, N, x="bf16", y="bf16", values="normal"):
    c = dict(kind="linear", rows=rows, K=K, N=N, x=x, y=y, values=values)
    return dict(name=name, **c) if name else c


def _experts(name, side, T, E, k, H, I, x="bf16", values="normal", routing="normal", empty=0):
    c = dict(kind="experts", side=side, T=T, E=E, k=k, H=H, I=I, x=x, values=values,
             routing=routing, empty=empty)
    return dict(name=name, **c) if name else c


def _balance(name, kind, T, E, k, dtype="f32", padded=0.0, closed=0.0, dropped=0.0, pitch=0):
    c = dict(kind=kind, T=T, E=E, k=k, dtype=dtype, padded=padded, closed=closed,
             dropped=dropped, pitch=pitch)
    return dict(name=name, **c) if name else c


def listed():
    return [
        # one token through a square layer: latency
        _linear("linear 1x4096x4096", 1, 4096, 4096),
        # a decode step of a batch, FP32 output
        _linear("linear 16x4096x4096", 16, 4096, 4096, y="f32"),
        # a prompt through the same layer
        _linear("linear 4096x4096x4096", 4096, 4096, 4096),
        # FP32 rows; no size is a multiple of a tile
        _linear("linear 333x1040x1999 f32", 333, 1040, 1999, x="f32", y="f32"),
        # one token's eight experts, gate and up
        _experts("gate/up e128 1 token", "gate_up", 1, 128, 8, 2048, 768),
        # a decode step of the large layer: about 100 of 256 experts touched
        _experts("gate/up e256 16 tokens", "gate_up", 16, 256, 8, 7168, 2048, values="t3"),
        # popularity-skewed routing, experts that nobody chose, the second product
        _experts("down e128 zipf 64 tokens", "down", 64, 128, 8, 2048, 768, routing="zipf",
                 empty=8),
        # a whole batch of prompts through the large layer
        _experts("gate/up e256 8192 tokens", "gate_up", 8192, 256, 8, 7168, 2048, values="t3"),
        # the router of a decode step: latency
        _balance("balance 64x128", "balance", 64, 128, 8),
        # the trainer's step of one micro-batch
        _balance("balance step 8192x256", "balance_step", 8192, 256, 8),
        # a long packed batch with padding behind it, BF16 logits
        _balance("balance step 65536x128 bf16", "balance_step", 65536, 128, 8, dtype="bf16",
                 padded=0.2),
        # an odd number of experts in rows of a wider tensor, experts closed to a
        # token, slots dropped by a capacity limit
        _balance("balance step 5003x60 closed", "balance_step", 5003, 60, 6, closed=0.3,
                 dropped=0.05, pitch=64),
    ]


MOST = 65536 * 4096 * 7168  # multiply-adds of the largest listed case


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["linear", "linear", "experts", "experts", "balance", "balance_step"])
    x = rng.choice(["bf16", "bf16", "f32"])
    values = rng.choice(["normal", "t3"])
    if kind == "linear":
        return _linear(None, _log_uniform(rng, 1, 8192), 16 * _log_uniform(rng, 4, 512),
                       _log_uniform(rng, 32, 16384), x, rng.choice(["bf16", "f32"]), values)
    if kind == "experts":
        while True:
            E, k = _log_uniform(rng, 4, 256), rng.randint(1, 10)
            H, I = 16 * _log_uniform(rng, 8, 448), 16 * _log_uniform(rng, 4, 128)
            T = _log_uniform(rng, 1, 8192)
            side = rng.choice(["gate_up", "down"])
            if k <= E and 2 * T * k * H * I <= MOST and T * k * max(H, 2 * I) <= 65536 * 7168:
                break
        zipf = rng.random() < 0.3 and E > k + 2 and E * T <= 262144
        return _experts(None, side, T, E, k, H, I, x, values, "zipf" if zipf else "normal",
                        rng.randint(0, E - k - 1) // 4 if zipf else 0)
    E = _log_uniform(rng, 4, 512)
    T = _log_uniform(rng, 1, 65536 * 128 // E)
    return _balance(None, kind, T, E, rng.randint(1, min(E, 10)), rng.choice(["f32", "f32", "bf16"]),
                    rng.choice([0.0, 0.0, 0.25]), rng.choice([0.0, 0.0, 0.5]),
                    rng.choice([0.0, 0.1]), rng.choice([0, 0, E + rng.randint(1, 40)]))


# ------------------------------------------------------------------ inputs
def _weights(g, G, N, K):
    """INT8 codes [G, N, K] and scales [G, N] of N(0, 0.02^2) weights, a few
    groups at a time."""
    codes = torch.empty((G, N, K), dtype=torch.int8, device=DEV)
    scales = torch.empty((G, N), device=DEV)
    few = max(1, (1 << 28) // (N * K))
    for a in range(0, G, few):
        w = torch.randn((min(few, G - a), N, K), generator=g, device=DEV)
        s = w.abs().amax(2) * (0.02 / 127.0)
        scales[a:a + few] = s
        codes[a:a + few] = w.mul_((0.02 / s)[:, :, None]).round_()
    return codes, scales


def _rows(g, rows, K, values):
    x = torch.randn((rows, K), generator=g, device=DEV)
    if values == "t3":  # Student-t with 3 degrees of freedom
        x /= (torch.randn((3, rows, K), generator=g, device=DEV).square().mean(0)).sqrt()
    else:               # 1% outlier channels
        ch = torch.randperm(K, generator=g, device=DEV)[:max(1, K // 100)]
        x[:, ch] *= 20.0
    return x


def _prepare_linear(c, g):
    return dict(kind="linear", x=_rows(g, c["rows"], c["K"], c["values"]).to(TYPES[c["x"]]),
                w=_weights(g, 1, c["N"], c["K"]), y=TYPES[c["y"]])


def _prepare_experts(c, g):
    T, E, k = c["T"], c["E"], c["k"]
    lg = torch.randn((T, E), generator=g, device=DEV)
    if c["routing"] == "zipf":
        rank = torch.randperm(E, generator=g, device=DEV)
        logp = -1.2 * torch.log(rank.float() + 1.0)
        logp[rank >= E - c["empty"]] = -math.inf
        u = torch.rand((T, E), generator=g, device=DEV, dtype=torch.float64).clamp_min(1e-12)
        lg = logp - torch.log(-torch.log(u)).float()
    expert, order = torch.sort(lg.topk(k, 1).indices.reshape(-1), stable=True)
    counts = torch.bincount(expert, minlength=E)
    offsets = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
    offsets[1:] = torch.cumsum(counts, 0)
    gate_up = c["side"] == "gate_up"
    N, K = (2 * c["I"], c["H"]) if gate_up else (c["H"], c["I"])
    if gate_up:
        x = _rows(g, T, K, c["values"])
    else:  # rows after SiLU*mul
        a = 0.4 * _rows(g, T * k, K, "normal")
        x = a * torch.sigmoid(a) * torch.randn((T * k, K), generator=g, device=DEV)
    return dict(kind="experts", x=x.to(TYPES[c["x"]]), w=_weights(g, E, N, K), offsets=offsets,
                gather=(order // k).int() if gate_up else None, rows=T * k, N=N, K=K,
                most=int(counts.max()))


def _prepare_balance(c, g):
    T, E, k = c["T"], c["E"], c["k"]
    lg = torch.randn((T, max(E, c["pitch"])), generator=g, device=DEV)
    lg *= 1.5
    lg += torch.linspace(0.0, 2.0, lg.shape[1], device=DEV)  # some experts are favourites
    if c["closed"]:  # experts on devices that a token may not go to; k stay open
        shut = torch.rand(lg.shape, generator=g, device=DEV) < c["closed"]
        shut[:, :k] = False
        lg.masked_fill_(shut, -math.inf)
    lg = lg.to(TYPES[c["dtype"]])
    ids = lg[:, :E].float().topk(k, 1).indices.int()
    if c["dropped"]:
        ids[torch.rand(ids.shape, generator=g, device=DEV) < c["dropped"]] = -1
    mask = None
    if c["padded"]:
        mask = torch.arange(T, device=DEV) < T - int(c["padded"] * T)
    lg = lg[:, :E]
    s = dict(kind=c["kind"], logits=lg, ids=ids, mask=mask)
    if c["kind"] == "balance_step":
        lg.requires_grad_()
        s["grad"] = torch.tensor([0.01, 0.001], device=DEV) * \
            (0.5 + torch.rand(2, generator=g, device=DEV))
    return s


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return dict(linear=_prepare_linear, experts=_prepare_experts, balance=_prepare_balance,
                balance_step=_prepare_balance)[case["kind"]](case, g)


# ------------------------------------------------------------- plain forms
def _quantize(x):
    """Codes (as 32-bit floats) and scale of every row: s = amax / 127 and 1 / s
    each rounded once to 32 bits, the code the nearest integer to x (1 / s)."""
    x = x.float()
    s = (x.abs().amax(1).double() / 127.0).float()
    r = torch.where(s > 0, 1.0 / s.double(), torch.zeros_like(s, dtype=torch.float64)).float()
    return torch.round(x * r[:, None]).clamp_(-127.0, 127.0), s


def _plain_linear(s):
    a, sa = _quantize(s["x"])
    codes, sw = s["w"]
    y = a @ codes[0].float().T
    return dict(y=(y * (sa[:, None] * sw[0][None, :])).to(s["y"]))


def _plain_experts(s):
    a, sa = _quantize(s["x"])
    codes, sw = s["w"]
    rows, off = s["rows"], s["offsets"].long()
    row = torch.arange(rows, device=off.device)
    grp = torch.searchsorted(off, row, right=True) - 1
    src = row if s["gather"] is None else s["gather"].long()
    if rows <= s["w"][0].shape[0]:  # few rows: a copy of its weights for each
        y = torch.matmul(codes[grp].float(), a[src][:, :, None])[:, :, 0]
    else:              # every expert's rows padded to the longest
        at = (off[:-1, None] + torch.arange(s["most"], device=off.device)).clamp_max(rows - 1)
        y = torch.matmul(codes.float(), a[src][at].transpose(1, 2).contiguous())
        y = y.transpose(1, 2)[grp, row - off[grp]]
    y = y * (sa[src][:, None] * sw[grp])
    if s["gather"] is None:
        return dict(y=y)
    I = s["N"] // 2
    gate, up = y[:, :I], y[:, I:]
    return dict(h=(gate / (1.0 + torch.exp(-gate)) * up).bfloat16())


def _plain_balance(s):
    z, ids = s["logits"].detach().float(), s["ids"]
    T, E = z.shape
    k = ids.shape[1]
    m = z.amax(1)
    live = m > -math.inf
    if s["mask"] is not None:
        live = live & s["mask"]
    m = torch.where(live, m, torch.zeros_like(m))
    e = torch.where(live[:, None], torch.exp(z - m[:, None]), torch.zeros_like(z))
    total = torch.where(live, e.sum(1), torch.ones_like(m))
    p = e / total[:, None]
    lse = torch.where(live, m + torch.log(total), torch.zeros_like(m))
    n = live.sum().double().clamp_min(1.0)
    took = live[:, None] & (ids >= 0)
    counts = torch.zeros(E, dtype=torch.int32, device=z.device)
    counts.scatter_add_(0, ids.clamp_min(0).long().reshape(-1), took.reshape(-1).int())
    mean = p.sum(0, dtype=torch.float64) / n
    losses = torch.stack([E / (k * n) * (counts * mean).sum(), lse.double().square().sum() / n])
    out = dict(losses=losses.float(), counts=counts, mean_probs=mean.float())
    if s["kind"] == "balance_step":
        c = counts.double()
        cp = (p.double() * c).sum(1, keepdim=True)
        f = s["grad"][0].double() * (E / (k * n * n)) * (c - cp) \
            + (s["grad"][1].double() * (2.0 / n)) * lse.double()[:, None]
        out["grad"] = (p * f).to(s["logits"].dtype)
    return out


# ---------------------------------------------------------------- one pass
def _own(s):
    from nvfp4_w4a4_moe_quant_amd import _lib as L
    from nvfp4_w4a4_moe_quant_amd import pipeline as P
    if s["kind"] == "linear":
        return dict(y=P.int8_linear(s["x"], L.INT8(*s["w"]), out_dtype=s["y"]))
    if s["kind"] == "experts":
        up = s["gather"] is not None
        y = L.int8_grouped_gemm(s["x"], L.INT8(*s["w"]), s["offsets"], N=s["N"], K=s["K"],
                                total_rows=s["rows"], gather_rows=s["gather"],
                                epilogue=L.NVFP4_EPI_SILU_MUL_BF16 if up else L.NVFP4_EPI_F32)
        return dict(h=y) if up else dict(y=y)
    if s["kind"] == "balance":
        r = L.moe_balance_loss(s["logits"], s["ids"], mask=s["mask"])
        return dict(losses=r.losses, counts=r.counts, mean_probs=r.mean_probs)
    r = P.moe_balance_loss(s["logits"], s["ids"], mask=s["mask"])
    grad, = torch.autograd.grad([r.losses], [s["logits"]], [s["grad"]])
    return dict(losses=r.losses.detach(), counts=r.counts, mean_probs=r.mean_probs, grad=grad)


def run(state):
    if own:
        return _own(state)
    with torch.no_grad():
        return dict(linear=_plain_linear, experts=_plain_experts, balance=_plain_balance,
                    balance_step=_plain_balance)[state["kind"]](state)


# -------------------------------------------------------------------- work
def _experts_touched(c):
    """Mean number of distinct experts that the tokens route to."""
    g = torch.Generator()
    g.manual_seed(7)
    T, E, k = c["T"], c["E"], c["k"]
    n = 0
    for _ in range(4):
        lg = torch.rand((T, E), generator=g, dtype=torch.float64).clamp_min(1e-12)
        lg = -torch.log(-torch.log(lg))
        if c["routing"] == "zipf":
            logp = -1.2 * torch.log(torch.arange(1, E + 1, dtype=torch.float64))
            logp[E - c["empty"]:] = -math.inf
            lg = lg + logp
        n += torch.unique(lg.topk(k, 1).indices).numel()
    return n / 4


def work(case):
    c = case
    if c["kind"] == "linear":
        rows, K, N = c["rows"], c["K"], c["N"]
        size = dict(bf16=2, f32=4)
        return dict(bytes=rows * K * size[c["x"]] + N * K + 4 * N + rows * N * size[c["y"]],
                    flops=2.0 * rows * K * N)
    if c["kind"] == "experts":
        up = c["side"] == "gate_up"
        T, rows, size = c["T"], c["T"] * c["k"], 2 if c["x"] == "bf16" else 4
        N, K = (2 * c["I"], c["H"]) if up else (c["H"], c["I"])
        io = T * K * size + rows * c["I"] * 2 if up else rows * K * size + rows * N * 4
        return dict(bytes=_experts_touched(c) * N * (K + 4) + io, flops=2.0 * rows * N * K)
    T, E = c["T"] - int(c["padded"] * c["T"]), c["E"]
    size = 4 if c["dtype"] == "f32" else 2
    if c["kind"] == "balance":
        return dict(bytes=T * (E * size + 4 * c["k"]) + 8 * E, flops=6.0 * T * E)
    return dict(bytes=T * (E * size + 4 * c["k"]) + c["T"] * E * size + 8 * E, flops=12.0 * T * E)


# ------------------------------------------------------------ definition
def _exact_codes(x):
    """The codes by the definition: every 32-bit rounding of a 64-bit value."""
    x = x.double()
    amax = torch.linalg.vector_norm(x, ord=math.inf, dim=1, keepdim=True)
    s = (amax / 127.0).float().double()
    r = torch.zeros_like(s)
    r[s > 0] = (1.0 / s[s > 0]).float().double()
    return torch.round((x * r).float().double()).clamp(-127, 127), s


def _exact_product(a, sa, codes, sw):
    return (a @ codes.double().T.contiguous()) * sa * sw.double()[None, :]


def _exact_experts(s):
    a, sa = _exact_codes(s["x"])
    off = s["offsets"].tolist()
    up = s["gather"] is not None
    I = s["N"] // 2
    y = torch.empty((s["rows"], I if up else s["N"]), dtype=torch.float64, device=a.device)
    for e in range(len(off) - 1):
        r = slice(off[e], off[e + 1])
        if off[e] < off[e + 1]:
            t = s["gather"][r].long() if up else r
            v = _exact_product(a[t], sa[t], s["w"][0][e], s["w"][1][e])
            y[r] = v[:, :I] * torch.sigmoid(v[:, :I]) * v[:, I:] if up else v
    return dict(h=y) if up else dict(y=y)


def _exact_balance(s):
    z, ids = s["logits"].detach().double(), s["ids"]
    keep = ~torch.isinf(z).all(1)
    if s["mask"] is not None:
        keep &= s["mask"]
    E, k, n = z.shape[1], ids.shape[1], max(1, int(keep.sum()))
    zk, taken = z[keep], ids[keep]
    lse = torch.logsumexp(zk, 1, keepdim=True)
    p = torch.exp(zk - lse)
    counts = torch.bincount(taken[taken >= 0].long(), minlength=E)
    f = counts.double() * (E / (k * n))
    losses = torch.stack([(f * p.mean(0)).sum(), lse.square().mean()])
    out = dict(losses=losses, counts=None, mean_probs=p.sum(0) / n)
    if s["kind"] == "balance_step":
        g = s["grad"].double()
        of_p = g[0] * f / n                               # dB/dp, the softmax's Jacobian behind it
        of_z = p * (of_p - p @ of_p[:, None]) + g[1] * (2.0 / n) * lse * p
        grad = torch.zeros_like(z)
        grad[keep] = of_z
        out["grad"] = grad
    return out


def exact(case, seed):
    with torch.no_grad():
        s = prepare(case, seed)
        if case["kind"] == "linear":
            a, sa = _exact_codes(s["x"])
            return dict(y=_exact_product(a, sa, s["w"][0][0], s["w"][1][0]))
        return (_exact_experts if case["kind"] == "experts" else _exact_balance)(s)
