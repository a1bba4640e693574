"""Cases of the decode-step MoE layer and of the token log-probabilities.

Two paths that a rollout takes next to the W4A4 layers of this package:

* `moe`: one whole MoE FFN layer for a few tokens on the NVFP4 expert weights
  (routing, gate/up, SiLU*mul, down, weighted combine), activations left
  unquantized, as the trainer's fake-quantized forward has them;
* `logprobs`: log-probability of a given token, entropy, and the largest
  alternatives of every row of vocabulary logits (what a rollout records);
* `train`: the same log-probabilities and entropies with the gradient of the
  logits (what the trainer computes from the rollout's tokens).

With `own` false, run() computes them from elementary torch operations in 32
bits; with `own` true it calls this package's operators.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------- cases
def _moe(name, T, E, k, H, I, dtype="bf16", x="normal", routing="normal", empty=0, padded=0):
    c = dict(kind="moe", T=T, E=E, k=k, H=H, I=I, dtype=dtype, x=x, routing=routing, empty=empty,
             padded=padded)
    return dict(name=name, **c) if name else c


def _logits(name, kind, T, V, dtype="bf16", top=0, temperature=False, masked=0.0, ignored=0.0):
    c = dict(kind=kind, T=T, V=V, dtype=dtype, top=top, temperature=temperature, masked=masked,
             ignored=ignored)
    return dict(name=name, **c) if name else c


def listed():
    return [
        # one token of one request: latency, eight experts' weights streamed
        _moe("moe e128 1 token", 1, 128, 8, 2048, 768),
        # the large layer for one token
        _moe("moe e256 1 token", 1, 256, 8, 7168, 2048, x="t3"),
        # the large layer for a batch of requests: about 100 experts touched
        _moe("moe e256 16 tokens", 16, 256, 8, 7168, 2048, x="t3"),
        # popularity-skewed routing with experts that are never chosen, in a
        # batch padded to a captured size (the padded rows route nowhere)
        _moe("moe e128 zipf 64 tokens", 64, 128, 8, 2048, 768, routing="zipf", empty=8, padded=7),
        # FP32 activations and output, an odd number of tokens
        _moe("moe e128 13 tokens f32", 13, 128, 8, 2048, 768, dtype="f32"),
        # ragged sizes: not multiples of the matrix tiles
        _moe("moe e60 5 tokens ragged", 5, 60, 4, 1056, 416),
        # one sampled token of one request, with the top alternatives
        _logits("logprobs 1x32768", "logprobs", 1, 32768, top=5),
        # a decode step of a batch, each request with its own temperature
        _logits("logprobs 16x131072", "logprobs", 16, 131072, top=20, temperature=True),
        # scoring whole sequences
        _logits("logprobs 4096x131072", "logprobs", 4096, 131072, top=8),
        # FP32 logits, an odd vocabulary, masked tokens, ignored positions
        _logits("logprobs 257x100003 f32", "logprobs", 257, 100003, dtype="f32", top=3,
                masked=0.4, ignored=0.1),
        # the trainer's step: log-probabilities, entropies and the gradient
        _logits("train 2048x131072", "train", 2048, 131072, ignored=0.2),
        _logits("train 300x32003 f32", "train", 300, 32003, dtype="f32", temperature=True,
                ignored=0.1),
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["moe", "moe", "logprobs", "train"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if kind == "moe":
        while True:
            E, k = _log_uniform(rng, 4, 256), rng.randint(1, 10)
            H, I = 32 * _log_uniform(rng, 4, 224), 32 * _log_uniform(rng, 2, 64)
            T = _log_uniform(rng, 1, 64)
            if k <= E and T * k * H * I <= 128 * 7168 * 2048 and E * H * I <= 256 * 7168 * 2048:
                break
        zipf = rng.random() < 0.3 and E > k + 2
        return _moe(None, T, E, k, H, I, dtype, rng.choice(["normal", "t3"]),
                    "zipf" if zipf else "normal", rng.randint(0, E - k - 1) // 4 if zipf else 0,
                    rng.randint(0, T - 1) if rng.random() < 0.3 else 0)
    V = _log_uniform(rng, 500, 160000)
    most = (2 if kind == "train" else 4) * 1024 * 131072 // (1 if dtype == "bf16" else 2)
    T = _log_uniform(rng, 1, min(8192, most // V))
    return _logits(None, kind, T, V, dtype, rng.randint(0, 20) if kind == "logprobs" else 0,
                   rng.random() < 0.5, rng.choice([0.0, 0.0, 0.3]), rng.choice([0.0, 0.2]))


# ------------------------------------------------------------------ inputs
def _nvfp4_pool(g, blocks):
    """Quantized blocks of N(0, 0.02^2) weights: 8 code bytes as one int64 and
    an E4M3 scale byte per block of 16, with their tensor scale."""
    w = torch.randn((blocks, 16), generator=g, device=DEV) * 0.02
    ts = w.abs().amax() / 2688.0
    s = (w.abs().amax(1) / (6.0 * ts)).to(torch.float8_e4m3fn)
    q = w / (s.float() * ts)[:, None]
    mid = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=DEV)
    idx = torch.bucketize(q.abs(), mid).to(torch.uint8)
    code = torch.where((q < 0) & (idx > 0), idx | 8, idx)
    by = (code[:, 0::2] | (code[:, 1::2] << 4)).contiguous()
    return by.view(torch.int64).view(-1), s.view(torch.uint8), ts


def _expert_weights(g, pool, E, N, K):
    codes, scales, ts = pool
    pick = torch.randint(0, codes.numel(), (E * N * (K // 16),), generator=g, device=DEV,
                         dtype=torch.int32)
    c = codes[pick].view(torch.uint8).view(E, N, K // 2)
    s = scales[pick].view(E, N, K // 16)
    return c, s, ts * (0.75 + 0.5 * torch.rand(E, generator=g, device=DEV))


def _prepare_moe(c, g):
    T, E, H, I = c["T"], c["E"], c["H"], c["I"]
    pool = _nvfp4_pool(g, 1 << 18)
    x = torch.randn((T, H), generator=g, device=DEV)
    if c["x"] == "t3":  # Student-t with 3 degrees of freedom
        x = x / (torch.randn((3, T, H), generator=g, device=DEV).square().mean(0)).sqrt()
    else:               # 1% outlier channels
        ch = torch.randperm(H, generator=g, device=DEV)[:max(1, H // 100)]
        x[:, ch] *= 20.0
    lg = torch.randn((T, E), generator=g, device=DEV)
    if c["routing"] == "zipf":
        rank = torch.randperm(E, generator=g, device=DEV)
        logp = -1.2 * torch.log(rank.float() + 1.0)
        logp[rank >= E - c["empty"]] = -math.inf
        u = torch.rand((T, E), generator=g, device=DEV, dtype=torch.float64).clamp_min(1e-12)
        lg = logp - torch.log(-torch.log(u)).float()
    if c["padded"]:
        lg[T - c["padded"]:] = -math.inf
    return dict(x=x.to(TYPES[c["dtype"]]), logits=lg, gu=_expert_weights(g, pool, E, 2 * I, H),
                down=_expert_weights(g, pool, E, H, I), I=I, H=H, k=c["k"], kind="moe")


def _prepare_logits(c, g):
    T, V = c["T"], c["V"]
    z = torch.randn((T, V), generator=g, device=DEV)
    z *= 2.0
    peak = torch.randint(0, V, (T, 8), generator=g, device=DEV)
    z.scatter_(1, peak, 6.0 + 8.0 * torch.rand((T, 8), generator=g, device=DEV))
    target = torch.where(torch.rand(T, generator=g, device=DEV) < 0.8, peak[:, 0],
                         torch.randint(0, V, (T,), generator=g, device=DEV))
    if c["masked"]:  # tokens that a grammar forbids; a whole row now and then
        z.masked_fill_(torch.rand((T, V), generator=g, device=DEV) < c["masked"], -math.inf)
        z[torch.rand(T, generator=g, device=DEV) < 0.02] = -math.inf
    if c["ignored"]:
        target[torch.rand(T, generator=g, device=DEV) < c["ignored"]] = -100
    s = dict(kind=c["kind"], logits=z.to(TYPES[c["dtype"]]), targets=target, top=c["top"],
             inv_t=None)
    if c["temperature"]:
        s["inv_t"] = 1.0 / (0.6 + 0.8 * torch.rand(T, generator=g, device=DEV))
    if c["kind"] == "train":
        s["g_logp"] = torch.randn(T, generator=g, device=DEV)
        s["g_ent"] = 0.01 * torch.randn(T, generator=g, device=DEV)
        s["logits"].requires_grad_()
    return s


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return (_prepare_moe if case["kind"] == "moe" else _prepare_logits)(case, g)


# ------------------------------------------------------------- plain forms
def _lut(dev):
    """Values of the two E2M1 codes in each byte, and of each E4M3 byte."""
    mag = torch.tensor(E2M1, device=dev)
    val = torch.cat([mag, -mag])
    b = torch.arange(256, device=dev)
    return torch.stack([val[b & 15], val[b >> 4]], 1), \
        b.to(torch.uint8).view(torch.float8_e4m3fn).float()


def _expert_products(v, ids, weights):
    """y[p] = W_{ids[p]} v[p] for every (token, slot) pair p, in 32 bits."""
    codes, scales, ts = weights
    P, N, K = ids.numel(), codes.shape[1], codes.shape[2] * 2
    pairs, e4m3 = _lut(v.device)
    w = pairs[codes[ids].int()].view(P, N, K // 16, 16)
    w *= e4m3[scales[ids].int()][..., None]
    return torch.matmul(w.view(P, N, K), v[:, :, None])[:, :, 0] * ts[ids][:, None]


def _plain_moe(s):
    lg, k, I = s["logits"], s["k"], s["I"]
    T, E = lg.shape
    # descending logits, ties to the lower expert index: one integer key
    bits = (lg + 0.0).view(torch.int32).long()
    key = torch.where(bits < 0, -(bits & 0x7FFFFFFF), bits) * E + (E - 1 - torch.arange(E, device=lg.device))
    ids = torch.topk(key, k, 1).indices
    top = lg.gather(1, ids)
    mx = top[:, :1]
    mx = torch.where(mx == -math.inf, torch.zeros_like(mx), mx)
    den = torch.exp(lg - mx).sum(1, keepdim=True)
    wts = torch.where(top == -math.inf, torch.zeros_like(top), torch.exp(top - mx) / den)
    flat = ids.reshape(-1)
    x = s["x"].float().repeat_interleave(k, 0)
    y = _expert_products(x, flat, s["gu"])
    gate, up = y[:, :I], y[:, I:]
    h = gate / (1.0 + torch.exp(-gate)) * up
    y = _expert_products(h, flat, s["down"]).view(T, k, -1)
    out = (wts[:, :, None] * y).sum(1)
    return dict(out=out.to(s["x"].dtype), topk_ids=ids.int(), topk_weights=wts)


def _plain_statistics(s):
    """(scaled logits, row maximum, log of the shifted sum, log-probability of
    the target, entropy), in 32 bits."""
    z = s["logits"].detach().float()
    if s["inv_t"] is not None:
        z = z * s["inv_t"][:, None]
    m = z.amax(1, keepdim=True)
    empty = m[:, 0] == -math.inf
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    d = z - m
    e = torch.exp(d)
    sum_e = e.sum(1)
    t = torch.where(e > 0, e * d, torch.zeros_like(e)).sum(1)
    log_s = torch.log(sum_e)
    ent = torch.where(empty, torch.zeros_like(t), log_s - t / sum_e)
    tgt = s["targets"]
    at = d.gather(1, tgt.clamp_min(0)[:, None])[:, 0]
    logp = torch.where(at == -math.inf, at, at - log_s)
    return d, log_s, torch.where(tgt < 0, torch.zeros_like(logp), logp), ent, empty


def _plain_logprobs(s):
    d, log_s, logp, ent, empty = _plain_statistics(s)
    out = dict(logprobs=logp, entropy=ent)
    if s["top"]:
        raw = s["logits"].float() + 0.0
        V = raw.shape[1]
        bits = raw.view(torch.int32).long()
        key = torch.where(bits < 0, -(bits & 0x7FFFFFFF), bits) * V
        key += V - 1 - torch.arange(V, device=raw.device)
        ids = torch.topk(key, s["top"], 1).indices
        v = d.gather(1, ids)
        out["top_ids"] = ids.int()
        out["top_logprobs"] = torch.where(v == -math.inf, v, v - log_s[:, None])
    return out


def _plain_train(s):
    d, log_s, logp, ent, empty = _plain_statistics(s)
    lp = d - torch.where(empty, torch.zeros_like(log_s), log_s)[:, None]
    p = torch.exp(lp)
    tgt = s["targets"]
    g_lp = torch.where((tgt < 0) | empty, torch.zeros_like(logp), s["g_logp"])
    lp = torch.where(p > 0, lp, torch.zeros_like(lp))
    grad = -p * (g_lp[:, None] + s["g_ent"][:, None] * (lp + ent[:, None]))
    grad.scatter_add_(1, tgt.clamp_min(0)[:, None], g_lp[:, None])
    if s["inv_t"] is not None:
        grad = grad * s["inv_t"][:, None]
    return dict(logprobs=logp, entropy=ent, grad=grad.to(s["logits"].dtype))


# ---------------------------------------------------------------- one pass
def _own(s):
    from nvfp4_w4a4_moe_quant_amd import _lib as L
    from nvfp4_w4a4_moe_quant_amd import pipeline as P
    if s["kind"] == "moe":
        wgu = P.QuantWeights(L.NVFP4(*s["gu"]), 2 * s["I"], s["H"])
        wd = P.QuantWeights(L.NVFP4(*s["down"]), s["H"], s["I"])
        r = P.moe_decode(s["x"], s["logits"], wgu, wd, s["k"])
        return dict(out=r.out, topk_ids=r.topk_ids, topk_weights=r.topk_weights)
    if s["kind"] == "logprobs":
        r = L.token_logprobs(s["logits"], s["targets"], top_k=s["top"], inv_temperature=s["inv_t"])
        out = dict(logprobs=r.logprobs, entropy=r.entropy)
        if s["top"]:
            out.update(top_ids=r.top_ids, top_logprobs=r.top_logprobs)
        return out
    logp, ent = P.token_logprobs(s["logits"], s["targets"], inv_temperature=s["inv_t"])
    grad, = torch.autograd.grad([logp, ent], [s["logits"]], [s["g_logp"], s["g_ent"]])
    return dict(logprobs=logp, entropy=ent, grad=grad)


def run(state):
    if own:
        return _own(state)
    with torch.no_grad():
        return dict(moe=_plain_moe, logprobs=_plain_logprobs, train=_plain_train)[state["kind"]](
            state)


# -------------------------------------------------------------------- work
def _experts_touched(c):
    """Mean number of distinct experts that the real tokens route to."""
    T, E, k = c["T"] - c["padded"], c["E"], c["k"]
    r = np.random.default_rng(7)
    n = []
    for _ in range(4):
        lg = r.gumbel(size=(T, E)) if c["routing"] == "zipf" else r.standard_normal((T, E))
        if c["routing"] == "zipf":
            logp = -1.2 * np.log(np.arange(1, E + 1))
            logp[E - c["empty"]:] = -np.inf
            lg = lg + logp
        n.append(np.unique(np.argsort(-lg, 1)[:, :k]).size)
    return float(np.mean(n))


def work(case):
    c = case
    size = 2 if c["dtype"] == "bf16" else 4
    if c["kind"] == "moe":
        T, H, I, k = c["T"] - c["padded"], c["H"], c["I"], c["k"]
        weights = _experts_touched(c) * 3 * H * I * (0.5 + 1 / 16)
        return dict(bytes=weights + c["T"] * (2 * H * size + 4 * c["E"] + 8 * k),
                    flops=2.0 * T * k * 3 * H * I)
    T, V = c["T"], c["V"]
    if c["kind"] == "logprobs":
        return dict(bytes=T * V * size + T * (16 + 8 * c["top"]), flops=5.0 * T * V)
    return dict(bytes=2 * T * V * size + T * 24, flops=10.0 * T * V)


# ------------------------------------------------------------ definition
def _exact_weight(w, e):
    """W_e in 64 bits from the bit fields of its codes and scales."""
    codes, scales, ts = w
    c = codes[e]
    n = torch.stack([c & 15, c >> 4], -1).flatten(1).to(torch.int32)
    ex, man = (n >> 1) & 3, n & 1
    mag = torch.where(ex == 0, man.double() * 0.5,
                      torch.ldexp(1.0 + 0.5 * man.double(), ex - 1))
    b = scales[e].to(torch.int32)
    be, bm = (b >> 3) & 15, (b & 7).double() / 8
    blk = torch.where(be == 0, torch.ldexp(bm, torch.full_like(be, -6)),
                      torch.ldexp(1.0 + bm, be - 7))
    sign = 1.0 - 2.0 * ((n >> 3) & 1).double()
    return sign * mag * blk.repeat_interleave(16, 1) * ts[e].double()


def _exact_moe(s):
    lg, k, I = s["logits"].double(), s["k"], s["I"]
    T, E = lg.shape
    order = torch.sort(lg.cpu(), dim=1, descending=True, stable=True).indices[:, :k].to(lg.device)
    val = lg.gather(1, order)
    real = val[:, 0] > -math.inf
    wts = torch.zeros_like(val)
    wts[real] = torch.exp(val[real] - torch.logsumexp(lg[real], 1, keepdim=True))
    out = torch.zeros((T, s["H"]), dtype=torch.float64, device=lg.device)
    for e in torch.unique(order[wts > 0]).tolist():
        t, slot = torch.nonzero((order == e) & (wts > 0), as_tuple=True)
        y = s["x"][t].double() @ _exact_weight(s["gu"], e).T.contiguous()
        h = y[:, :I] * torch.sigmoid(y[:, :I]) * y[:, I:]
        out.index_add_(0, t, wts[t, slot][:, None] * (h @ _exact_weight(s["down"], e).T.contiguous()))
    return dict(out=out, topk_ids=None, topk_weights=wts)


def _exact_logits(s):
    z = s["logits"].detach().double()
    T, V = z.shape
    if s["inv_t"] is not None:
        z = z * s["inv_t"].double()[:, None]
    res = dict(logprobs=[], entropy=[], top=[], grad=[])
    for r0 in range(0, T, 512):
        r = slice(r0, min(T, r0 + 512))
        zr, tg = z[r], s["targets"][r]
        lse = torch.logsumexp(zr, 1, keepdim=True)
        gone = torch.isinf(lse)
        lp = torch.where(gone | (zr == -math.inf), torch.full_like(zr, -math.inf), zr - lse)
        p = torch.exp(lp)
        ent = -torch.special.xlogy(p, p).sum(1)
        at = lp.gather(1, tg.clamp(min=0)[:, None])[:, 0]
        res["logprobs"].append(torch.where(tg < 0, torch.zeros_like(at), at))
        res["entropy"].append(ent)
        if s["top"]:
            res["top"].append(torch.topk(lp, s["top"], 1).values)
        if s["kind"] == "train":
            a = torch.where((tg < 0) | gone[:, 0], torch.zeros_like(ent), s["g_logp"][r].double())
            one = torch.zeros_like(p)
            one.scatter_(1, tg.clamp(min=0)[:, None], 1.0)
            gr = a[:, None] * (one - p)
            gr -= s["g_ent"][r].double()[:, None] * (torch.special.xlogy(p, p) + p * ent[:, None])
            if s["inv_t"] is not None:
                gr = gr * s["inv_t"][r].double()[:, None]
            res["grad"].append(gr)
    out = dict(logprobs=torch.cat(res["logprobs"]), entropy=torch.cat(res["entropy"]))
    if s["kind"] == "train":
        out["grad"] = torch.cat(res["grad"])
    elif s["top"]:
        out["top_ids"] = None
        out["top_logprobs"] = torch.cat(res["top"])
    return out


def exact(case, seed):
    with torch.no_grad():
        return (_exact_moe if case["kind"] == "moe" else _exact_logits)(prepare(case, seed))
