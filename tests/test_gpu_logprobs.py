"""GPU tests of token_logprobs and its gradient against plain 64-bit
references: vocabularies of every alignment, masked and empty rows, ignored
and invalid targets, ties, strides, streams and graphs."""
import numpy as np
import pytest
import torch

from nvfp4_w4a4_moe_quant_amd import _lib as L
from nvfp4_w4a4_moe_quant_amd import pipeline as P
import decode_ref as R

pytestmark = pytest.mark.gpu
from gpu_util import DEV, eq, host, say, to_dev


def _case(seed, T, V, dtype, masked=0.0, temperature=True, ties=False, scale=3.0):
    g = np.random.default_rng(seed)
    z = (g.standard_normal((T, V)) * scale).astype(np.float32)
    z[np.arange(T), g.integers(0, V, T)] += 8
    if ties:
        z = np.round(z)
    if masked:
        z[g.random((T, V)) < masked] = -np.inf
    y = g.integers(0, V, T)
    inv_t = (1 / g.uniform(0.5, 2.0, T)).astype(np.float32) if temperature else None
    return to_dev_any(z, dtype), y, inv_t


def to_dev_any(z, dtype):
    t = torch.from_numpy(np.ascontiguousarray(z)).to(DEV)
    return t.to(torch.bfloat16) if dtype == "bf16" else t


def up(a):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def near(got, ref, tol, what):
    got = host(got).astype(np.float64)
    fin = np.isfinite(ref)
    np.testing.assert_array_equal(got[~fin], np.asarray(ref)[~fin], what)
    bad = ~(np.abs(got[fin] - ref[fin]) <= np.asarray(tol)[fin])
    assert not bad.any(), (what, got[fin][bad][:4], ref[fin][bad][:4], np.asarray(tol)[fin][bad][:4])


def check(z, y, inv_t, top_k, r=None):
    if r is None:
        r = L.token_logprobs(z, up(y), top_k=top_k, inv_temperature=up(inv_t))
    zs = host(z.float())
    ref = R.log_probs(zs, y, inv_t, top_k)
    near(r.logprobs, ref["logprobs"], ref["tol_logprobs"], "logprobs")
    near(r.entropy, ref["entropy"], ref["tol_entropy"], "entropy")
    nrm = host(r.norm).astype(np.float64)
    lse = nrm[:, 0] * (1.0 if inv_t is None else inv_t) + nrm[:, 1] * np.log(2)
    with np.errstate(invalid="ignore"):
        near_lse = np.abs(lse - ref["lse"]) <= ref["tol_lp"].min(1) + 8 * R.U32 * np.abs(ref["lse"])
    assert (near_lse | (lse == ref["lse"])).all()
    if top_k:
        eq(host(r.top_ids), ref["top_ids"], "top ids")
        near(r.top_logprobs, ref["top_logprobs"], ref["tol_top"], "top logprobs")
    return r, ref


VOCABS = [1, 2, 7, 32, 63, 64, 65, 255, 257, 1000, 1023, 4096, 4099, 8192, 16384, 16391, 32003,
          65536, 65537, 100003, 131072, 140001]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V", VOCABS)
def test_vocabularies(V, dtype):
    say(f"logprobs V={V} {dtype}")
    for T, top_k in ((1, min(V, 5)), (3, 0), (6, min(V, 32))):
        check(*_case(V + T, T, V, dtype), top_k)


@pytest.mark.parametrize("T", [1, 2, 15, 16, 17, 63, 64, 65, 300, 1030])
def test_row_counts(T):
    say(f"logprobs T={T}")
    for V in (1500, 33000):
        check(*_case(T + V, T, V, "bf16", temperature=T % 2 == 0), 4)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_ties_go_to_the_lower_index(dtype):
    say(f"logprobs ties {dtype}")
    for T, V in ((4, 40000), (70, 3000), (2, 131072)):
        check(*_case(V, T, V, dtype, ties=True), 32)
    z = torch.zeros((3, 70001), device=DEV, dtype=torch.bfloat16)
    z[1, 69000:] = 1
    z[2, ::2] = -0.0        # equal to +0
    check(z, np.array([0, 1, 2]), None, 32)
    # all alternatives inside one thread's share, then rising, then falling
    z = torch.arange(50000, device=DEV).float()[None] / 1e3
    check(torch.cat([z, -z]), np.array([49999, 0]), None, 32)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_masks(dtype):
    """Masked tokens, rows of nothing else, a masked target, fewer live tokens
    than alternatives."""
    say(f"logprobs masks {dtype}")
    for V in (300, 40001):
        z, y, it = _case(V, 12, V, dtype, masked=0.5)
        z[2] = float("-inf")
        z[3, 4:] = float("-inf")
        z[4, y[4]] = float("-inf")
        z[5, :] = float("-inf")
        z[5, V - 1] = 2.5
        z[6, :] = torch.finfo(z.dtype).min      # the type's lowest value is a number
        y[5], y[7], y[2] = V - 1, -100, 0
        r, _ = check(z, y, None, 8)
        assert host(r.logprobs)[2] == -np.inf and host(r.logprobs)[4] == -np.inf
        assert host(r.logprobs)[5] == 0 and host(r.entropy)[5] == 0
        assert list(host(r.top_ids)[2]) == list(range(8))
        check(z, y, it, 8)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_masks_of_the_lowest_value(dtype):
    """Tokens masked with the type's lowest number instead of -inf, some rows
    with fewer live tokens than alternatives."""
    say(f"logprobs masked by the lowest value {dtype}")
    for V in (700, 40001, 131072):
        z, y, _ = _case(V + 1, 6, V, dtype)
        low = torch.finfo(z.dtype).min
        z[torch.rand(6, V, device=DEV, generator=torch.Generator(device=DEV).manual_seed(V)) < 0.6] = low
        z[2, 3:] = low
        z[3, 1:] = float("-inf")
        z[4, y[4]] = low
        check(z, y, None, 8)
        check(z, y, np.array([1, .5, .25, 1, .75, 1], np.float32), 8)
        r = L.token_logprobs(z, up(y))
        g = L.token_logprobs_backward(z, up(y), r.norm, r.entropy, torch.ones(6, device=DEV),
                                      torch.ones(6, device=DEV))
        want, tol = R.log_probs_grad(R.log_probs(host(z.float()), y, None, 0), y, None, np.ones(6),
                                     np.ones(6), dtype)
        near(g.float(), want, tol, "gradient")


def test_ignored_rows_are_not_read():
    """Ignored positions without an entropy gradient get a gradient of 0 even
    where their logits are NaN; the other rows are what they are alone."""
    say("logprobs gradient of ignored rows")
    for V in (77, 5000):
        z, y, _ = _case(V, 5, V, "bf16")
        y[1], y[3] = -100, -1
        z[1], z[3, 5] = float("nan"), float("inf")
        r = L.token_logprobs(z, up(y))
        ga = torch.randn(5, device=DEV)
        g = L.token_logprobs_backward(z, up(y), r.norm, None, ga)
        assert (g[[1, 3]] == 0).all() and (r.logprobs[[1, 3]] == 0).all()
        keep = [0, 2, 4]
        alone = L.token_logprobs_backward(z[keep].contiguous(), up(y[keep]),
                                          r.norm[keep].contiguous(), None, ga[keep])
        assert torch.equal(g[keep], alone) and torch.isfinite(alone).all()
        odd = torch.full((5, V + 1), 7.0, dtype=z.dtype, device=DEV)
        L.token_logprobs_backward(z, up(y), r.norm, None, ga, out=odd[:, 1:])
        assert torch.equal(odd[:, 1:], g) and (odd[:, 0] == 7).all()


def test_invalid_targets_and_numbers():
    say("logprobs: targets outside the vocabulary, NaN and inf logits")
    z, y, _ = _case(3, 6, 5000, "f32")
    y[0], y[1], y[2] = 5000, 2 ** 40, -(2 ** 40)
    z[3, 17], z[4, 99] = float("nan"), float("inf")
    r = L.token_logprobs(z, up(y), top_k=3)
    lp, ent = host(r.logprobs), host(r.entropy)
    assert np.isnan(lp[[0, 1, 3, 4]]).all() and lp[2] == 0 and np.isnan(ent[[3, 4]]).all()
    check(z[5:], y[5:], None, 3)
    assert (host(r.top_ids)[3] != 17).all() and host(r.top_ids)[4, 0] == 99
    g = L.token_logprobs_backward(z, up(y), r.norm, r.entropy, torch.ones(6, device=DEV))
    assert torch.isnan(g[[0, 1]]).all() and (g[2] == 0).all() and torch.isfinite(g[5]).all()


def test_large_logits_and_temperatures():
    say("logprobs: large logits, sharp and flat temperatures")
    z, y, _ = _case(4, 8, 9000, "f32", scale=300.0)
    check(z, y, np.array([1e-3, 1e-2, .1, 1, 2, 8, 50, 100], np.float32), 6)


def test_no_targets_and_no_rows():
    say("logprobs without targets; T = 0")
    z, _, _ = _case(5, 4, 777, "bf16")
    r = L.token_logprobs(z, top_k=2)
    ref = R.log_probs(host(z.float()), None, None, 2)
    assert r.logprobs is None
    near(r.entropy, ref["entropy"], ref["tol_entropy"], "entropy")
    r = L.token_logprobs(z[:0], torch.empty(0, dtype=torch.int64, device=DEV), top_k=2)
    assert r.logprobs.shape == (0,) and r.top_ids.shape == (0, 2)
    g = L.token_logprobs_backward(z[:0], None, r.norm, r.entropy, None, r.entropy)
    assert g.shape == (0, 777)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("pad,off", [(0, 0), (1, 0), (3, 1), (8, 0), (5, 2), (16, 7)])
def test_strides(pad, off, dtype):
    """Rows that start at any element of a wider buffer."""
    say(f"logprobs strides pad={pad} off={off} {dtype}")
    for V in (4099, 33000):
        z, y, it = _case(V + pad, 5, V, dtype)
        big = torch.full((5, V + pad + off), float("nan"), dtype=z.dtype, device=DEV)
        big[:, off:off + V] = z
        v = big[:, off:off + V]
        a = L.token_logprobs(v, up(y), top_k=9, inv_temperature=up(it))
        check(z, y, it, 9, a)
        ga, gb = torch.randn(5, device=DEV), torch.randn(5, device=DEV)
        ref = L.token_logprobs_backward(z, up(y), a.norm, a.entropy, ga, gb, inv_temperature=up(it))
        out = torch.full_like(big, 7.0)
        L.token_logprobs_backward(v, up(y), a.norm, a.entropy, ga, gb, inv_temperature=up(it),
                                  out=out[:, off:off + V])
        assert torch.equal(out[:, off:off + V], ref)
        out[:, off:off + V] = 7.0
        assert (out == 7.0).all()
        L.token_logprobs_backward(v, up(y), a.norm, a.entropy, ga, gb, inv_temperature=up(it), out=v)
        assert torch.equal(v, ref)     # in place


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,V", [(1, 1), (3, 7), (5, 1000), (4, 32003), (2, 131072), (70, 257)])
def test_gradient(T, V, dtype):
    say(f"logprobs gradient T={T} V={V} {dtype}")
    z, y, it = _case(T * V, T, V, dtype, masked=0.2 if V > 20 else 0.0)
    if T > 2:
        y[1] = -1
        if V > 20:
            z[2] = float("-inf")
    g = np.random.default_rng(9)
    ga, gb = (g.standard_normal(T).astype(np.float32) for _ in range(2))
    for a, b, inv in ((ga, gb, it), (ga, None, None), (None, gb, it)):
        r = L.token_logprobs(z, up(y), inv_temperature=up(inv))
        got = L.token_logprobs_backward(z, up(y) if a is not None else None, r.norm, r.entropy,
                                        up(a), up(b), inv_temperature=up(inv))
        ref = R.log_probs(host(z.float()), y, inv, 0)
        want, tol = R.log_probs_grad(ref, y, inv, a, b, dtype)
        near(got.float(), want, tol, "gradient")


def test_autograd_matches_the_call_and_differences():
    """pipeline.token_logprobs under autograd, against the library call, and
    against central differences of the 64-bit reference (step 2^-10, whose
    truncation and rounding are below 1e-5 for values of this size)."""
    say("logprobs autograd")
    z, y, it = _case(8, 4, 50, "f32")
    y[1] = -100
    z.requires_grad_()
    lp, ent = P.token_logprobs(z, up(y), up(it))
    g = np.random.default_rng(2)
    ga, gb = (g.standard_normal(4).astype(np.float32) for _ in range(2))
    (lp * up(ga) + ent * up(gb)).sum().backward()
    r = L.token_logprobs(z.detach(), up(y), inv_temperature=up(it))
    assert torch.equal(z.grad, L.token_logprobs_backward(z.detach(), up(y), r.norm, r.entropy,
                                                         up(ga), up(gb), inv_temperature=up(it)))
    zs = host(z.detach()).astype(np.float64)
    eps = 2.0 ** -10

    def f(zz):
        q = R.log_probs(zz, y, it, 0)
        return q["logprobs"] * ga + q["entropy"] * gb
    num = np.zeros_like(zs)
    for j in range(50):
        d = np.zeros_like(zs)
        d[:, j] = eps
        num[:, j] = (f(zs + d) - f(zs - d)) / (2 * eps)
    assert np.abs(host(z.grad) - num).max() < 1e-5
    # one of the two outputs unused, and neither needed
    z2 = z.detach().clone().requires_grad_()
    P.token_logprobs(z2, up(y))[1].sum().backward()
    assert torch.isfinite(z2.grad).all()
    assert not P.token_logprobs(z.detach(), up(y))[0].requires_grad


def test_rows_beyond_32_bit_offsets():
    say("logprobs: 16500 x 131072 bf16")
    T, V = 16500, 131072
    z = torch.empty((T, V), dtype=torch.bfloat16, device=DEV)
    z.normal_(generator=torch.Generator(device=DEV).manual_seed(1))
    y = np.random.default_rng(1).integers(0, V, T)
    r = L.token_logprobs(z, up(y), top_k=4)
    rows = [0, 1, 16383, 16384, 16385, T - 1]
    sub = L.LogprobsOut(r.logprobs[rows], r.entropy[rows], r.norm[rows], r.top_ids[rows],
                        r.top_logprobs[rows])
    zr = z[rows].clone()
    check(zr, y[rows], None, 4, sub)
    ga = torch.ones(T, device=DEV)
    want = L.token_logprobs_backward(zr, up(y[rows]), sub.norm, sub.entropy, ga[rows])
    L.token_logprobs_backward(z, up(y), r.norm, r.entropy, ga, out=z)
    assert torch.equal(z[rows], want)


def test_more_rows_than_a_grid_dimension():
    """70001 short rows: past the 65535 of a grid's second dimension."""
    say("logprobs: 70001 x 33")
    T, V = 70001, 33
    z, y, it = _case(12, T, V, "bf16")
    r, ref = check(z, y, it, 2)
    ga = np.random.default_rng(3).standard_normal(T).astype(np.float32)
    g = L.token_logprobs_backward(z, up(y), r.norm, r.entropy, up(ga), up(ga[::-1]),
                                  inv_temperature=up(it))
    want, tol = R.log_probs_grad(ref, y, it, ga, ga[::-1], "bf16")
    near(g.float(), want, tol, "gradient")


@pytest.mark.parametrize("off", [0, 3])
def test_gradient_larger_than_the_caches(off):
    """1300 x 65537 bf16 (170 MB), whose gradient takes another way to memory
    than one of a few rows does: the same bits, ignored rows, aligned or not,
    in place or not."""
    say(f"logprobs gradient 1300 x 65537 off={off}")
    T, V = 1300, 65537
    big = torch.empty((T, V + 7 + off), dtype=torch.bfloat16, device=DEV)
    big.normal_(generator=torch.Generator(device=DEV).manual_seed(off))
    z = big[:, off:off + V]
    y = torch.from_numpy(np.random.default_rng(off).integers(-V // 4, V, T)).to(DEV)
    y[y < 0] = -100
    r = L.token_logprobs(z, y)
    ga = torch.randn(T, device=DEV)
    parts = [L.token_logprobs_backward(z[i:i + 100], y[i:i + 100], r.norm[i:i + 100], None,
                                       ga[i:i + 100]) for i in range(0, T, 100)]
    want = torch.cat(parts)
    same = torch.full_like(big, 7.0)
    L.token_logprobs_backward(z, y, r.norm, None, ga, out=same[:, off:off + V])
    assert torch.equal(same[:, off:off + V], want)
    same[:, off:off + V] = 7.0
    assert (same == 7.0).all()
    L.token_logprobs_backward(z, y, r.norm, None, ga, out=z)
    assert torch.equal(z, want)


def test_one_long_row():
    """A row of 2^24 + 9 tokens in 64 parts, at an odd address."""
    say("logprobs: 1 x 16777225")
    V = 2 ** 24 + 9
    z = torch.empty(V + 3, dtype=torch.bfloat16, device=DEV)
    z.normal_(generator=torch.Generator(device=DEV).manual_seed(4))
    z = z[3:].view(1, V)
    z[0, V - 2] = 9.0
    y = np.array([V - 1])
    r, _ = check(z, y, None, 20)
    assert int(r.top_ids[0, 0]) == V - 2


def test_repeatable_on_streams_and_graphs():
    say("logprobs: streams and graphs")
    cases = [_case(40 + i, 9, 40000, "bf16") for i in range(3)]
    ga = torch.randn(9, device=DEV)

    def step(z, y, it):
        r = L.token_logprobs(z, y, top_k=6, inv_temperature=it)
        g = L.token_logprobs_backward(z, y, r.norm, r.entropy, ga, ga, inv_temperature=it)
        return [r.logprobs, r.entropy, r.top_ids, r.top_logprobs, g]
    cases = [(z, up(y), up(it)) for z, y, it in cases]
    ref = [[t.clone() for t in step(*c)] for c in cases]
    same = lambda a, b: all(torch.equal(u, v) for u, v in zip(a, b))  # noqa: E731
    torch.cuda.synchronize()
    got = []
    for c in cases:
        with torch.cuda.stream(torch.cuda.Stream()):
            got.append([step(*c) for _ in range(3)])
    torch.cuda.synchronize()
    assert all(same(s, r) for steps, r in zip(got, ref) for s in steps)
    bufs = [[t.clone() for t in cases[0]], [t.clone() for t in cases[1]]]
    graphs = []
    for b in bufs:
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            o = step(*b)
        graphs.append((gr, o))
    for rep in range(4):
        n = rep % 3
        for d, s in zip(bufs[0], cases[n]):
            d.copy_(s)
        graphs[1][0].replay()
        graphs[0][0].replay()
        step(*cases[2])
        torch.cuda.synchronize()
        assert same(graphs[0][1], ref[n]) and same(graphs[1][1], ref[1])


@pytest.mark.parametrize("dtype,T", [("bf16", 2064), ("f32", 1032)])
def test_logits_larger_than_the_caches(dtype, T):
    """270 MB of logits with alternatives, read another way than a few rows
    are: the same bits."""
    say(f"logprobs {T} x 65539 {dtype}")
    V = 65539
    z = torch.empty((T, V), dtype=torch.float32 if dtype == "f32" else torch.bfloat16, device=DEV)
    z.normal_(generator=torch.Generator(device=DEV).manual_seed(8))
    y = torch.from_numpy(np.random.default_rng(8).integers(0, V, T)).to(DEV)
    it = torch.full((T,), 0.75, device=DEV)
    r = L.token_logprobs(z, y, top_k=5, inv_temperature=it)
    n = T // 4
    parts = [L.token_logprobs(z[i:i + n], y[i:i + n], top_k=5, inv_temperature=it[i:i + n])
             for i in range(0, T, n)]
    for k in range(5):
        assert torch.equal(r[k], torch.cat([p[k] for p in parts])), k
    rows = [0, 1, T - 1]
    check(z[rows].clone(), host(y[rows]), host(it[rows]), 5,
          L.LogprobsOut(*(t[rows] for t in r)))
