"""GPU tests of nvfp4_moe_decode against a plain 64-bit reference: sizes that
are not multiples of the kernels' tiles, more than 16 rows of one expert,
masked and NaN logits, padded rows, strides, magnitudes, streams and graphs."""
import numpy as np
import pytest
import torch

from nvfp4_w4a4_moe_quant_amd import _lib as L
from nvfp4_w4a4_moe_quant_amd import datagen as D
from nvfp4_w4a4_moe_quant_amd import pipeline as P
import decode_ref as R

pytestmark = pytest.mark.gpu
from gpu_util import DEV, eq, host, say, to_dev


class Layer:
    """Random NVFP4 expert weights on the GPU and their exact values."""

    def __init__(self, seed, E, H, I):
        g = np.random.default_rng(seed)
        self.E, self.H, self.I = E, H, I
        self.q = {}
        for name, N, K in (("gu", 2 * I, H), ("down", H, I)):
            codes = g.integers(0, 256, (E, N, K // 2), dtype=np.uint8)
            scales = g.integers(0x20, 0x50, (E, N, K // 16), dtype=np.uint8)
            scales[g.random(scales.shape) < 0.05] = 0          # blocks of zero
            scales[g.random(scales.shape) < 0.02] = 0x7E       # and the largest scale
            ts = (g.uniform(0.5, 2.0, E) / (8.0 * np.sqrt(K))).astype(np.float32)
            self.q[name] = (codes, scales, ts)
        self.cache = {}
        up = lambda n: L.NVFP4(*(torch.from_numpy(a).to(DEV) for a in self.q[n]))  # noqa: E731
        self.wgu = P.QuantWeights(up("gu"), 2 * I, H)
        self.wd = P.QuantWeights(up("down"), H, I)

    def exact(self, name):
        def get(e):
            if (name, e) not in self.cache:
                c, s, t = self.q[name]
                self.cache[name, e] = (R.dequantize(c[e], s[e]), float(t[e]))
            return self.cache[name, e]
        return get

    def __call__(self, x, lg, k, **kw):
        return P.moe_decode(x, lg, self.wgu, self.wd, k, **kw)

    def check(self, r, x, lg, k, dtype):
        """Against the reference; x and lg as the kernel saw them."""
        xs, ls = host(x.float()), host(lg)
        ids, w, out, tol = R.moe_layer(xs, ls, self.exact("gu"), self.exact("down"), k, dtype)
        eq(host(r.topk_ids), ids, "ids")
        np.testing.assert_allclose(host(r.topk_weights), w, rtol=2.0 ** -20, atol=1e-37)
        got = host(r.out.float()).astype(np.float64)
        bad = ~(np.abs(got - out) <= tol)
        assert not bad.any(), (np.argwhere(bad)[:4], got[bad][:4], out[bad][:4], tol[bad][:4])


def _inputs(seed, T, E, H, dtype):
    g = np.random.default_rng(seed)
    x = g.standard_t(3, (T, H)).astype(np.float32)
    x[:, g.integers(0, H, 3)] *= 20
    return to_dev(x, dtype), torch.from_numpy(g.standard_normal((T, E)).astype(np.float32)).to(DEV)


SIZES = [  # T, E, k, H, I
    (1, 8, 2, 256, 128), (1, 2, 1, 32, 32), (2, 4, 4, 1056, 416), (3, 60, 4, 1056, 416),
    (7, 5, 3, 2080, 96), (16, 16, 8, 32, 32), (16, 1, 1, 160, 64), (17, 130, 16, 512, 96),
    (5, 1024, 16, 64, 32), (33, 3, 2, 96, 160), (64, 8, 2, 96, 160), (64, 1, 1, 64, 32),
    (64, 128, 8, 512, 256), (2, 4, 2, 7168, 64), (1, 3, 2, 64, 2048), (4, 2, 2, 4128, 2080),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,E,k,H,I", SIZES)
def test_sizes(T, E, k, H, I, dtype):
    say(f"moe decode T={T} E={E} k={k} H={H} I={I} {dtype}")
    lay = Layer(T + H, E, H, I)
    x, lg = _inputs(T * 3 + E, T, E, H, dtype)
    lay.check(lay(x, lg, k), x, lg, k, dtype)


def test_every_token_count():
    say("moe decode T = 0 .. 64")
    lay = Layer(5, 12, 96, 64)
    for T in list(range(0, 20)) + [31, 32, 33, 47, 48, 49, 63]:
        x, lg = _inputs(T, T, 12, 96, "bf16")
        r = lay(x, lg, 3)
        assert r.out.shape == (T, 96)
        if T:
            lay.check(r, x, lg, 3, "bf16")


def test_all_tokens_on_the_same_experts():
    say("moe decode: 64 rows of one expert, and ties")
    lay = Layer(6, 9, 160, 96)
    x, _ = _inputs(1, 64, 9, 160, "bf16")
    lg = torch.zeros((64, 9), device=DEV)          # all tied: experts 0 .. k-1
    r = lay(x, lg, 4)
    assert (host(r.topk_ids) == np.arange(4)).all()
    lay.check(r, x, lg, 4, "bf16")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_masked_logits_and_padded_rows(dtype):
    """Rows of -inf give 0 and their x is not read; fewer finite logits than k
    fill up with weight 0; NaN logits rank as -inf."""
    say(f"moe decode masks {dtype}")
    lay = Layer(7, 10, 128, 64)
    x, lg = _inputs(2, 21, 10, 128, dtype)
    inf = float("inf")
    lg[3] = -inf
    lg[20] = -inf
    lg[4, 2:] = -inf
    lg[5, 1:] = float("nan")
    lg[6] = float("nan")
    lg[7, ::2] = -inf
    x[3], x[20] = float("nan"), inf
    r = lay(x, lg, 4)
    assert (r.out[[3, 6, 20]] == 0).all() and (r.topk_weights[[3, 6, 20]] == 0).all()
    assert torch.isfinite(r.out).all()
    xs = x.clone()
    xs[3], xs[20] = 0, 0
    lay.check(r, xs, lg, 4, dtype)


def test_non_finite_rows_stay_in_their_rows():
    say("moe decode: NaN and inf in one row of x")
    lay = Layer(8, 6, 96, 64)
    x, lg = _inputs(3, 12, 6, 96, "bf16")
    ref = lay(x, lg, 2).out.clone()
    x[5, 7], x[8, 1] = float("nan"), float("inf")
    got = lay(x, lg, 2).out
    keep = [i for i in range(12) if i not in (5, 8)]
    assert torch.equal(got[keep], ref[keep])
    assert torch.isnan(got[5]).all() and not torch.isfinite(got[8]).any()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_magnitudes(dtype):
    """Rows of very different size, a zero row, and one value far above the
    rest of its row."""
    say(f"moe decode magnitudes {dtype}")
    lay = Layer(9, 4, 288, 96)
    x, lg = _inputs(4, 8, 4, 288, dtype)
    for row, f in enumerate((1e-18, 1e-9, 1e-4, 1.0, 1e4, 1e8)):
        x[row] *= f
    x[6] = 0
    x[7, 11] = 3e6
    lay.check(lay(x, lg, 2), x, lg, 2, dtype)


def test_strides_and_guards():
    """Row strides of x, logits and out; nothing outside out's rows is written."""
    say("moe decode strides")
    lay = Layer(10, 12, 96, 64)
    x, lg = _inputs(5, 9, 12, 96, "bf16")
    ref = lay(x, lg, 3)
    xb = torch.full((9, 96 + 40), float("nan"), dtype=torch.bfloat16, device=DEV)
    lb = torch.full((9, 12 + 5), 1e30, device=DEV)
    ob = torch.full((11, 96 + 8), 7.0, dtype=torch.bfloat16, device=DEV)
    xb[:, :96], lb[:, :12] = x, lg
    r = lay(xb[:, :96], lb[:, :12], 3, out=ob[1:10, :96])
    assert torch.equal(ob[1:10, :96], ref.out) and torch.equal(r.topk_ids, ref.topk_ids)
    ob[1:10, :96] = 7.0
    assert (ob == 7.0).all()


def test_weights_beyond_32_bit_offsets():
    say("moe decode: 5 GB of gate/up codes")
    E, H, I = 600, 2048, 4096
    g = torch.Generator(device=DEV)
    g.manual_seed(3)
    q = {}
    for name, N, K in (("gu", 2 * I, H), ("down", H, I)):
        q[name] = L.NVFP4(
            torch.randint(0, 256, (E, N, K // 2), dtype=torch.uint8, device=DEV, generator=g),
            torch.randint(0x20, 0x50, (E, N, K // 16), dtype=torch.uint8, device=DEV, generator=g),
            torch.full((E,), 1 / (8.0 * K ** 0.5), device=DEV))
    assert q["gu"].codes.numel() > 2 ** 32
    lg = torch.zeros((2, E), device=DEV)
    lg[0, E - 1], lg[0, 0], lg[1, E - 1], lg[1, 40] = 5, 4, 5, 4
    x, _ = _inputs(6, 2, E, H, "bf16")
    r = L.nvfp4_moe_decode(x, lg, q["gu"], q["down"], 2)

    def exact(name):
        return lambda e: (R.dequantize(host(q[name].codes[e]), host(q[name].scales[e])),
                          float(q[name].tscale[e]))
    ids, w, out, tol = R.moe_layer(host(x.float()), host(lg), exact("gu"), exact("down"), 2, "bf16")
    eq(host(r.topk_ids), ids, "ids")
    assert (np.abs(host(r.out.float()) - out) <= tol).all()


def test_routing_agrees_with_moe_route():
    say("moe decode routing vs moe_route")
    lay = Layer(11, 33, 64, 32)
    x, lg = _inputs(7, 40, 33, 64, "bf16")
    r, rt = lay(x, lg, 8), L.moe_route(lg, 8)
    eq(host(r.topk_ids), host(rt.topk_ids), "ids")
    np.testing.assert_allclose(host(r.topk_weights), host(rt.topk_weights), rtol=2.0 ** -20)


def test_repeatable_on_streams_and_graphs():
    """The same bits from two calls, from a side stream, from two calls at
    once, and from two captured graphs replayed with eager work between."""
    say("moe decode: streams and graphs")
    lay = Layer(12, 24, 512, 192)
    xs = [_inputs(20 + i, 12, 24, 512, "bf16") for i in range(3)]
    ref = [lay(x, lg, 4) for x, lg in xs]
    ref = [(r.out.clone(), r.topk_ids.clone()) for r in ref]
    for (x, lg), (o, i) in zip(xs, ref):
        r = lay(x, lg, 4)
        assert torch.equal(r.out, o) and torch.equal(r.topk_ids, i)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = []
    for st, (x, lg) in zip(streams, xs):
        with torch.cuda.stream(st):
            got.append([lay(x, lg, 4).out for _ in range(4)])
    torch.cuda.synchronize()
    for outs, (o, _) in zip(got, ref):
        assert all(torch.equal(a, o) for a in outs)
    x, lg = xs[0][0].clone(), xs[0][1].clone()
    x2, lg2 = xs[1][0].clone(), xs[1][1].clone()
    graphs = []
    for a, b in ((x, lg), (x2, lg2)):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            o = lay(a, b, 4).out
        graphs.append((gr, o))
    for rep in range(4):
        n = rep % 3
        x.copy_(xs[n][0])
        lg.copy_(xs[n][1])
        graphs[1][0].replay()
        graphs[0][0].replay()
        lay(*xs[2], 4)
        torch.cuda.synchronize()
        assert torch.equal(graphs[0][1], ref[n][0]) and torch.equal(graphs[1][1], ref[1][0])


def test_layer_near_the_bf16_trainer():
    """The layer against the trainer's own forward: qdq weights and bf16
    matmuls in torch (which round y and h to bf16 and sum in another order)."""
    say("moe decode vs fake-quantized trainer forward")
    rng = np.random.default_rng(3)
    E, H, I, T, k = 6, 256, 128, 10, 2
    mats = {n: [to_dev((rng.standard_normal((N, K)) * 0.02).astype(np.float32), "bf16")
                for _ in range(E)] for n, N, K in (("gu", 2 * I, H), ("down", H, I))}
    wgu = P.quantize_weights(enumerate(mats["gu"]), E, 2 * I, H, DEV)
    wd = P.quantize_weights(enumerate(mats["down"]), E, H, I, DEV)
    x, lg = _inputs(8, T, E, H, "bf16")
    r = P.moe_decode(x, lg, wgu, wd, k)
    out = torch.zeros((T, H), device=DEV)
    for t in range(T):
        for s in range(k):
            e = int(r.topk_ids[t, s])
            y = L.nvfp4_qdq(mats["gu"][e], out_dtype=torch.float32) @ x[t].float()
            h = torch.nn.functional.silu(y[:I]) * y[I:]
            out[t] += r.topk_weights[t, s] * (L.nvfp4_qdq(mats["down"][e], out_dtype=torch.float32) @ h)
    d = (r.out.float() - out).norm() / out.norm()
    assert d <= 2.0 ** -8, float(d)  # one bf16 rounding of the output bounds the rest
