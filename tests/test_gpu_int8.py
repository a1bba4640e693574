"""GPU tests of the INT8 rows and grouped products: codes, scales, FP32 and
bf16 products bit for bit against the 64-bit reference, SiLU*mul within a
derived bound; ragged sizes, groups of every length, strides, streams, graphs."""
import numpy as np
import pytest
import torch

from nvfp4_w4a4_moe_quant_amd import _lib as L
from nvfp4_w4a4_moe_quant_amd import datagen as D
from nvfp4_w4a4_moe_quant_amd import logprob_gap
from nvfp4_w4a4_moe_quant_amd import pipeline as P
import int8_ref as R

pytestmark = pytest.mark.gpu
from gpu_util import DEV, eq, host, say, to_dev

EPIS = {"f32": L.NVFP4_EPI_F32, "bf16": L.NVFP4_EPI_BF16, "silu": L.NVFP4_EPI_SILU_MUL_BF16}


def up(a):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def rows_of(rng, rows, K, dtype):
    x = (rng.standard_normal((rows, K)) * np.exp(rng.uniform(-3, 3, (rows, 1)))).astype(np.float32)
    x[:, rng.integers(0, K, max(1, K // 100))] *= 20
    if rows > 4:
        x[0] = 0
        x[1] = np.linspace(-127, 127, K).astype(np.float32)   # halves among the quotients
        x[2] = 1e-42                                          # subnormal
        x[3, K // 2] = 1e30                                   # one outlier
    return D.bf16_to_f32(D.bf16_bits(x)) if dtype == "bf16" else x


def weights_of(rng, G, N, K):
    w = rng.integers(-127, 128, (G, N, K)).astype(np.int8)
    return w, (rng.random((G, N)) * 1e-3 + 1e-4).astype(np.float32)


def offsets_of(rng, sizes):
    return np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)


def check_out(got, y, epi):
    if epi == "f32":
        eq(host(got).view(np.int32), y.view(np.int32), "FP32 product")
    elif epi == "bf16":
        eq(host(got.float()).view(np.int32), R.bf16(y).view(np.int32), "bf16 product")
    else:
        h, tol = R.silu_mul(y)
        v = host(got.float()).astype(np.float64)
        with np.errstate(invalid="ignore"):
            bad = ~(np.abs(v - h) <= tol)
        bad &= ~((np.abs(h) > 3.38e38) & np.isinf(v) & (np.sign(v) == np.sign(h)))   # beyond bf16's range
        assert not bad.any(), f"{bad.sum()} of {bad.size} beyond the bound, first {np.argwhere(bad)[:4].tolist()}"


def run(seed, sizes, N, K, epi, gather=False, dtype="bf16", given="x", src=None):
    rng = np.random.default_rng(seed)
    off = offsets_of(rng, sizes)
    total = int(off[-1])
    src = src or (max(1, total // 3) if gather else total)
    x = rows_of(rng, src, K, dtype)
    w, sw = weights_of(rng, len(sizes), N, K)
    gat = rng.integers(0, src, total).astype(np.int32) if gather else None
    a, sa = R.quantize(x)
    y = R.product(a, sa, w, sw, off, gat)
    act = to_dev(x, dtype) if given == "x" else L.INT8(up(a), up(sa))
    out = L.int8_grouped_gemm(act, L.INT8(up(w), up(sw)), up(off), N=N, K=K, total_rows=total,
                              gather_rows=up(gat), epilogue=EPIS[epi], validate=True)
    check_out(out, y, epi)


@pytest.mark.parametrize("rows,K,dtype", [
    (1, 16, "f32"), (1, 32, "bf16"), (7, 48, "bf16"), (1000, 768, "bf16"), (257, 2048, "f32"),
    (33, 4112, "f32"), (5, 7168, "bf16"), (3, 16384, "bf16"), (6, 8208, "f32"), (1, 131056, "bf16"),
    (2, 65536, "f32"), (4099, 1040, "bf16"), (20000, 64, "f32")])
def test_rows(rows, K, dtype):
    say(f"int8 rows {rows}x{K} {dtype}")
    rng = np.random.default_rng(rows + K)
    x = rows_of(rng, rows, K, dtype)
    q = L.int8_quantize_rows(to_dev(x, dtype))
    codes, scales = R.quantize(x)
    eq(host(q.scales).view(np.int32), scales.view(np.int32), "scales")
    eq(host(q.codes), codes, "codes")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_with_infinities(dtype):
    say(f"int8 rows, not finite, {dtype}")
    rng = np.random.default_rng(9)
    for K in (32, 1024, 7168, 20000):
        K -= K % 16
        x = rows_of(rng, 9, K, dtype)
        x[4, 3], x[5, K - 1], x[6, 0], x[7] = np.nan, np.inf, -np.inf, np.nan
        q = L.int8_quantize_rows(to_dev(x, dtype))
        codes, scales = R.quantize(x)
        s = host(q.scales)
        eq(np.isnan(s), np.isnan(scales), "rows not finite")
        eq(s[~np.isnan(s)], scales[~np.isnan(s)], "scales")
        eq(host(q.codes), codes, "codes")


def test_rows_strided_and_given_out():
    say("int8 rows, strided")
    rng = np.random.default_rng(2)
    x = rows_of(rng, 37, 96, "bf16")
    big = torch.full((37, 200), 9e9, device=DEV, dtype=torch.bfloat16)
    big[:, 8:104] = to_dev(x, "bf16")
    buf = L.INT8(torch.empty(37, 96, dtype=torch.int8, device=DEV), torch.empty(37, device=DEV))
    q = L.int8_quantize_rows(big[:, 8:104], out=buf)
    codes, scales = R.quantize(x)
    assert q.codes.data_ptr() == buf.codes.data_ptr()
    eq(host(q.codes), codes, "codes")
    eq(host(q.scales), scales, "scales")
    with pytest.raises(L.NVFP4Error):
        L.int8_quantize_rows(big[:, 1:97])                 # 2-byte alignment
    with pytest.raises(ValueError):
        L.int8_quantize_rows(big.t())
    with pytest.raises(ValueError):
        L.int8_quantize_rows(big[:, 8:104], out=L.INT8(buf.codes[:, :80], buf.scales))
    assert L.int8_quantize_rows(big[:0, 8:104]).codes.shape == (0, 96)


DENSE = [(1, 16, 16), (1, 1, 32), (1, 4096, 4096), (2, 100, 48), (3, 65, 64), (7, 384, 1024),
         (16, 512, 2048), (17, 130, 1040), (31, 96, 7168), (33, 250, 80), (64, 1999, 512),
         (65, 256, 128), (100, 255, 272), (128, 384, 384), (200, 1000, 1056), (256, 512, 640),
         (300, 260, 4112), (700, 1028, 208), (2300, 512, 256), (1, 128, 131056), (70, 1030, 4112), (100, 2048, 7168),
         (129, 384, 8192), (200, 67, 16384), (65, 128, 131056), (300, 1024, 4096)]


@pytest.mark.parametrize("rows,N,K", DENSE)
def test_dense(rows, N, K):
    say(f"int8 dense {rows}x{N}x{K}")
    for i, (epi, given, dtype) in enumerate([("f32", "x", "bf16"), ("bf16", "q", "f32"),
                                             ("silu", "x", "f32")]):
        run(rows + N + K, [rows], N + (N & 1 if epi == "silu" else 0), K, epi, given=given,
            dtype=dtype)


GROUPS = [
    (0, [0, 0, 3, 0], 64, 64), (1, [1] * 8, 256, 512), (2, [5, 0, 17, 1, 33], 130, 80),
    (3, [0], 32, 48), (4, [64, 0, 1, 200, 16], 384, 256), (5, [2] * 70, 96, 208),
    (6, [300, 12], 514, 1040), (7, [0] * 63 + [9] + [0] * 64 + [20], 64, 128),
    (8, [1000, 0, 600, 24], 768, 320), (9, [30] * 40, 256, 2048), (10, [0, 2, 1, 0, 4] * 60, 48, 96),
    (18, [20] * 300, 64, 64), (19, ([0] * 9 + [2]) * 100, 2050, 48), (20, ([0] * 30 + [41]) * 33, 130, 80),
    (13, [256, 240, 288, 250, 230], 300, 1104), (14, [1200, 0, 0, 0, 50], 514, 400),
    (15, [100, 64, 0, 65, 128, 33], 270, 1104), (16, [200, 190, 129], 258, 1136),
    (17, [321, 200, 33], 260, 272), (11, [15, 16, 17, 31, 32, 33, 47, 48, 49], 320, 624), (12, [127, 128, 129, 255, 256, 257], 260, 176),
]


@pytest.mark.parametrize("seed,sizes,N,K", GROUPS)
def test_grouped(seed, sizes, N, K):
    say(f"int8 grouped {seed}: {len(sizes)} groups, N={N} K={K}")
    run(seed, sizes, N, K, "silu", gather=True)
    run(seed + 50, sizes, N, K, "f32", given="q")
    run(seed + 90, sizes, N, K, "bf16", gather=True, dtype="f32", given="x")
    run(seed + 70, sizes, N, K, "f32", dtype="bf16")


@pytest.mark.parametrize("T", [1, 2, 4, 16])
def test_few_tokens_of_many_experts(T):
    say(f"int8 decode {T} tokens")
    rng = np.random.default_rng(T)
    E, k, H, I = 128, 8, 2048, 768
    ids = np.argsort(rng.standard_normal((T, E)), 1)[:, :k]
    sizes = np.bincount(ids.ravel(), minlength=E)
    run(T, sizes, 2 * I, H, "silu", gather=True, src=T)
    run(T, sizes, H, I, "f32")


def test_rows_that_are_not_finite_stay_alone():
    say("int8 product, a row not finite")
    rng = np.random.default_rng(1)
    for rows in (5, 40, 300):
        x = rows_of(rng, rows, 128, "f32")
        x[4, 7] = np.inf
        w, sw = weights_of(rng, 1, 96, 128)
        y = host(P.int8_linear(to_dev(x, "f32"), L.INT8(up(w), up(sw)), out_dtype=torch.float32))
        a, sa = R.quantize(x)
        ref = R.product(a, sa, w, sw, [0, rows])
        assert np.isnan(y[4]).all()
        eq(np.delete(y, 4, 0), np.delete(ref, 4, 0), "other rows")


def test_split_rows_gathered():
    """One group without offsets, its rows gathered, K split over workgroups."""
    say("int8 dense, gathered")
    rng = np.random.default_rng(4)
    for rows, N, K in ((90, 200, 6160), (20, 64, 512), (400, 129, 4096)):
        x = rows_of(rng, 50, K, "f32")
        w, sw = weights_of(rng, 1, N, K)
        gat = rng.integers(0, 50, rows).astype(np.int32)
        a, sa = R.quantize(x)
        y = R.product(a, sa, w, sw, [0, rows], gat)
        for epi in ("f32", "bf16"):
            for act in (to_dev(x, "f32"), L.INT8(up(a), up(sa))):
                out = L.int8_grouped_gemm(act, L.INT8(up(w), up(sw)), N=N, K=K, total_rows=rows,
                                          gather_rows=up(gat), epilogue=EPIS[epi])
                check_out(out, y, epi)


def test_extreme_codes():
    """Every product 127^2 over the longest K, and codes of -128."""
    say("int8 extreme codes")
    for K in (131056, 8192):
        for v, u in ((127, 127), (-127, 127), (-128, -128)):
            a = L.INT8(torch.full((18, K), v, dtype=torch.int8, device=DEV), torch.ones(18, device=DEV))
            w = L.INT8(torch.full((1, 33, K), u, dtype=torch.int8, device=DEV),
                       torch.ones(1, 33, device=DEV))
            y = host(L.int8_grouped_gemm(a, w, N=33, K=K, total_rows=18))
            assert (y == np.float32(v * u * K)).all()


def test_rows_outside_the_groups_are_left_alone():
    say("int8 rows behind the last group")
    rng = np.random.default_rng(8)
    for rows, sizes in ((40, [3, 0, 5]), (400, [100, 0, 130]), (2000, [600, 700])):
        off = offsets_of(rng, sizes)
        x = rows_of(rng, rows, 256, "bf16")
        w, sw = weights_of(rng, len(sizes), 192, 256)
        for epi, n, dt in (("f32", 192, torch.float32), ("silu", 96, torch.bfloat16)):
            out = torch.full((rows, n), 7.0, dtype=dt, device=DEV)
            L.int8_grouped_gemm(to_dev(x, "bf16"), L.INT8(up(w), up(sw)), up(off), N=192, K=256,
                                total_rows=rows, epilogue=EPIS[epi], out=out)
            a, sa = R.quantize(x)
            check_out(out[:off[-1]], R.product(a, sa, w, sw, off), epi)
            assert (out[off[-1]:] == 7).all()


def test_binding_refusals():
    say("int8 refusals")
    x = torch.zeros(4, 32, device=DEV)
    w = L.INT8(torch.zeros(2, 8, 32, dtype=torch.int8, device=DEV), torch.zeros(2, 8, device=DEV))
    off = torch.tensor([0, 2, 4], dtype=torch.int32, device=DEV)
    ok = dict(N=8, K=32, total_rows=4)
    assert L.int8_grouped_gemm(x, w, off, **ok).shape == (4, 8)
    assert L.int8_grouped_gemm(x[:0], w, off, N=8, K=32, total_rows=0).shape == (0, 8)
    bad = [((x, w, off), dict(ok, K=16)), ((x, w, off), dict(ok, N=16)), ((x, w, off.long()), ok),
           ((x, w, off[:2]), ok), ((x, w, None), ok), ((x, w, off), dict(ok, total_rows=5)),
           ((x.t(), w, off), ok), ((x, L.INT8(w.codes.transpose(0, 1), w.scales), off), ok),
           ((x, w, off), dict(ok, gather_rows=off)), ((x, w, off), dict(ok, out=x)),
           ((L.INT8(w.codes[0], w.scales), w, off), ok)]
    for a, k in bad:
        with pytest.raises(ValueError):
            L.int8_grouped_gemm(*a, **k)
    with pytest.raises(L.NVFP4Error):
        L.int8_grouped_gemm(x, w, off, **ok, validate=True,
                            gather_rows=torch.tensor([0, 1, 2, 4], dtype=torch.int32, device=DEV))
    with pytest.raises(L.NVFP4Error):
        L.int8_grouped_gemm(x, w, torch.tensor([0, 3, 2], dtype=torch.int32, device=DEV), **ok,
                            validate=True)


def test_strided_rows_and_another_stream():
    say("int8 strides and streams")
    rng = np.random.default_rng(12)
    for rows in (3, 50, 500):
        x = rows_of(rng, rows, 256, "bf16")
        w, sw = weights_of(rng, 1, 320, 256)
        wd = L.INT8(up(w), up(sw))
        big = torch.full((rows, 304), float("nan"), device=DEV, dtype=torch.bfloat16)
        big[:, 16:272] = to_dev(x, "bf16")
        a, sa = R.quantize(x)
        ref = R.product(a, sa, w, sw, [0, rows])
        st = torch.cuda.Stream()
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st):
            ys = [P.int8_linear(big[:, 16:272], wd, out_dtype=torch.float32) for _ in range(3)]
        y = P.int8_linear(big[:, 16:272], wd, out_dtype=torch.float32)   # both at once
        torch.cuda.current_stream().wait_stream(st)
        for t in ys + [y]:
            eq(host(t), ref, "product")


def test_moe_block_together():
    """Routing, both products and the combine as one run, eager and captured."""
    say("int8 MoE block")
    w = D.small_moe(5, T=48, E=8, topk=3, H=256, I=128)
    x, lg = D.activations(w), D.router_logits(w)
    gu, dn = dict(D.expert_weights(w, "gate_up")), dict(D.expert_weights(w, "down"))
    dev = lambda m: ((e, to_dev(a, "bf16")) for e, a in m.items())  # noqa: E731
    wgu = P.int8_quantize_weights(dev(gu), w.E, 2 * w.I, w.H, DEV)
    wd = P.int8_quantize_weights(dev(dn), w.E, w.H, w.I, DEV)
    qgu = [R.quantize(R.bf16(gu[e])) for e in range(w.E)]
    eq(host(wgu.codes), np.stack([q[0] for q in qgu]), "weight codes")
    for T in (48, 1, 7):
        xd, ld = to_dev(x[:T], "bf16"), up(lg[:T])
        d = P.int8_moe_block(xd, ld, wgu, wd, w.topk, out_dtype=torch.float32)
        off, gat = host(d["route"].expert_offsets), host(d["route"].gather_rows)
        a, sa = R.quantize(R.bf16(x[:T]))
        y = R.product(a, sa, host(wgu.codes), host(wgu.scales), off, gat)
        check_out(d["h"], y, "silu")
        a, sa = R.quantize(host(d["h"].float()))
        y = R.product(a, sa, host(wd.codes), host(wd.scales), off)
        eq(host(d["y"]), y, "down")
        ro, wt = host(d["route"].row_of), host(d["route"].topk_weights)
        acc = np.zeros((T, w.H), np.float32)
        for s in range(w.topk):
            acc = acc + wt[:, s, None] * y[ro[:, s]]
        eq(host(d["out"]), acc, "combined")
        # captured, replayed on new inputs with eager work between
        sx, sl = xd.clone(), ld.clone()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            o = P.int8_moe_block(sx, sl, wgu, wd, w.topk)["out"]
        for i in range(4):
            sx.copy_(xd.flip(0) * (i + 1))
            sl.copy_(ld.roll(i, 1))
            g.replay()
            e = P.int8_moe_block(sx.clone(), sl.clone(), wgu, wd, w.topk)["out"]
            torch.cuda.synchronize()
            assert torch.equal(o, e)


def test_command_and_router():
    """The log-prob gap command with the INT8 rollout, which lies nearer to its
    trainer than naive W4A4 to its own, and the router's figures."""
    say("int8 in the log-prob gap command")
    res = dict(logprob_gap.gaps(3, vocab=2000, int8=True))
    assert len(res) == 4
    assert 0 < res["INT8 W8A8"]["mean"] < res["naive W4A4"]["mean"]
    r = logprob_gap.router(3)
    assert 0 <= r["emptiest"] <= 1 <= r["fullest"] and r["balance"] > 0 and r["z"] > 0


def test_offsets_beyond_32_bits():
    """Rows, codes and weights more than 4 GB into their tensors."""
    say("int8 beyond 4 GB")
    K, src = 65536, 70000
    g = torch.Generator(device=DEV)
    g.manual_seed(3)
    codes = torch.randint(-127, 128, (src, K), generator=g, device=DEV, dtype=torch.int8)
    sa = torch.rand(src, generator=g, device=DEV) + 0.5
    w = torch.randint(-127, 128, (2, 96, K), generator=g, device=DEV, dtype=torch.int8)
    sw = torch.rand(2, 96, generator=g, device=DEV) + 0.5
    for rows in (9, 80, 140, 300):
        gat = torch.randint(src - 200, src, (rows,), generator=g, device=DEV, dtype=torch.int32)
        gat[::3] = torch.randint(0, src, gat[::3].shape, generator=g, device=DEV, dtype=torch.int32)
        off = torch.tensor([0, rows // 2, rows], dtype=torch.int32, device=DEV)
        y = L.int8_grouped_gemm(L.INT8(codes, sa), L.INT8(w, sw), off, N=96, K=K, total_rows=rows,
                                gather_rows=gat)
        idx = host(gat)
        ref = R.product(host(codes[gat.long()]), host(sa)[idx], host(w), host(sw), host(off))
        eq(host(y), ref, f"{rows} gathered rows")
    x = torch.empty(40000, K, dtype=torch.bfloat16, device=DEV)
    x[:-3] = 0
    x[-3:] = torch.randn(3, K, generator=g, device=DEV)
    q = L.int8_quantize_rows(x)
    c, s = R.quantize(host(x[-3:].float()))
    eq(host(q.codes[-3:]), c, "last rows' codes")
    eq(host(q.scales[-3:]), s, "last rows' scales")
    assert not q.codes[:-3].any()


def test_outputs_off_16_bytes():
    """Outputs that start anywhere; what lies beside them stays."""
    say("int8, outputs off 16 bytes")
    rng = np.random.default_rng(21)
    for rows in (3, 40, 100, 500):
        x = rows_of(rng, rows, 272, "bf16")
        w, sw = weights_of(rng, 1, 64, 272)
        a, sa = R.quantize(x)
        y = R.product(a, sa, w, sw, [0, rows])
        for epi, n, dt in (("f32", 64, torch.float32), ("bf16", 64, torch.bfloat16),
                           ("silu", 32, torch.bfloat16)):
            buf = torch.full((rows * n + 8,), 5.0, dtype=dt, device=DEV)
            out = buf[1:1 + rows * n].view(rows, n)
            L.int8_grouped_gemm(to_dev(x, "bf16"), L.INT8(up(w), up(sw)), N=64, K=272,
                                total_rows=rows, epilogue=EPIS[epi], out=out)
            check_out(out, y, epi)
            assert buf[0] == 5 and (buf[1 + rows * n:] == 5).all()


def test_empty_layers():
    say("int8, no rows")
    w = L.INT8(torch.zeros(4, 64, 32, dtype=torch.int8, device=DEV), torch.zeros(4, 64, device=DEV))
    d = L.INT8(torch.zeros(4, 32, 32, dtype=torch.int8, device=DEV), torch.zeros(4, 32, device=DEV))
    x = torch.zeros(0, 32, device=DEV, dtype=torch.bfloat16)
    o = P.int8_moe_block(x, torch.zeros(0, 4, device=DEV), w, d, 2)["out"]
    assert o.shape == (0, 32)
    one = L.INT8(w.codes[:1], w.scales[:1])
    assert P.int8_linear(x, one).shape == (0, 64)
    with pytest.raises(ValueError):
        P.int8_linear(x, w)                                 # four groups are not a layer


def test_deterministic():
    say("int8 deterministic")
    rng = np.random.default_rng(3)
    w, sw = weights_of(rng, 16, 512, 1024)
    wd = L.INT8(up(w), up(sw))
    for rows in (16, 640):
        x = to_dev(rows_of(rng, rows, 1024, "bf16"), "bf16")
        off = up(offsets_of(rng, [rows // 16] * 16))
        a = [L.int8_grouped_gemm(x, wd, off, N=512, K=1024, total_rows=rows,
                                 epilogue=L.NVFP4_EPI_SILU_MUL_BF16) for _ in range(3)]
        assert torch.equal(a[0], a[1]) and torch.equal(a[0], a[2])
