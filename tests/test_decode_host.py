"""Host-side checks (no GPU needed) of nvfp4_moe_decode, token_logprobs and
token_logprobs_backward: invalid arguments are refused before any work is
enqueued, and the 64-bit references of the GPU tests agree with torch."""
import ctypes

import numpy as np
import pytest
import torch

from nvfp4_w4a4_moe_quant_amd import _lib as L
from nvfp4_w4a4_moe_quant_amd import pipeline as P
import decode_ref as R

OK, ENULL, ESHAPE, EDTYPE, EALIGN, EWS, EHIP = range(7)
FAKE, MIS = 0x100000, 0x100004  # never dereferenced


@pytest.fixture(scope="module")
def lib():
    return L.load()


def _args(**kw):
    a = dict(T=4, E=8, k=2, H=64, I=32, x=FAKE, x_dtype=1, ldx=64, logits=FAKE, ld_logits=8,
             gu_codes=FAKE, gu_scales=FAKE, gu_tscale=FAKE, d_codes=FAKE, d_scales=FAKE,
             d_tscale=FAKE, out=FAKE, ldo=64, topk_ids=FAKE, topk_weights=FAKE)
    a.update(kw)
    return L.MoEDecodeArgs(**a)


@pytest.mark.parametrize("want,kw", [
    (ESHAPE, dict(T=65)), (ESHAPE, dict(T=-1)), (ESHAPE, dict(E=0)), (ESHAPE, dict(E=1025)),
    (ESHAPE, dict(k=0)), (ESHAPE, dict(k=9)), (ESHAPE, dict(k=17, E=32, ld_logits=32)),
    (ESHAPE, dict(H=48)), (ESHAPE, dict(H=0, ldx=0)), (ESHAPE, dict(I=16)), (ESHAPE, dict(I=-32)),
    (ESHAPE, dict(H=65568, ldx=65568, ldo=65568)), (ESHAPE, dict(ldx=32)), (ESHAPE, dict(ldo=32)),
    (ESHAPE, dict(ld_logits=7)), (EDTYPE, dict(x_dtype=2)), (EALIGN, dict(ldx=68)),
    (EALIGN, dict(ldo=68)), (EALIGN, dict(x=MIS)), (EALIGN, dict(out=MIS)),
    (EALIGN, dict(gu_codes=MIS)), (EALIGN, dict(d_scales=MIS)), (EALIGN, dict(logits=FAKE + 2)),
    (EALIGN, dict(topk_ids=FAKE + 1)), (ENULL, dict(x=None)), (ENULL, dict(logits=None)),
    (ENULL, dict(gu_tscale=None)), (ENULL, dict(d_codes=None)), (ENULL, dict(out=None)),
    (OK, dict(T=0, x=None, logits=None, out=None)),
])
def test_moe_decode_refusals(lib, want, kw):
    a = _args(**kw)
    assert lib.nvfp4_moe_decode(ctypes.byref(a), FAKE, 1 << 30, None) == want


def test_moe_decode_workspace(lib):
    a = _args()
    n = lib.nvfp4_moe_decode_workspace_size(ctypes.byref(a))
    assert n > 4 * 2 * 32 * 4
    assert lib.nvfp4_moe_decode(ctypes.byref(a), FAKE, n - 1, None) == EWS
    assert lib.nvfp4_moe_decode(ctypes.byref(a), None, n, None) == EWS
    assert lib.nvfp4_moe_decode(ctypes.byref(a), MIS, n, None) == EWS
    assert lib.nvfp4_moe_decode(None, FAKE, n, None) == ENULL
    # sizes that the call refuses need no workspace
    for kw in (dict(T=65), dict(T=2 ** 62), dict(k=0), dict(I=2 ** 40), dict(H=2 ** 40)):
        lib.nvfp4_moe_decode_workspace_size(ctypes.byref(_args(**kw)))
    lib.nvfp4_moe_decode_workspace_size(None)


def _fwd(lib, logits=FAKE, dtype=1, T=4, V=100, ld=100, y=FAKE, it=None, k=2, lp=FAKE, ent=FAKE,
         norm=FAKE, ids=FAKE, tlp=FAKE, ws=FAKE, n=1 << 30):
    return lib.token_logprobs(logits, dtype, T, V, ld, y, it, k, lp, ent, norm, ids, tlp, ws, n,
                              None)


@pytest.mark.parametrize("want,kw", [
    (EDTYPE, dict(dtype=2)), (ESHAPE, dict(T=-1)), (ESHAPE, dict(T=2 ** 31)), (ESHAPE, dict(V=0)),
    (ESHAPE, dict(V=2 ** 31, ld=2 ** 31)), (ESHAPE, dict(ld=99)), (ESHAPE, dict(k=-1)),
    (ESHAPE, dict(k=33)), (ESHAPE, dict(V=3, k=4)), (ENULL, dict(logits=None)),
    (ENULL, dict(y=None)), (ENULL, dict(lp=None)), (ENULL, dict(ids=None)),
    (ENULL, dict(tlp=None)), (EALIGN, dict(logits=FAKE + 1)),
    (EALIGN, dict(logits=FAKE + 2, dtype=0)), (EWS, dict(ws=None, V=2 ** 20, ld=2 ** 20)),
    (EWS, dict(n=0, V=2 ** 20, ld=2 ** 20)), (EWS, dict(ws=MIS)), (OK, dict(T=0, logits=None, y=None, lp=None, ids=None)),
])
def test_logprobs_refusals(lib, want, kw):
    assert _fwd(lib, **kw) == want


@pytest.mark.parametrize("want,kw", [
    (ESHAPE, dict(T=2 ** 24)), (ESHAPE, dict(V=2 ** 30 + 1, ld=2 ** 31)),
    (EALIGN, dict(ent=FAKE + 2)), (EALIGN, dict(norm=FAKE + 1)), (EALIGN, dict(ids=FAKE + 2)),
    (EALIGN, dict(it=FAKE + 2)),
])
def test_logprobs_limits_and_alignment(lib, want, kw):
    assert _fwd(lib, **kw) == want


@pytest.mark.parametrize("want,kw", [
    (ESHAPE, dict(T=2 ** 24)), (ESHAPE, dict(V=2 ** 30 + 1, ld=2 ** 31, ldg=2 ** 31)),
    (EALIGN, dict(ga=FAKE + 2)), (EALIGN, dict(gb=FAKE + 1)), (EALIGN, dict(ent=FAKE + 2)),
    (EALIGN, dict(norm=FAKE + 2)),
])
def test_logprobs_backward_limits_and_alignment(lib, want, kw):
    assert _bwd(lib, **kw) == want


def _bwd(lib, logits=FAKE, dtype=1, T=4, V=100, ld=100, y=FAKE, it=None, norm=FAKE, ent=FAKE,
         ga=FAKE, gb=FAKE, g=2 * FAKE, ldg=100):
    return lib.token_logprobs_backward(logits, dtype, T, V, ld, y, it, norm, ent, ga, gb, g, ldg,
                                       None)


@pytest.mark.parametrize("want,kw", [
    (EDTYPE, dict(dtype=7)), (ESHAPE, dict(T=-1)), (ESHAPE, dict(V=0)), (ESHAPE, dict(ld=99)),
    (ESHAPE, dict(ldg=99)), (ESHAPE, dict(g=FAKE, ldg=101)), (ENULL, dict(logits=None)),
    (ENULL, dict(norm=None)), (ENULL, dict(g=None)), (ENULL, dict(y=None)),
    (ENULL, dict(ent=None)), (EALIGN, dict(g=FAKE + 1)), (EALIGN, dict(logits=FAKE + 2, dtype=0)),
    (OK, dict(T=0, logits=None, norm=None, g=None)),
])
def test_logprobs_backward_refusals(lib, want, kw):
    assert _bwd(lib, **kw) == want


def test_binding_refuses_before_the_library():
    """Shapes, types and devices that the C side cannot see."""
    x, lg = torch.zeros((2, 64), dtype=torch.bfloat16), torch.zeros((2, 4))
    w = L.NVFP4(torch.zeros((4, 64, 32), dtype=torch.uint8), torch.zeros((4, 64, 4), dtype=torch.uint8),
                torch.zeros(4))
    with pytest.raises(ValueError, match="GPU"):
        L.nvfp4_moe_decode(x, lg, w, w, 2)
    with pytest.raises(ValueError):
        L.nvfp4_moe_decode(x[:1], lg, w, w, 2)
    with pytest.raises(TypeError):
        L.nvfp4_moe_decode(x.half(), lg, w, w, 2)
    with pytest.raises(ValueError, match="GPU"):
        L.token_logprobs(lg)
    with pytest.raises(ValueError):
        L.token_logprobs(lg[0])
    with pytest.raises(TypeError):
        L.token_logprobs(lg.double())
    with pytest.raises(ValueError, match="GPU"):
        P.token_logprobs(lg, torch.zeros(2, dtype=torch.int64))
    with pytest.raises(ValueError, match="rows"):
        L._row_stride(torch.zeros((4, 8)).T, "t")
    with pytest.raises(ValueError, match="overlap"):
        L._row_stride(torch.zeros(8).expand(4, 8), "t")
    with pytest.raises(ValueError, match="targets"):
        L._vector(torch.zeros(4, dtype=torch.int32), 4, torch.int64, torch.device("cpu"), "targets")


def test_references_against_torch():
    g = np.random.default_rng(0)
    z = g.standard_normal((5, 40))
    z[2, 3:9] = -np.inf
    y = np.array([1, -1, 4, 39, 0])
    it = np.array([1, .5, 2, 1, 3], np.float32)
    zt = torch.from_numpy(z).requires_grad_()
    lp = torch.log_softmax(zt * torch.from_numpy(it).double()[:, None], 1)
    p = lp.exp()
    ent = -torch.where(p > 0, p * torch.where(p > 0, lp, 0.0), 0.0).sum(1)
    sel = lp[torch.arange(5), torch.from_numpy(y).clamp(min=0)]
    r = R.log_probs(z, y, it, 3)
    live = y >= 0
    fin = np.isfinite(r["logprobs"])
    np.testing.assert_allclose(r["entropy"], ent.detach().numpy(), rtol=1e-12)
    np.testing.assert_allclose(r["logprobs"][live & fin], sel.detach().numpy()[live & fin], rtol=1e-12)
    y[2] = 20
    ga, gb = g.standard_normal(5), g.standard_normal(5)
    r = R.log_probs(z, y, it, 0)
    want, _ = R.log_probs_grad(r, y, it, ga, gb, "f32")
    sel = torch.log_softmax(torch.where(torch.isinf(zt), -1e300, zt) * torch.from_numpy(it).double()[:, None], 1)
    p = sel.exp()
    ent = -torch.where(p > 0, p * sel, 0.0).sum(1)
    a = torch.from_numpy(np.where(y < 0, 0, ga))
    (sel[torch.arange(5), torch.from_numpy(y).clamp(min=0)] * a + ent * torch.from_numpy(gb)).sum().backward()
    np.testing.assert_allclose(want[~np.isinf(z)], zt.grad.numpy()[~np.isinf(z)], rtol=1e-9, atol=1e-12)


def test_moe_reference_against_torch():
    g = np.random.default_rng(1)
    E, H, I, T, k = 3, 32, 32, 4, 2
    c = {n: (g.integers(0, 256, (E, N, K // 2), dtype=np.uint8),
             g.integers(0x20, 0x50, (E, N, K // 16), dtype=np.uint8))
         for n, N, K in (("gu", 2 * I, H), ("d", H, I))}
    x, lg = g.standard_normal((T, H)), g.standard_normal((T, E))
    lg[1] = -np.inf
    get = lambda n: (lambda e: (R.dequantize(c[n][0][e], c[n][1][e]), 0.25))  # noqa: E731
    ids, w, out, tol = R.moe_layer(x, lg, get("gu"), get("d"), k, "f32")
    assert (out[1] == 0).all() and (w[1] == 0).all()
    for t in (0, 2, 3):
        pr = torch.softmax(torch.from_numpy(lg[t]), 0)
        v, i = torch.topk(pr, k)
        assert list(i.numpy()) == list(ids[t])
        o = 0
        for s in range(k):
            wg, wd = get("gu")(int(i[s]))[0], get("d")(int(i[s]))[0]
            y = 0.25 * torch.from_numpy(wg) @ torch.from_numpy(x[t])
            o = o + v[s] * 0.25 * torch.from_numpy(wd) @ (torch.nn.functional.silu(y[:I]) * y[I:])
        np.testing.assert_allclose(out[t], o.numpy(), rtol=1e-9)
    e4 = R.e4m3(np.arange(0x7F, dtype=np.uint8))
    t8 = torch.arange(0x7F, dtype=torch.uint8).view(torch.float8_e4m3fn).float().numpy()
    np.testing.assert_array_equal(e4, t8)
