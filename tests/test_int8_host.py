"""Host-side checks of the INT8 and balance-loss calls (no GPU needed): each
invalid argument is refused with its status before any work is enqueued."""
import ctypes

import pytest
import torch

from nvfp4_w4a4_moe_quant_amd import _lib as L
from nvfp4_w4a4_moe_quant_amd import pipeline as P

OK, ENULL, ESHAPE, EDTYPE, EALIGN, EWS, EHIP = range(7)
FAKE = ctypes.c_void_p(0x100000)
MIS = {n: ctypes.c_void_p(0x100000 + n) for n in (1, 2, 4, 8)}


@pytest.fixture(scope="module")
def lib():
    return L.load()


def test_rows_validation(lib):
    def q(x=FAKE, dt=1, rows=4, K=32, ldx=32, codes=FAKE, sc=FAKE):
        return lib.int8_quantize_rows(x, dt, rows, K, ldx, codes, sc, None)
    assert q(x=None) == ENULL and q(codes=None) == ENULL and q(sc=None) == ENULL
    assert q(dt=2) == EDTYPE and q(dt=-1) == EDTYPE
    assert q(K=24, ldx=32) == ESHAPE and q(K=0) == ESHAPE and q(rows=-1) == ESHAPE
    assert q(K=(1 << 24) + 16, ldx=1 << 25) == ESHAPE
    assert q(ldx=16) == ESHAPE
    assert q(ldx=36) == EALIGN
    assert q(x=MIS[8]) == EALIGN and q(codes=MIS[8]) == EALIGN and q(sc=MIS[2]) == EALIGN
    assert q(rows=0, x=None, codes=None, sc=None) == OK


def _gemm(lib, ws=None, wsb=0, size=False, **kw):
    a = L.Int8GemmArgs(num_groups=2, N=100, K=48, total_rows=10, group_offsets=FAKE,
                       a_codes=FAKE, a_scales=FAKE, src_rows=10, w_codes=FAKE, w_scales=FAKE,
                       epilogue=0, out=FAKE)
    for k, v in kw.items():
        setattr(a, k, v)
    if size:
        return lib.int8_grouped_gemm_workspace_size(ctypes.byref(a))
    return lib.int8_grouped_gemm(ctypes.byref(a), ws, wsb, None)


def test_gemm_validation(lib):
    def g(**kw):
        return _gemm(lib, **kw)
    assert lib.int8_grouped_gemm(None, None, 0, None) == ENULL
    assert lib.int8_grouped_gemm_workspace_size(None) == 0
    for k in ("out", "a_codes", "a_scales", "w_codes", "w_scales", "group_offsets"):
        assert g(**{k: None}) == ENULL, k
    assert g(out=None, total_rows=0) == OK
    assert g(total_rows=0, w_scales=None) == ENULL
    assert g(epilogue=3) == EDTYPE and g(epilogue=-1) == EDTYPE
    assert g(K=40) == ESHAPE and g(K=0) == ESHAPE and g(K=131072) == ESHAPE
    assert g(N=0) == ESHAPE and g(N=(1 << 24) + 1) == ESHAPE
    assert g(N=101, epilogue=1) == ESHAPE               # gate and up columns in pairs
    assert g(num_groups=0) == ESHAPE and g(num_groups=(1 << 20) + 1) == ESHAPE
    assert g(total_rows=-1) == ESHAPE and g(total_rows=1 << 31) == ESHAPE
    assert g(src_rows=9) == ESHAPE                      # fewer than total_rows, no gather
    assert g(src_rows=0, gather_rows=FAKE) == ESHAPE
    assert g(src_rows=1 << 33, K=48) == ESHAPE
    assert g(src_rows=(1 << 30) + 1, K=64, gather_rows=FAKE) == ESHAPE    # 2^36 bytes
    assert g(a_codes=MIS[8]) == EALIGN and g(w_codes=MIS[8]) == EALIGN
    assert g(a_scales=MIS[2]) == EALIGN and g(w_scales=MIS[2]) == EALIGN
    assert g(out=MIS[2]) == EALIGN and g(out=MIS[1], epilogue=2) == EALIGN
    assert g(gather_rows=MIS[2]) == EALIGN and g(group_offsets=MIS[2]) == EALIGN


def test_gemm_of_unquantized_rows_validation(lib):
    x = dict(a_codes=None, a_scales=None, x=FAKE, x_dtype=1, ldx=48, src_rows=10)

    def g(**kw):
        return _gemm(lib, **{**dict(ws=FAKE, wsb=1 << 20), **x, **kw})
    assert g(a_codes=FAKE) == ESHAPE                    # both forms
    assert g(x_dtype=2) == EDTYPE
    assert g(ldx=32) == ESHAPE and g(ldx=52) == EALIGN
    assert g(src_rows=9) == ESHAPE                      # fewer than total_rows, no gather
    assert g(src_rows=0, gather_rows=FAKE) == ESHAPE
    assert g(src_rows=-1, gather_rows=FAKE) == ESHAPE
    assert g(x=MIS[8]) == EALIGN
    # more tiles than a grid holds: refused before the rows are quantized
    assert g(total_rows=1 << 30, src_rows=1, gather_rows=FAKE, N=1 << 24) == ESHAPE
    assert g(num_groups=1 << 20, total_rows=1 << 25, src_rows=1, gather_rows=FAKE,
             N=1 << 20) == ESHAPE
    need = _gemm(lib, size=True, **{**x, "src_rows": 5000, "gather_rows": FAKE, "total_rows": 9999})
    assert need >= 5000 * 52
    assert _gemm(lib, size=True) == 0                   # quantized: none
    # a long K split over workgroups needs room for its sums, quantized rows or not
    one = dict(num_groups=1, group_offsets=None, N=2048, K=7168, total_rows=100)
    split = _gemm(lib, size=True, src_rows=100, **one)
    assert split >= 2 * 4 * 100 * 2048
    assert _gemm(lib, size=True, **{**x, **one, "src_rows": 100, "ldx": 7168}) >= split + 100 * 7172
    assert _gemm(lib, src_rows=100, **one) == EWS
    assert _gemm(lib, src_rows=100, ws=FAKE, wsb=split - 1, **one) == EWS
    assert _gemm(lib, size=True, src_rows=100, epilogue=1, **one) == 0
    big = dict(src_rows=5000, gather_rows=FAKE, total_rows=9999)
    assert g(ws=None, **big) == EWS and g(wsb=need - 1, **big) == EWS and g(ws=MIS[4], **big) == EWS
    assert g(total_rows=0, out=None, ws=None) == OK


def test_balance_validation(lib):
    def f(logits=FAKE, dt=0, T=8, E=16, ld=16, ids=FAKE, k=2, mask=None, counts=FAKE, tok=FAKE,
          mean=None, losses=FAKE, ws=FAKE, wsb=1 << 22):
        return lib.moe_balance_loss(logits, dt, T, E, ld, ids, k, mask, counts, tok, mean, losses,
                                    ws, wsb, None)
    for k in ("logits", "ids", "counts", "tok", "losses"):
        assert f(**{k: None}) == ENULL, k
    assert f(dt=2) == EDTYPE
    assert f(T=-1) == ESHAPE and f(E=0) == ESHAPE and f(E=1025, ld=1025) == ESHAPE
    assert f(k=0) == ESHAPE and f(k=17) == ESHAPE and f(ld=15) == ESHAPE
    assert f(T=1 << 30, k=2) == ESHAPE                  # T k
    assert f(logits=MIS[2]) == EALIGN and f(logits=MIS[1], dt=1) == EALIGN
    assert f(counts=MIS[2]) == EALIGN and f(ids=MIS[2]) == EALIGN and f(mean=MIS[2]) == EALIGN
    assert f(ws=None) == EWS and f(wsb=lib.moe_balance_loss_workspace_size(8, 16) - 1) == EWS
    assert f(ws=MIS[2]) == EWS
    assert lib.moe_balance_loss_workspace_size(-1, 16) == 0
    assert lib.moe_balance_loss_workspace_size(0, 16) > 0

    def b(logits=FAKE, dt=0, T=8, E=16, ld=16, k=2, mask=None, counts=FAKE, tok=FAKE, g=FAKE,
          out=FAKE, ldg=16):
        return lib.moe_balance_loss_backward(logits, dt, T, E, ld, k, mask, counts, tok, g, out,
                                             ldg, None)
    other = ctypes.c_void_p(0x900000)
    for k in ("logits", "counts", "tok", "g", "out"):
        assert b(**{k: None}) == ENULL, k
    assert b(dt=7) == EDTYPE and b(ldg=15) == ESHAPE and b(ld=15) == ESHAPE and b(k=17) == ESHAPE
    assert b(ld=20) == ESHAPE                           # in place with another row stride
    assert b(out=MIS[2]) == EALIGN and b(g=MIS[2]) == EALIGN and b(logits=MIS[2], out=other) == EALIGN
    assert b(T=0, logits=None, out=None) == OK


def test_binding_refuses_host_tensors():
    x = torch.zeros(4, 32)
    w = L.INT8(torch.zeros(1, 8, 32, dtype=torch.int8), torch.zeros(1, 8))
    with pytest.raises(ValueError):
        L.int8_quantize_rows(x)
    with pytest.raises(ValueError):
        L.int8_grouped_gemm(x, w, N=8, K=32, total_rows=4)
    with pytest.raises(ValueError):
        L.moe_balance_loss(x, torch.zeros(4, 2, dtype=torch.int32))
    with pytest.raises(ValueError):
        L.moe_balance_loss_backward(x, 2, torch.zeros(32, dtype=torch.int32),
                                    torch.zeros(1, dtype=torch.int32), torch.zeros(2))
    with pytest.raises(TypeError):
        L.int8_quantize_rows(x.half())


def test_layers_refuse_a_gradient():
    x = torch.zeros(4, 32, requires_grad=True)
    w = L.INT8(torch.zeros(1, 8, 32, dtype=torch.int8), torch.zeros(1, 8))
    with pytest.raises(RuntimeError, match="no gradient"):
        P.int8_linear(x, w)
    with pytest.raises(RuntimeError, match="no gradient"):
        P.int8_moe_block(x.detach(), torch.zeros(4, 8, requires_grad=True), w, w, 2)
    with pytest.raises(TypeError):
        P.int8_linear(x.detach(), w, out_dtype=torch.float16)
