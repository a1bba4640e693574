"""validate=True of the INT8 products checks what the call documents: groups may
end before total_rows, and gather indices behind the last group are not read."""
import numpy as np
import pytest
import torch

from nvfp4_w4a4_moe_quant_amd import _lib as L
import int8_ref as R

pytestmark = pytest.mark.gpu
from gpu_util import DEV, say, to_dev
from test_gpu_int8 import check_out, rows_of, up, weights_of


@pytest.mark.parametrize("gather", [False, True])
def test_groups_that_end_before_the_rows(gather):
    say(f"int8 validated, fewer rows in the groups, gather {gather}")
    rng = np.random.default_rng(3)
    off = np.array([0, 5, 5, 29], np.int32)
    x = rows_of(rng, 40, 64, "f32")
    w, sw = weights_of(rng, 3, 48, 64)
    gat = rng.integers(0, 40, 40).astype(np.int32) if gather else None
    if gather:
        gat[29:] = -1
    out = torch.full((40, 48), 7.0, device=DEV)
    call = dict(N=48, K=64, total_rows=40, gather_rows=up(gat), validate=True)
    L.int8_grouped_gemm(to_dev(x, "f32"), L.INT8(up(w), up(sw)), up(off), out=out, **call)
    a, sa = R.quantize(x)
    check_out(out[:29], R.product(a, sa, w, sw, off, gat), "f32")
    assert (out[29:] == 7).all()


def test_what_is_refused():
    say("int8 validated, refusals")
    x = torch.zeros(8, 32, device=DEV)
    w = L.INT8(torch.zeros(2, 16, 32, dtype=torch.int8, device=DEV), torch.zeros(2, 16, device=DEV))

    def call(off, gat=None, total=8):
        L.int8_grouped_gemm(x, w, torch.tensor(off, dtype=torch.int32, device=DEV), N=16, K=32,
                            total_rows=total, validate=True,
                            gather_rows=None if gat is None else
                            torch.tensor(gat, dtype=torch.int32, device=DEV))
    call([0, 3, 8])
    call([0, 3, 7])
    call([0, 0, 0])
    call([0, 1, 2], [7, 0, 99, -1], total=4)
    for off in ([0, 3, 9], [0, 4, 3], [1, 3, 8], [0, 3, -1], [0, -2, 8]):
        with pytest.raises(L.NVFP4Error):
            call(off)
    for gat in ([8, 0, 0, 0], [0, -1, 0, 0]):
        with pytest.raises(L.NVFP4Error):
            call([0, 1, 2], gat, total=4)
    one = L.INT8(w.codes[:1], w.scales[:1])             # one group without offsets: all rows
    assert L.int8_grouped_gemm(x, one, N=16, K=32, total_rows=8, validate=True).shape == (8, 16)
    with pytest.raises(L.NVFP4Error):
        L.int8_grouped_gemm(x, one, N=16, K=32, total_rows=2, validate=True,
                            gather_rows=torch.tensor([0, 8], dtype=torch.int32, device=DEV))
