"""GPU tests of the decode-step layer at the ends of FP32's range: an h beyond
it, and outputs near the bottom of it."""
import numpy as np
import pytest
import torch

from nvfp4_w4a4_moe_quant_amd import _lib as L
import decode_ref as R
from test_gpu_moe_decode import Layer, _inputs

pytestmark = pytest.mark.gpu
from gpu_util import DEV, host, say


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("I", [64, 1024])
def test_an_infinite_h_keeps_its_sign(I, dtype):
    """One column of h overflows FP32 (g and u are 8.6e22 there, 3.1e16
    elsewhere): the outputs are its infinity with the sign of the down weight,
    whatever the other columns' exponents."""
    say(f"moe decode: one infinite h, I={I} {dtype}")
    H, N = 32, 2 * I
    for col in (0, I - 1):
        codes = torch.full((1, N, H // 2), 0x11, dtype=torch.uint8)        # 0.5
        scales = torch.full((1, N, H // 16), 0x01, dtype=torch.uint8)      # 2^-9
        codes[0, [col, I + col]], scales[0, [col, I + col]] = 0x77, 0x7E   # 6 * 448
        gu = L.NVFP4(codes.to(DEV), scales.to(DEV), torch.full((1,), 1e18, device=DEV))
        codes = torch.full((1, H, I // 2), 0x22, dtype=torch.uint8)        # 1.0
        codes[0, 1::2] = 0xAA                                              # -1.0
        scales = torch.full((1, H, I // 16), 0x38, dtype=torch.uint8)      # 1.0
        wd = L.NVFP4(codes.to(DEV), scales.to(DEV), torch.full((1,), 1e-3, device=DEV))
        for T in (1, 3):
            x = torch.ones((T, H), dtype=torch.bfloat16 if dtype == "bf16" else torch.float32,
                           device=DEV)
            out = host(L.nvfp4_moe_decode(x, torch.zeros((T, 1), device=DEV), gu, wd, 1).out.float())
            assert (out[:, 0::2] == np.inf).all() and (out[:, 1::2] == -np.inf).all(), out[0]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("size", [1e-12, 1e-14, 1e-15, 1e-16])
def test_small_outputs_keep_their_bits(size, dtype):
    """Small x with tensor scales as real weights have them: h and the outputs
    are small but normal numbers, and as exact as others."""
    say(f"moe decode: x of {size} {dtype}")
    lay = Layer(15, 4, 288, 160)
    for name in lay.q:
        lay.q[name][2][:] *= 2.0 ** -10 if name == "down" else 1.0
    up = lambda n: L.NVFP4(*(torch.from_numpy(a).to(DEV) for a in lay.q[n]))  # noqa: E731
    lay.wgu, lay.wd = lay.wgu._replace(w=up("gu")), lay.wd._replace(w=up("down"))
    x, lg = _inputs(5, 9, 4, 288, dtype)
    x = (x.float() * size).to(x.dtype)
    r = lay(x, lg, 2)
    lay.check(r, x, lg, 2, dtype)
    _, _, out, tol = R.moe_layer(host(x.float()), host(lg), lay.exact("gu"), lay.exact("down"), 2,
                                 dtype)
    assert np.median(np.abs(out)) > 2.0 ** -126 and np.linalg.norm(tol) < 0.1 * np.linalg.norm(out)
