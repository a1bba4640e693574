"""Host-side limits of the INT8 products (no GPU needed): the first call beyond
what the kernels can address is refused, the last one within it is not."""
import ctypes

import pytest

from nvfp4_w4a4_moe_quant_amd import _lib as L

OK, ESHAPE = 0, 2
FAKE = 0x100000


@pytest.mark.parametrize("K,most", [
    # the 16-byte units of a gathered row and the seven behind its start that a
    # chunk of 128 k asks for count in 32 bits: (src_rows - 1) K / 16 + 7 < 2^32
    (16, (1 << 31) - 1), (32, (1 << 31) - 3), (48, 1431655763), (64, (1 << 30) - 1),
    (80, 858993458), (112, 613566756), (128, 1 << 29), (144, 477218588)])
def test_gathered_rows_count_in_32_bits(K, most):
    def size(src_rows, gather):
        a = L.Int8GemmArgs(num_groups=2, N=100, K=K, total_rows=10, group_offsets=FAKE,
                           gather_rows=gather, x=FAKE, x_dtype=1, ldx=K, src_rows=src_rows,
                           w_codes=FAKE, w_scales=FAKE, epilogue=0, out=FAKE)
        return L.load().int8_grouped_gemm_workspace_size(ctypes.byref(a))

    def call(src_rows, gather):
        a = L.Int8GemmArgs(num_groups=2, N=100, K=K, total_rows=10, group_offsets=FAKE,
                           gather_rows=gather, a_codes=FAKE, a_scales=FAKE, src_rows=src_rows,
                           w_codes=FAKE, w_scales=FAKE, epilogue=0, out=None)
        return L.load().int8_grouped_gemm(ctypes.byref(a), None, 0, None)

    last = (most - 1) * (K // 16) + 7
    assert last < 1 << 32 and most * K <= 1 << 36
    assert size(most, FAKE) >= most * K
    assert call(most, FAKE) != ESHAPE                   # refused for its output alone
    if most < (1 << 31) - 1:
        assert size(most + 1, FAKE) == 0 and call(most + 1, FAKE) == ESHAPE
    assert size(min(most + 1, (1 << 36) // K, (1 << 31) - 1), None) > 0    # rows in order: 64 bits
