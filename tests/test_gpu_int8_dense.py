"""GPU tests of the INT8 products as a dense layer calls them, with no group
offsets: the split of K over workgroups, every tile, several waves and row tiles
of the kernel for few rows.  FP32 and bf16 products bit for bit against the
64-bit reference, SiLU*mul within its derived bound."""
import ctypes

import numpy as np
import pytest
import torch

from nvfp4_w4a4_moe_quant_amd import _lib as L
import int8_ref as R

pytestmark = pytest.mark.gpu
from gpu_util import DEV, eq, host, say, to_dev
from test_gpu_int8 import EPIS, check_out, rows_of, up, weights_of


def parts_of(rows, N, K, epi):
    """Parts of K that the call on quantized rows sums up in its workspace."""
    a = L.Int8GemmArgs(num_groups=1, N=N, K=K, total_rows=rows, a_codes=256, a_scales=256,
                       src_rows=rows, w_codes=256, w_scales=256, epilogue=EPIS[epi], out=256)
    need = L.lib().int8_grouped_gemm_workspace_size(ctypes.byref(a))
    parts, left = divmod(need, 4 * rows * (N + -N % 4))
    assert left == 0
    return parts


def run(rows, N, K, parts=0, gather=False):
    rng = np.random.default_rng(rows + N + K)
    src = rows // 2 + 1 if gather else rows
    gat = rng.integers(0, src, rows).astype(np.int32) if gather else None
    for epi, given, dtype in (("f32", "x", "bf16"), ("bf16", "q", "f32"), ("f32", "q", "f32"),
                              ("bf16", "x", "f32"), ("silu", "x", "bf16")):
        n = N + (N & 1) if epi == "silu" else N
        assert parts_of(rows, n, K, epi) == (0 if epi == "silu" else parts)
        x = rows_of(rng, src, K, dtype)
        w, sw = weights_of(rng, 1, n, K)
        a, sa = R.quantize(x)
        y = R.product(a, sa, w, sw, [0, rows], gat)
        act = to_dev(x, dtype) if given == "x" else L.INT8(up(a), up(sa))
        out = L.int8_grouped_gemm(act, L.INT8(up(w), up(sw)), N=n, K=K, total_rows=rows,
                                  gather_rows=up(gat), epilogue=EPIS[epi])
        check_out(out, y, epi)


@pytest.mark.parametrize("rows,N,K,parts", [
    (130, 4099, 6160, 2), (193, 2050, 5136, 2), (100, 4090, 4112, 4), (66, 1999, 2080, 4),
    (300, 1024, 4096, 4), (70, 1030, 4112, 8), (100, 2048, 7168, 8), (129, 384, 8192, 8),
    (200, 67, 16384, 8), (65, 128, 131056, 8), (300, 260, 4112, 8)])
def test_split(rows, N, K, parts):
    say(f"int8 dense, {rows}x{N}x{K} in {parts} parts")
    run(rows, N, K, parts)
    if N < 2000:
        run(rows, N, K, parts, gather=True)


@pytest.mark.parametrize("rows,N,K", [
    (700, 1028, 1104), (12000, 520, 80), (2300, 512, 1040),        # 64 x 128 tiles
    (1100, 4097, 272), (1600, 4000, 1104), (4096, 2048, 64),       # 128 x 256
    (4000, 2050, 400), (2560, 4096, 80), (2500, 4090, 1104),       # 256 x 256
    (5000, 4096, 1104), (9000, 4100, 208), (8192, 2050, 400)])     # 320 x 256
def test_tiles(rows, N, K):
    say(f"int8 dense tiles, {rows}x{N}x{K}")
    run(rows, N, K)


def test_tiles_gathered():
    say("int8 dense tiles, gathered")
    for rows, N, K in ((700, 1028, 208), (1100, 4097, 272), (4000, 2050, 144), (9000, 4100, 80)):
        run(rows, N, K, gather=True)


@pytest.mark.parametrize("rows,N,K", [
    # 4 waves to a block of 16 columns with 1, 2 and 4 row tiles, then 2 waves
    (16, 6160, 96), (9, 8191, 1040), (32, 8192, 64), (20, 6150, 208), (64, 6144, 512), (49, 6161, 1040),
    (5, 12288, 80), (3, 16001, 64), (17, 12288, 512), (32, 16384, 80), (64, 16384, 64), (33, 12301, 272)])
def test_few_rows_of_wide_layers(rows, N, K):
    """SiLU*mul pairs its columns, so the same kernels take it at twice the width."""
    say(f"int8 dense, few rows, {rows}x{N}x{K}")
    run(rows, N, K)
    run(rows, N, K, gather=True)
    rng = np.random.default_rng(N)
    x = rows_of(rng, rows, K, "bf16")
    w, sw = weights_of(rng, 1, 2 * N, K)
    a, sa = R.quantize(x)
    out = L.int8_grouped_gemm(to_dev(x, "bf16"), L.INT8(up(w), up(sw)), N=2 * N, K=K,
                              total_rows=rows, epilogue=EPIS["silu"])
    check_out(out, R.product(a, sa, w, sw, [0, rows]), "silu")


@pytest.mark.parametrize("K,src", [(64, (1 << 30) - 1), (48, 1431655763), (32, (1 << 31) - 3)])
def test_last_rows_that_a_gather_reaches(K, src):
    """The largest tensors of rows shorter than a chunk that a gather may take: the
    last rows' 16-byte units end at 2^32."""
    say(f"int8 gathered from {src} rows of {K}")
    g = torch.Generator(device=DEV)
    g.manual_seed(K)
    codes = torch.empty((src, K), dtype=torch.int8, device=DEV)
    near, far = 50, src - 50
    for at in (0, far):
        codes[at:at + 50] = torch.randint(-127, 128, (50, K), generator=g, device=DEV,
                                          dtype=torch.int8)
    sa = torch.empty(src, device=DEV)
    sa[:near] = 1.5
    sa[far:] = 0.75
    w = torch.randint(-127, 128, (2, 200, K), generator=g, device=DEV, dtype=torch.int8)
    sw = torch.rand(2, 200, generator=g, device=DEV) + 0.5
    rng = np.random.default_rng(K)
    for rows in (20, 400):                              # the kernel for few rows, and tiles
        gat = np.concatenate([rng.integers(0, near, rows // 2), rng.integers(far, src, rows // 2)])
        gat[-1] = src - 1
        off = np.array([0, rows // 2 + 3, rows], np.int32)
        y = L.int8_grouped_gemm(L.INT8(codes, sa), L.INT8(w, sw), up(off), N=200, K=K,
                                total_rows=rows, gather_rows=up(gat.astype(np.int32)))
        idx = up(gat)
        eq(host(y), R.product(host(codes[idx]), host(sa[idx]), host(w), host(sw), off),
           f"{rows} gathered rows")
    del codes, sa
    torch.cuda.empty_cache()
