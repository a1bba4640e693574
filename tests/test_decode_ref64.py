"""The 64-bit layer for large sizes against the one for small sizes (no GPU
needed)."""
import numpy as np
import pytest
import torch

import decode_ref as R
import decode_ref64 as R64


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_references_agree(dtype):
    g = np.random.default_rng(4)
    E, H, I, T, k = 5, 96, 64, 9, 3
    q = {n: (g.integers(0, 256, (E, N, K // 2), dtype=np.uint8),
             g.integers(0, 0x7F, (E, N, K // 16), dtype=np.uint8),
             g.uniform(0.01, 0.05, E).astype(np.float32))
         for n, N, K in (("gu", 2 * I, H), ("d", H, I))}
    x, lg = g.standard_normal((T, H)), g.standard_normal((T, E)).astype(np.float32)
    lg[2], lg[3, 1:] = -np.inf, -np.inf
    get = lambda n: (lambda e: (R.dequantize(q[n][0][e], q[n][1][e]), float(q[n][2][e])))  # noqa: E731
    want = R.moe_layer(x, lg, get("gu"), get("d"), k, dtype)
    up = lambda n: tuple(torch.from_numpy(a) for a in q[n])  # noqa: E731
    got = R64.moe_layer(torch.from_numpy(x), torch.from_numpy(lg), up("gu"), up("d"), k, dtype,
                        chain=lambda K: K * R.U32)
    for a, b in zip(got, want):
        np.testing.assert_allclose(np.asarray(a), b, rtol=1e-10, atol=1e-300)
