"""GPU tests of the router's balance loss over many rows and at the ends of its
range: sums whose rounding errors all point one way, batches of more than 64
rows to a lane, a z-loss whose rows lie beyond the square root of FP32's range.
u = 2^-24."""
import numpy as np
import pytest
import torch

from nvfp4_w4a4_moe_quant_amd import _lib as L
import balance_ref as B

pytestmark = pytest.mark.gpu
from gpu_util import DEV, eq, host, say
from test_gpu_balance import case, check, near

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
LONG = [
    # a lane's rows: T / 4096 for each of the wave's 64 / lanes rows; 2^24 rows of
    # five experts are 1024 of a lane
    (1 << 24, 5, 5, "f32"), (1 << 24, 9, 9, "bf16"), (1 << 23, 60, 60, "f32"),
    (1 << 22, 100, 104, "f32"), (1 << 22, 100, 101, "bf16"), (1 << 21, 250, 256, "f32"),
    (1 << 21, 1000, 1000, "f32"), (1 << 21, 1000, 1001, "f32"), (1 << 21, 1000, 1000, "bf16")]


def equal_rows(T, E, pitch, dtype):
    """Logits of zero: every probability 1/E, every log-sum ln E, the loss 1."""
    say(f"balance, equal rows {T}x{E} of {pitch} {dtype}")
    z = torch.zeros((T, pitch), dtype=TYPES[dtype], device=DEV)[:, :E]
    ids = torch.arange(T, dtype=torch.int32, device=DEV).remainder_(E)[:, None]
    return L.moe_balance_loss(z, ids)


@pytest.mark.parametrize("T,E,pitch,dtype", LONG)
def test_z_loss_of_equal_rows(T, E, pitch, dtype):
    """A log-sum is off by a step of the hardware's logarithm (2 u), its factor and
    its product (u each), its square by twice that; the sum is FP64 and the mean
    rounded once."""
    r = equal_rows(T, E, pitch, dtype)
    assert int(r.tokens) == T
    z = np.log(np.float64(E)) ** 2
    near(r.losses[1], z, 10 * B.U * z, "z-loss")


def test_z_loss_of_large_logits():
    """Squares beyond FP32's range whose mean is within it, and a mean beyond it."""
    say("balance, z-loss of large logits")
    for T in (40, 300, 5000):
        z, ids, _ = case(T, T, 48, 4)
        z[3] = 2e19
        z[5, 1] = -3e38
        z[7] = -1e19
        assert 4e38 < 2e19 ** 2 + 1e19 ** 2 and (2e19 ** 2 + 1e19 ** 2) / T < 3e38
        check(z, ids, None, g=(0.01, 0.002))
        z[9] = 1e30
        r = L.moe_balance_loss(z, torch.from_numpy(ids).to(DEV))
        assert torch.isinf(r.losses[1]) and torch.isfinite(r.losses[0])


@pytest.mark.parametrize("T,E,pitch,dtype", LONG)
def test_mean_probabilities_of_equal_rows(T, E, pitch, dtype):
    """A mean probability is a sum in FP32 over up to 64 rows of a lane, three row
    slots and 16 waves, rounded once between them, and in FP64 above that: at most
    64 + 3 + 15 + 2 roundings, beside two of the probability itself."""
    r = equal_rows(T, E, pitch, dtype)
    eq(host(r.counts), np.bincount(np.arange(T) % E, minlength=E), "counts")
    near(r.mean_probs, np.full(E, 1.0 / E), 86 * B.U / E, "mean probabilities")
    near(r.losses[0], 1.0, 87 * B.U, "balance loss")


@pytest.mark.parametrize("T,E,dtype", [
    (262144, 130, "f32"), (262145, 130, "f32"), (300007, 130, "f32"), (270001, 600, "bf16")])
def test_more_rows_than_a_chain(T, E, dtype):
    """64 rows of a lane, and more; masks, padding, dropped slots."""
    say(f"balance, {T}x{E} {dtype}")
    check(*case(T + E, T, E, 4, dtype, masked=0.2, padded=0.1, dropped=0.1))
