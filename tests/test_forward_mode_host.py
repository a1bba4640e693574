"""Forward-mode derivatives (no GPU needed): the calls without one refuse a dual
tensor instead of returning a result that lost its tangent.  A dual tensor's
requires_grad is False, and torch.no_grad() leaves its tangent alone."""
import pytest
import torch
from torch.autograd import forward_ad

from nvfp4_w4a4_moe_quant_amd import _lib as L
from nvfp4_w4a4_moe_quant_amd import pipeline as P


def dual(t):
    return forward_ad.make_dual(t, torch.ones_like(t))


def balance(x, z):
    P.moe_balance_loss(z, torch.zeros(4, 2, dtype=torch.int32))


@pytest.mark.parametrize("no_grad", [False, True])
def test_balance_loss(no_grad):
    x, z = torch.zeros(4, 32), torch.zeros(4, 8)
    with forward_ad.dual_level():
        with torch.set_grad_enabled(not no_grad):
            with pytest.raises(RuntimeError, match="forward-mode"):
                balance(x, dual(z))
            with pytest.raises(RuntimeError, match="forward-mode"):
                balance(x, dual(z.clone().requires_grad_()))
            with pytest.raises(ValueError, match="GPU"):     # plain ones pass
                balance(x, z)
            with pytest.raises(ValueError, match="GPU"):
                balance(x, dual(z).detach())


def test_balance_loss_in_a_transform():
    z = torch.zeros(4, 8)
    with pytest.raises(RuntimeError, match="forward-mode"):
        torch.func.jvp(lambda t: balance(None, t), (z,), (z,))
