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


INT8 = L.INT8(torch.zeros(1, 8, 32, dtype=torch.int8), torch.zeros(1, 8))


def int8_linear(x, z):
    P.int8_linear(x, INT8)


def int8_block(x, z):
    P.int8_moe_block(x, z, INT8, INT8, 2)


@pytest.mark.parametrize("layer", [int8_linear, int8_block])
@pytest.mark.parametrize("no_grad", [False, True])
def test_int8_layers(layer, no_grad):
    x, z = torch.zeros(4, 32), torch.zeros(4, 8)
    with forward_ad.dual_level(), torch.set_grad_enabled(not no_grad):
        with pytest.raises(RuntimeError, match="forward-mode"):
            layer(dual(x), z)
        if layer is int8_block:
            with pytest.raises(RuntimeError, match="forward-mode"):
                layer(x, dual(z))
        else:
            with pytest.raises(ValueError, match="GPU"):
                layer(dual(x).detach(), z)


def test_decode_step_layer():
    x, z = torch.zeros(4, 32), torch.zeros(4, 8)
    w = P.QuantWeights(None, 64, 32)
    with forward_ad.dual_level():
        for a in ((dual(x), z), (x, dual(z))):
            with pytest.raises(RuntimeError, match="forward-mode"):
                P.moe_decode(*a, w, w, 2)
