"""GPU tests of the decode-step layer and the token log-probabilities
together, as a rollout and its trainer use them: layer -> vocabulary head ->
recorded log-probabilities -> the gradient of a policy loss on them."""
import numpy as np
import pytest
import torch

from nvfp4_w4a4_moe_quant_amd import _lib as L
from nvfp4_w4a4_moe_quant_amd import logprob_gap
from nvfp4_w4a4_moe_quant_amd import pipeline as P
import decode_ref as R
from test_gpu_moe_decode import Layer, _inputs

pytestmark = pytest.mark.gpu
from gpu_util import DEV, host, say


def _policy_loss(z, tokens, old, advantage):
    lp, ent = P.token_logprobs(z, tokens)
    ratio = torch.exp(lp - old)
    clipped = torch.minimum(ratio * advantage, torch.clamp(ratio, 0.8, 1.2) * advantage)
    return -(clipped + 0.01 * ent).mean()


@pytest.mark.parametrize("norm", [False, True])
def test_rollout_step_and_policy_gradient(norm):
    """The recorded log-probabilities against 64 bits, and the loss's gradient
    of the head's weight against torch's own log-softmax in 64 bits.  Bound: the
    error of the logits' gradient, 2^-20 of its size, through an FP32 product
    of 16 terms; and what lies below FP32's range: without a norm before the
    head the logits are of the order of 1e5, every probability but one is
    under exp(-100) < 2^-126, and FP32 has 0 for it, where 64 bits have a
    number (off by at most 2^-126 times the factors of the sum, |y| and 1)."""
    say(f"rollout step, then the policy gradient, norm={norm}")
    T, E, k, H, I, V = 16, 12, 3, 256, 128, 4001
    lay = Layer(31, E, H, I)
    x, lg = _inputs(31, T, E, H, "bf16")
    g = torch.Generator(device=DEV)
    g.manual_seed(5)
    head = torch.randn((H, V), generator=g, device=DEV) / 16
    layer = P.GraphedMoEDecode(lay.wgu, lay.wd, k, T=T, E=E, x_dtype=torch.bfloat16, device=DEV)
    for step in range(3):
        y = layer(x, lg).out
        assert torch.equal(y, P.moe_decode(x, lg, lay.wgu, lay.wd, k).out)
        if norm:
            y = (y.float() * y.float().square().mean(1, keepdim=True).rsqrt()).bfloat16()
        z = y.float() @ head
        tokens = torch.multinomial(torch.softmax(z, 1), 1, generator=g)[:, 0]
        r = L.token_logprobs(z, tokens, top_k=4)
        ref = R.log_probs(host(z), host(tokens), None, 4)
        assert (np.abs(host(r.logprobs) - ref["logprobs"]) <= ref["tol_logprobs"]).all()
        assert (host(r.top_ids) == ref["top_ids"]).all()
        hw = (head * 1.01).requires_grad_()
        adv = torch.randn(T, generator=g, device=DEV)
        _policy_loss(y.float() @ hw, tokens, r.logprobs, adv).backward()
        h64 = hw.detach().double().requires_grad_()
        lp = torch.log_softmax(y.double() @ h64, 1)
        sel = lp.gather(1, tokens[:, None])[:, 0]
        ratio = torch.exp(sel - r.logprobs.double())
        a64 = adv.double()
        loss = -(torch.minimum(ratio * a64, torch.clamp(ratio, 0.8, 1.2) * a64)
                 - 0.01 * (lp.exp() * lp).sum(1)).mean()
        loss.backward()
        d = (hw.grad.double() - h64.grad).norm()
        floor = 2.0 ** -126 * float(y.double().abs().sum()) * (H * V) ** 0.5
        assert d <= 2.0 ** -17 * h64.grad.norm() + floor, float(d)
        assert not norm or h64.grad.norm() > 1e6 * floor
        x = (x + y).contiguous()


def test_padded_batch_in_a_captured_size():
    """Fewer tokens than the captured size: the rows behind them are -inf in
    the logits, give 0, and change nothing else."""
    say("padded batch in a captured layer")
    lay = Layer(32, 10, 96, 64)
    layer = P.GraphedMoEDecode(lay.wgu, lay.wd, 2, T=24, E=10, x_dtype=torch.float32, device=DEV)
    for T in (24, 1, 17, 5):
        x, lg = _inputs(T, T, 10, 96, "f32")
        layer.logits.fill_(float("-inf"))
        layer.x[:T], layer.logits[:T] = x, lg
        out = layer().out
        lay.check(L.MoEDecodeOut(out[:T], layer.out.topk_ids[:T], layer.out.topk_weights[:T]), x,
                  lg, 2, "f32")
        assert (out[T:] == 0).all()


def test_captured_training_step():
    """Forward and gradient of non-leaf logits captured whole and replayed."""
    say("captured policy gradient")
    T, H, V = 8, 64, 3001
    g = torch.Generator(device=DEV)
    g.manual_seed(9)
    y, head = torch.randn((T, H), generator=g, device=DEV), torch.randn((H, V), generator=g, device=DEV)
    tokens = torch.randint(0, V, (T,), generator=g, device=DEV)
    ones = torch.ones(T, device=DEV)

    def step(z):
        r = L.token_logprobs(z, tokens)
        return L.token_logprobs_backward(z, tokens, r.norm, r.entropy, ones, ones)
    z = y @ head
    step(z)
    torch.cuda.synchronize()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        out = step(z)
    for rep in range(3):
        z.copy_((y * (rep + 1)) @ head)
        want = step(z.clone())
        gr.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


def test_refused_uses():
    say("refused: leaf logits under capture, gradient of temperatures, double backward")
    z = torch.randn((3, 50), device=DEV, requires_grad=True)
    y = torch.zeros(3, dtype=torch.int64, device=DEV)
    with pytest.raises(ValueError):
        P.token_logprobs(z, y, torch.ones(3, device=DEV, requires_grad=True))
    lp, _ = P.token_logprobs(z, y)
    with pytest.raises(RuntimeError, match="second derivative"):
        torch.autograd.grad(lp.sum(), z, create_graph=True)
    with pytest.raises(ValueError):
        L.token_logprobs(z.detach(), y.int())
    with pytest.raises(ValueError):
        L.token_logprobs(z.detach(), y.cpu())
    with pytest.raises(ValueError):
        L.token_logprobs(z.detach().T, torch.zeros(50, dtype=torch.int64, device=DEV))
    with pytest.raises(L.NVFP4Error):
        L.token_logprobs(z.detach(), y, top_k=33)
    lay = Layer(33, 4, 64, 32)
    x, lg = _inputs(1, 65, 4, 64, "bf16")
    with pytest.raises(L.NVFP4Error):
        lay(x, lg, 2)
    with pytest.raises(ValueError):
        lay(x[:4], lg[:4].double(), 2)
    with pytest.raises(ValueError):
        P.moe_decode(x[:4], lg[:4], lay.wd, lay.wgu, 2)
    with pytest.raises(ValueError):
        lay(x[:4], lg[:4], 2, out=torch.empty((4, 64), device=DEV))


def test_logprob_gap_command():
    say("log-prob gap command")
    res = dict(logprob_gap.gaps(3, vocab=2000))
    assert len(res) == 3
    for f in res.values():
        assert all(np.isfinite(v) for v in f.values()) and f["max"] >= f["mean"] >= 0
