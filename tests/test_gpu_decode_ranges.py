"""GPU tests of the decode-step layer and the token log-probabilities at the
ends of their ranges and in the uses that a graph allows: layers with more
column blocks than workgroups, the longest sums, the large layer of the
benchmark, captured layers that own their weights, autograd under capture."""
import gc

import numpy as np
import pytest
import torch

from nvfp4_w4a4_moe_quant_amd import _lib as L
from nvfp4_w4a4_moe_quant_amd import pipeline as P
import decode_ref64 as R64

pytestmark = pytest.mark.gpu
from gpu_util import DEV, eq, host, say


def layer(seed, E, H, I):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    q = {}
    for name, N, K in (("gu", 2 * I, H), ("down", H, I)):
        q[name] = L.NVFP4(
            torch.randint(0, 256, (E, N, K // 2), dtype=torch.uint8, device=DEV, generator=g),
            torch.randint(0x20, 0x50, (E, N, K // 16), dtype=torch.uint8, device=DEV, generator=g),
            (0.5 + torch.rand(E, device=DEV, generator=g)) / (8.0 * K ** 0.5))
    return P.QuantWeights(q["gu"], 2 * I, H), P.QuantWeights(q["down"], H, I)


def inputs(seed, T, E, H, dtype):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    x = torch.randn((T, H), device=DEV, generator=g)
    return (x.bfloat16() if dtype == "bf16" else x), torch.randn((T, E), device=DEV, generator=g)


def check(r, x, lg, wgu, wd, k, dtype):
    ids, w, out, tol = R64.moe_layer(x, lg, wgu.w, wd.w, k, dtype)
    eq(host(r.topk_ids), ids, "ids")
    np.testing.assert_allclose(host(r.topk_weights), w, rtol=2.0 ** -20, atol=1e-37)
    off = (r.out.double() - out).abs()
    assert bool((off <= tol).all()), (float((off / tol).max()), int((off > tol).sum()))
    # the bound says something: it is well below the values
    assert float(tol.norm()) <= 0.5 * float(out.norm())


@pytest.mark.parametrize("T,E,k,H,I,dtype", [
    (3, 2, 1, 65536, 2048, "bf16"),    # 1024 column blocks of the down product
    (33, 2, 1, 16416, 1600, "bf16"),   # 513: one workgroup takes a second
    (40, 3, 2, 16448, 1024, "f32"),    # 514
    (2, 1, 1, 64, 65536, "bf16"), (2, 1, 1, 64, 65536, "f32"),
    (1, 2, 2, 65536, 64, "bf16"), (5, 2, 2, 65536, 32, "f32"),
    (16, 256, 8, 7168, 2048, "bf16"),  # the large layer, a batch of requests
    (64, 8, 2, 2048, 768, "bf16"), (64, 10, 10, 2048, 768, "f32"),  # many rows of an expert
])
def test_layer_sizes(T, E, k, H, I, dtype):
    say(f"moe decode T={T} E={E} k={k} H={H} I={I} {dtype}")
    wgu, wd = layer(T + E, E, H, I)
    x, lg = inputs(T, T, E, H, dtype)
    check(P.moe_decode(x, lg, wgu, wd, k), x, lg, wgu, wd, k, dtype)


def test_captured_layer_owns_its_weights():
    """A captured layer whose caller kept neither weights nor inputs, with
    other tensors made since."""
    say("captured layer, weights kept by the graph alone")
    T, E, k, H, I = 6, 8, 2, 256, 128
    wgu, wd = layer(3, E, H, I)
    x, lg = inputs(3, T, E, H, "bf16")
    want = P.moe_decode(x, lg, wgu, wd, k).out.clone()
    g = P.GraphedMoEDecode(wgu, wd, k, T=T, E=E, x_dtype=torch.bfloat16, device=DEV)
    sizes = [t.numel() for w in (wgu, wd) for t in w.w]
    del wgu, wd
    gc.collect()
    torch.cuda.synchronize()
    junk = [torch.full((n,), 0x7F, dtype=torch.uint8, device=DEV) for n in sizes for _ in range(4)]
    for _ in range(3):
        assert torch.equal(g(x, lg).out, want)
    # in two steps, the first rows of a padded batch
    g.logits.fill_(float("-inf"))
    g.x[:2], g.logits[:2] = x[:2], lg[:2]
    out = g().out
    assert torch.equal(out[:2], want[:2]) and (out[2:] == 0).all()
    with pytest.raises(ValueError):
        g(x[:1], lg[:1])
    assert torch.equal(g(x, lg).out, want) and len(junk) > 0


def test_captured_block_and_linear_own_their_weights():
    say("captured block and linear, weights kept by the graph alone")
    T, E, k, H, I = 16, 4, 2, 256, 128
    wgu, wd = layer(4, E, H, I)
    x, lg = inputs(4, T, E, H, "bf16")
    want = P.moe_block(x, lg, wgu, wd, k, 16, 16)["out"].clone()
    w1, _ = layer(5, 1, H, I)
    dense = P.dense_forward(x, w1, 16)["y"].clone()
    block = P.GraphedMoEBlock(wgu, wd, k, 16, 16, T=T, E=E, x_dtype=torch.bfloat16, device=DEV)
    linear = P.GraphedDense(w1, 16, rows=T, x_dtype=torch.bfloat16, device=DEV)
    sizes = [t.numel() for w in (wgu, wd, w1) for t in w.w]
    del wgu, wd, w1
    gc.collect()
    torch.cuda.synchronize()
    junk = [torch.full((n,), 0x7F, dtype=torch.uint8, device=DEV) for n in sizes for _ in range(4)]
    for _ in range(3):
        assert torch.equal(block(x, lg), want) and torch.equal(linear(x), dense)
    assert len(junk) > 0


def test_leaf_logits_are_refused_under_capture():
    say("leaf logits under capture")
    z = torch.randn((3, 50), device=DEV, requires_grad=True)
    y = torch.zeros(3, dtype=torch.int64, device=DEV)
    L.token_logprobs(z.detach(), y)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        with pytest.raises(RuntimeError, match="leaf"):
            P.token_logprobs(z, y)
        lp, ent = P.token_logprobs(z.detach(), y)
    g.replay()
    want = L.token_logprobs(z.detach(), y)
    assert torch.equal(lp, want.logprobs) and torch.equal(ent, want.entropy)


def test_captured_autograd_of_inner_logits():
    """pipeline.token_logprobs of logits that an operation gave, captured with
    the gradient of those logits: every replay against the eager calls."""
    say("autograd of non-leaf logits under capture")
    T, V = 8, 3001
    gen = torch.Generator(device=DEV)
    gen.manual_seed(2)
    base = torch.randn((T, V), device=DEV, generator=gen)
    y = torch.randint(0, V, (T,), device=DEV, generator=gen)
    ga, gb = (torch.randn(T, device=DEV, generator=gen) for _ in range(2))
    r = L.token_logprobs(base, y)
    L.token_logprobs_backward(base, y, r.norm, r.entropy, ga, gb)
    src = base.clone()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        z = src.detach().requires_grad_() * 0.5
        lp, ent = P.token_logprobs(z, y)
        grad, = torch.autograd.grad([lp, ent], [z], [ga, gb])
    for rep in range(4):
        src.copy_(base * (rep + 1))
        g.replay()
        e = base * (rep + 1) * 0.5
        r = L.token_logprobs(e, y)
        want = L.token_logprobs_backward(e, y, r.norm, r.entropy, ga, gb)
        torch.cuda.synchronize()
        assert torch.equal(lp.detach(), r.logprobs) and torch.equal(ent.detach(), r.entropy)
        assert torch.equal(grad, want)
