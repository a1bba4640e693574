"""Host-side checks (no GPU needed) of the captured layers, with the capture
itself replaced by a stand-in: what the object holds, and which calls it
refuses."""
import contextlib
import gc
import types
import weakref

import pytest
import torch

from nvfp4_w4a4_moe_quant_amd import _lib as L
from nvfp4_w4a4_moe_quant_amd import pipeline as P

T, E, H, I, K = 4, 3, 32, 32, 2


@pytest.fixture
def capture(monkeypatch):
    """Streams and graphs that do nothing; counts the replays."""
    seen = types.SimpleNamespace(replays=0)

    class Graph:
        def replay(self):
            seen.replays += 1

    stream = lambda *a, **k: types.SimpleNamespace(wait_stream=lambda other: None)  # noqa: E731
    nothing = lambda *a, **k: contextlib.nullcontext()  # noqa: E731
    for name, fake in (("Stream", stream), ("current_stream", stream), ("stream", nothing),
                       ("device", nothing), ("graph", nothing), ("CUDAGraph", Graph)):
        monkeypatch.setattr(torch.cuda, name, fake)
    monkeypatch.setattr(L, "nvfp4_moe_decode", lambda x, lg, wgu, wd, k, out=None: L.MoEDecodeOut(
        torch.zeros_like(x), torch.zeros((x.shape[0], k), dtype=torch.int32),
        torch.zeros((x.shape[0], k))))
    return seen


def weights(N, Kw):
    return P.QuantWeights(L.NVFP4(torch.zeros((E, N, Kw // 2), dtype=torch.uint8),
                                  torch.zeros((E, N, Kw // 16), dtype=torch.uint8),
                                  torch.zeros(E)), N, Kw)


def decode(wgu=None, wd=None, **kw):
    return P.GraphedMoEDecode(wgu or weights(2 * I, H), wd or weights(H, I), K, T=T, E=E,
                              x_dtype=torch.bfloat16, device="cpu", **kw)


def tensors(*ws):
    """Weak references to the tensors of weights."""
    return [weakref.ref(t) for w in ws for t in w.w]


def test_captured_decode_layer_keeps_its_weights(capture):
    """The captured kernels hold addresses only, so the object keeps what lies
    there: weights that only the constructor call had stay alive as long as
    it does, and no longer."""
    wgu, wd = weights(2 * I, H), weights(H, I)
    refs, g = tensors(wgu, wd), decode(wgu, wd)
    del wgu, wd
    gc.collect()
    assert all(r() is not None for r in refs)
    g()
    assert capture.replays == 1
    del g
    gc.collect()
    assert all(r() is None for r in refs)


def test_captured_block_keeps_its_weights(capture, monkeypatch):
    monkeypatch.setattr(P, "moe_block", lambda x, *a: dict(out=torch.zeros_like(x)))
    wgu, wd = weights(2 * I, H), weights(H, I)
    refs, g = tensors(wgu, wd), P.GraphedMoEBlock(wgu, wd, K, None, None, T=T, E=E,
                                                  x_dtype=torch.bfloat16, device="cpu")
    del wgu, wd
    gc.collect()
    assert all(r() is not None for r in refs)
    del g
    gc.collect()
    assert all(r() is None for r in refs)


def test_captured_linear_keeps_its_weights(capture, monkeypatch):
    monkeypatch.setattr(P, "dense_forward", lambda x, *a: dict(y=torch.zeros_like(x)))
    w = weights(I, H)
    refs, g = tensors(w), P.GraphedDense(w, None, rows=T, x_dtype=torch.bfloat16, device="cpu")
    del w
    gc.collect()
    assert all(r() is not None for r in refs)
    del g
    gc.collect()
    assert all(r() is None for r in refs)


@pytest.mark.parametrize("x,logits", [
    ((1, H), (1, E)),             # one token would have filled every row
    ((2, H), (2, E)),
    ((T, 1), None), ((H,), None), ((T, H, 1), None),
    (None, (T, 1)), (None, (E,)), (None, (1, E)), ((T, H), (1, E)),
])
def test_captured_decode_layer_refuses_other_shapes(capture, x, logits):
    g = decode()
    g.x.fill_(3), g.logits.fill_(4)
    xs = None if x is None else torch.ones(x, dtype=torch.bfloat16)
    lg = None if logits is None else torch.ones(logits)
    with pytest.raises(ValueError):
        g(xs, lg)
    assert (g.x == 3).all() and (g.logits == 4).all() and capture.replays == 0


def test_captured_decode_layer_refuses_other_types(capture):
    g = decode()
    for xs, lg in ((torch.ones((T, H)), None), (torch.ones((T, H), dtype=torch.float16), None),
                   (None, torch.ones((T, E), dtype=torch.bfloat16)),
                   (None, torch.ones((T, E), dtype=torch.float64))):
        with pytest.raises(ValueError):
            g(xs, lg)
    assert capture.replays == 0
    xs, lg = torch.rand((T, H)).bfloat16(), torch.rand((T, E))
    g(xs, lg)
    assert torch.equal(g.x, xs) and torch.equal(g.logits, lg) and capture.replays == 1


def test_captured_decode_layer_views_of_its_inputs(capture):
    """A tensor that starts where the static input does is that input only if
    it is laid out alike."""
    g = decode()
    g.x.copy_(torch.rand((T, H)))
    want = g.x.clone()
    g(g.x), g(g.x[:]), g(g.x.view(-1).view(T, H))
    assert torch.equal(g.x, want) and capture.replays == 3
    g(g.x[:1].expand(T, H))
    assert torch.equal(g.x, want[:1].expand(T, H))
    with pytest.raises(ValueError):
        g(g.x[:2], g.logits[:2])      # the first rows of a batch
    one = P.GraphedMoEDecode(weights(2 * I, H), weights(H, I), K, T=1, E=E,
                             x_dtype=torch.bfloat16, device="cpu")
    one(one.x.as_strided((1, H), (7, 1)))   # one row: its stride says nothing
    assert capture.replays == 5


def test_decode_layer_refuses_to_cut_gradients(capture):
    """The layer has no backward pass: under autograd, inputs that require a
    gradient are refused instead of giving a result without one."""
    wgu, wd = weights(2 * I, H), weights(H, I)
    x, lg = torch.ones((T, H), dtype=torch.bfloat16), torch.ones((T, E))
    xg, lgg = x.clone().requires_grad_(), lg.clone().requires_grad_()
    g = decode()
    for a, b in ((xg, lg), (x, lgg), (xg * 2, lg)):
        with pytest.raises(RuntimeError, match="gradient"):
            P.moe_decode(a, b, wgu, wd, K)
        with pytest.raises(RuntimeError, match="gradient"):
            g(a, b)
        with torch.no_grad():
            assert not P.moe_decode(a, b, wgu, wd, K).out.requires_grad
            g(a, b)
    with pytest.raises(RuntimeError, match="gradient"):
        decode(x=xg)
    assert not g.x.requires_grad and not g.logits.requires_grad
    assert not P.moe_decode(x, lg, wgu, wd, K).out.requires_grad
    assert not P.moe_decode(xg.detach(), lg, wgu, wd, K).out.requires_grad


def test_captured_decode_layer_refuses_inputs_elsewhere(capture):
    """Inputs on another device than the graph's: the launches would go to that
    device's stream, outside the capture, and replays would do nothing."""
    x, lg = torch.ones((T, H), dtype=torch.bfloat16), torch.ones((T, E))
    for kw in (dict(x=x.to("meta"), logits=lg), dict(x=x, logits=lg.to("meta"))):
        with pytest.raises(ValueError, match="device"):
            decode(**kw)
    assert decode(x=x, logits=lg).x is x
