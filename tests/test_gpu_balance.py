"""GPU tests of the router's balance loss and its gradient against the 64-bit
reference and its derived tolerances."""
import numpy as np
import pytest
import torch

from nvfp4_w4a4_moe_quant_amd import _lib as L
from nvfp4_w4a4_moe_quant_amd import pipeline as P
import balance_ref as B

pytestmark = pytest.mark.gpu
from gpu_util import DEV, eq, host, say

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def up(a):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def case(seed, T, E, k, dtype="f32", masked=0.0, padded=0.0, dropped=0.0, scale=2.0):
    rng = np.random.default_rng(seed)
    z = torch.from_numpy((rng.standard_normal((T, E)) * scale + np.linspace(0, 2, E))
                         .astype(np.float32)).to(TYPES[dtype])
    z[torch.from_numpy(rng.random((T, E)) < masked)] = float("-inf")
    ids = np.argsort(-z.float().numpy(), 1, kind="stable")[:, :k].astype(np.int32)
    ids[rng.random(ids.shape) < dropped] = -1
    mask = rng.random(T) >= padded if padded else None
    return z.to(DEV), ids, mask


def near(got, ref, tol, what):
    got, ref = host(got.float()).astype(np.float64), np.asarray(ref, np.float64)
    ref = np.where(np.abs(ref) > 3.4029e38, np.sign(ref) * np.inf, ref)   # beyond FP32's range
    eq(np.isnan(got), np.isnan(ref), what + ": NaN")
    with np.errstate(invalid="ignore"):
        bad = ~(np.abs(got - ref) <= tol) & ~np.isnan(ref) & (got != ref)
    assert not bad.any(), (what, int(bad.sum()), np.argwhere(bad)[:3].tolist(), got[bad][:3],
                           ref[bad][:3], np.broadcast_to(tol, ref.shape)[bad][:3])


def check(z, ids, mask, g=(0.01, 0.002), out=None):
    half = 2.0 ** -8 if z.dtype == torch.bfloat16 else 2.0 ** -24
    gl = np.array(g, np.float32)
    ref = B.balance(host(z.float()), ids, mask, gl, half)
    r = L.moe_balance_loss(z, up(ids), mask=up(mask))
    eq(host(r.counts), ref["counts"], "counts")
    assert int(r.tokens) == ref["tokens"]
    near(r.mean_probs, ref["mean_probs"], ref["tol_mean_probs"], "mean probabilities")
    near(r.losses, ref["losses"], ref["tol_losses"], "losses")
    grad = L.moe_balance_loss_backward(z, ids.shape[1], r.counts, r.tokens, up(gl), mask=up(mask),
                                       out=out)
    near(grad, ref["grad"], ref["tol_grad"], "gradient")
    return r, grad, ref


EXPERTS = [1, 2, 3, 4, 7, 8, 16, 31, 32, 33, 60, 64, 65, 100, 127, 128, 129, 160, 255, 256, 257, 384,
           512, 513, 1000, 1024]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("E", EXPERTS)
def test_experts(E, dtype):
    say(f"balance E={E} {dtype}")
    for T, k in ((1, 1), (5, min(E, 3)), (70, min(E, 8)), (517, min(E, 2))):
        check(*case(E + T, T, E, k, dtype))


@pytest.mark.parametrize("T", [1, 2, 3, 4, 15, 16, 17, 63, 64, 65, 255, 256, 257, 1000, 1025, 4100,
                               20011, 70001])
def test_tokens(T):
    say(f"balance T={T}")
    check(*case(T, T, 64, 6, "f32", padded=0.2, dropped=0.1))
    check(*case(T, T, 40, 4, "bf16", masked=0.3))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_masks(dtype):
    """Closed experts, rows of nothing else, rows that the mask takes out and
    that hold anything, the type's lowest value, all rows out."""
    say(f"balance masks {dtype}")
    for T, E in ((40, 60), (300, 128), (50, 256), (33, 600)):
        z, ids, mask = case(T + E, T, E, 4, dtype, masked=0.4, padded=0.3)
        z[0] = float("-inf")
        z[1, :E - 1] = float("-inf")
        z[2] = torch.finfo(z.dtype).min
        z[3, 1:] = torch.finfo(z.dtype).min
        mask[:5] = True
        mask[5:7] = False
        z[5], z[6] = float("nan"), float("inf")
        ids[5:7] = 2 ** 31 - 1
        check(z, ids, mask, g=(0.01, 0.0))
        r, grad, _ = check(z, ids, np.zeros(T, bool))
        assert int(r.tokens) == 0 and not host(r.losses).any() and not host(grad.float()).any()


def test_large_logits_and_z_loss():
    say("balance, large logits")
    for s in (1e-6, 30.0, 1000.0):
        check(*case(7, 90, 64, 4, "f32", scale=s))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_nan_and_infinity_stay_in_their_rows(dtype):
    say(f"balance NaN {dtype}")
    z, ids, _ = case(3, 20, 48, 4, dtype)
    clean = z.clone()
    z[4, 7], z[9, 0] = float("nan"), float("inf")
    r = L.moe_balance_loss(z, up(ids))
    assert torch.isnan(r.losses).all()
    eq(host(r.counts), np.bincount(ids.ravel(), minlength=48), "counts")
    g = torch.tensor([0.1, 0.1], device=DEV)
    a = host(L.moe_balance_loss_backward(z, 4, r.counts, r.tokens, g).float())
    b = host(L.moe_balance_loss_backward(clean, 4, r.counts, r.tokens, g).float())
    bad = np.zeros(20, bool)
    bad[[4, 9]] = True
    assert np.isnan(a[bad]).any(1).all()
    eq(a[~bad], b[~bad], "other rows")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_rows_of_nan_and_masks_alone(dtype):
    """A row of NaN and -inf counts and is NaN; one of -inf alone does not."""
    say(f"balance, rows without a number, {dtype}")
    for E in (8, 60, 64, 200):
        z, ids, _ = case(E, 9, E, 2, dtype)
        z[2], z[5], z[7] = float("-inf"), float("nan"), float("-inf")
        z[7, E - 1] = float("nan")
        r = L.moe_balance_loss(z, up(ids))
        assert int(r.tokens) == 8 and torch.isnan(r.losses).all()
        eq(host(r.counts), np.bincount(np.delete(ids, 2, 0).ravel(), minlength=E), "counts")
        g = L.moe_balance_loss_backward(z, 2, r.counts, r.tokens, torch.ones(2, device=DEV))
        g = host(g.float())
        assert np.isnan(g[[5, 7]]).any(1).all() and not g[2].any()
        assert np.isfinite(np.delete(g, [5, 7], 0)).all()


def test_repeated_and_dropped_slots():
    say("balance, repeated slots")
    z, ids, _ = case(1, 30, 16, 5)
    ids[:, 1] = ids[:, 0]
    ids[3] = -1
    ids[4] = 16
    ids[5] = -2 ** 31
    check(z, ids, None)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_strides_and_alignment(dtype):
    """Views of wider tensors: every offset from a 16-byte boundary, odd row
    strides, a gradient in place and in rows of another stride; what lies beside
    the gradient stays."""
    say(f"balance strides {dtype}")
    for E, pitch in ((60, 64), (64, 71), (128, 136), (100, 101), (256, 264), (8, 24), (512, 520)):
        for at in (0, 1, 3, 4, 8):
            z, ids, mask = case(E + at, 37, E, 3, dtype, padded=0.2)
            big = torch.full((37, pitch + at), 5.0, device=DEV, dtype=z.dtype)
            v = big[:, at:at + E]
            v.copy_(z)
            out = torch.full((37, pitch + 9), 3.0, device=DEV, dtype=z.dtype)
            r, grad, ref = check(v, ids, mask, out=out[:, at:at + E])
            assert (out[:, :at] == 3).all() and (out[:, at + E:] == 3).all()
            check(z, ids, mask)
            # in place: the same values, whatever the rows of the gradient were
            L.moe_balance_loss_backward(v, 3, r.counts, r.tokens,
                                        torch.tensor([0.01, 0.002], device=DEV), mask=up(mask), out=v)
            assert torch.equal(v, grad)
            assert (big[:, :at] == 5).all() and (big[:, at + E:] == 5).all()


def test_refusals():
    say("balance refusals")
    z, ids, _ = case(1, 12, 16, 2)
    i = up(ids)
    ok = torch.ones(12, dtype=torch.bool, device=DEV)
    r = L.moe_balance_loss(z, i, mask=ok)
    for a, m in (((z, i.long()), None), ((z, i[:5]), None), ((z.t(), i), None), ((z[0], i), None),
                 ((z, i.t()), None), ((z, i), ok[:5]), ((z, i), ok.float()), ((z, i), ok.cpu()),
                 ((z[:, :1].expand(12, 16), i), None)):
        with pytest.raises(ValueError):
            L.moe_balance_loss(*a, mask=m)
    with pytest.raises(TypeError):
        L.moe_balance_loss(z.half(), i)
    g = torch.ones(2, device=DEV)
    for a in ((z, 2, r.counts[:3], r.tokens, g), (z, 2, r.counts, r.tokens, g[:1]),
              (z, 2, r.counts.long(), r.tokens, g), (z, 2, r.counts, r.counts, g)):
        with pytest.raises(ValueError):
            L.moe_balance_loss_backward(*a)
    with pytest.raises(L.NVFP4Error):
        L.moe_balance_loss_backward(z, 17, r.counts, r.tokens, g)


def test_empty():
    say("balance, no rows")
    z = torch.zeros(0, 16, device=DEV)
    r = L.moe_balance_loss(z, torch.zeros(0, 2, dtype=torch.int32, device=DEV))
    assert not host(r.losses).any() and not host(r.counts).any() and int(r.tokens) == 0
    assert not host(r.mean_probs).any()
    assert L.moe_balance_loss_backward(z, 2, r.counts, r.tokens,
                                       torch.ones(2, device=DEV)).shape == (0, 16)


def test_autograd_with_the_router():
    """The loss on moe_route's choice: autograd's gradient, through a layer
    before it, against the reference; no gradient, a second one, capture."""
    say("balance autograd")
    rng = np.random.default_rng(2)
    h = up(rng.standard_normal((96, 24)).astype(np.float32))
    w = up((rng.standard_normal((24, 32)) * 0.3).astype(np.float32)).requires_grad_()
    z = h @ w
    rt = L.moe_route(z.detach(), 4)
    mask = up(np.arange(96) < 80)
    r = P.moe_balance_loss(z, rt.topk_ids, mask)
    assert not r.counts.requires_grad and not r.mean_probs.requires_grad
    (0.01 * r.losses[0] + 0.001 * r.losses[1]).backward()
    ref = B.balance(host(z.detach()), host(rt.topk_ids), host(mask), [0.01, 0.001])
    near(r.losses.detach(), ref["losses"], ref["tol_losses"], "losses")
    hw = host(h).astype(np.float64)
    # the product behind it adds 96 terms of 32 bits
    tol = np.abs(hw).T @ (ref["tol_grad"] + 100 * B.U * np.abs(ref["grad"]))
    near(w.grad, hw.T @ ref["grad"], tol + 1e-12, "weights")
    offs = host(rt.expert_offsets)
    full = P.moe_balance_loss(z.detach(), rt.topk_ids)
    eq(host(full.counts), np.diff(offs), "counts are the products' group sizes")
    leaf = z.detach().requires_grad_()
    r = P.moe_balance_loss(leaf, rt.topk_ids)
    r.losses.mul_(2.0)                                  # an output like any other
    g2, = torch.autograd.grad(r.losses[0], leaf)
    g1, = torch.autograd.grad(P.moe_balance_loss(leaf, rt.topk_ids).losses[0], leaf)
    assert torch.equal(g2, 2 * g1)
    r = P.moe_balance_loss(leaf, rt.topk_ids)
    r.counts.zero_()                                    # the backward pass needs them
    with pytest.raises(RuntimeError, match="inplace"):
        torch.autograd.grad(r.losses.sum(), leaf)
    r = P.moe_balance_loss(leaf, rt.topk_ids)
    with pytest.raises(RuntimeError, match="second derivative"):
        torch.autograd.grad(r.losses.sum(), leaf, create_graph=True)
    g, = torch.autograd.grad(r.losses[1], leaf, allow_unused=True)
    assert torch.isfinite(g).all()


def test_captured():
    """Both calls in a graph: replayed on new inputs with eager work between;
    two graphs that hold their own workspaces."""
    say("balance captured")
    for T, E, k in ((30, 64, 4), (5000, 128, 8)):
        z, ids, mask = case(T, T, E, k, padded=0.2)
        sz, si, sm = z.clone(), up(ids), up(mask)
        gl = torch.tensor([0.3, 0.1], device=DEV)
        L.moe_balance_loss(sz, si, mask=sm)
        graphs = []
        for _ in range(2):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                r = L.moe_balance_loss(sz, si, mask=sm)
                grad = L.moe_balance_loss_backward(sz, k, r.counts, r.tokens, gl, mask=sm)
            graphs.append((g, r, grad))
        for i in range(4):
            sz.copy_(z.roll(i, 0) * (1 + i))
            si.copy_(up(ids).roll(i, 0))
            for g, _, _ in graphs:
                g.replay()
            e = L.moe_balance_loss(sz, si, mask=sm)
            eg = L.moe_balance_loss_backward(sz, k, e.counts, e.tokens, gl, mask=sm)
            torch.cuda.synchronize()
            for _, r, grad in graphs:
                assert torch.equal(r.losses, e.losses) and torch.equal(r.counts, e.counts)
                assert torch.equal(r.mean_probs, e.mean_probs) and torch.equal(grad, eg)


def test_another_stream_and_deterministic():
    say("balance streams")
    z, ids, mask = case(4, 9000, 96, 6, padded=0.1)
    zi, ii, mi = z, up(ids), up(mask)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        a = [L.moe_balance_loss(zi, ii, mask=mi) for _ in range(3)]
    b = L.moe_balance_loss(zi, ii, mask=mi)
    torch.cuda.current_stream().wait_stream(st)
    for r in a:
        assert torch.equal(r.losses, b.losses) and torch.equal(r.mean_probs, b.mean_probs)
        assert torch.equal(r.counts, b.counts)
