"""The rollout-trainer log-prob gap of one MoE layer, by how the rollout
computes it.

    python -m nvfp4_w4a4_moe_quant_amd.logprob_gap [seed]

The QUADS pages judge a rollout by the gap between the log-probabilities that
it sampled with and the trainer's (blog post, section "What it buys").  Here,
on a small seeded layer and vocabulary head: the trainer's forward takes the
fake-quantized weights (nvfp4_qdq) and unquantized activations; the rollout
is naive W4A4, W4A4 with RAC, the decode-step layer, which leaves the
activations alone too, or an INT8 layer (W8A8) on the plain weights, which is
measured against a trainer on those: the gaps to the two trainers do not compare.
Prints, per rollout, the mean and largest absolute difference of the sampled
tokens' log-probabilities, the mean entropy and which trainer, and how evenly
the layer's router spreads the tokens.
"""
from __future__ import annotations

import sys
from typing import Dict, Iterator, Tuple

import torch

from . import _lib as L
from . import datagen as D
from . import pipeline as P


def _bf16(a, dev) -> torch.Tensor:
    return torch.from_numpy(a).to(dev).to(torch.bfloat16)


def gaps(seed: int = 1, vocab: int = 32000, device: str = "cuda:0", int8: bool = False
         ) -> Iterator[Tuple[str, Dict[str, float]]]:
    """(rollout, figures) for the three rollouts of one seeded layer, and with
    int8 for the INT8 one."""
    w = D.small_moe(seed, T=64, E=16, topk=4, H=512, I=256, n_outliers=8)
    gen = torch.Generator(device=device)
    gen.manual_seed(seed)
    x, lg = _bf16(D.activations(w), device), torch.from_numpy(D.router_logits(w)).to(device)
    gu = {e: _bf16(m, device) for e, m in D.expert_weights(w, "gate_up")}
    down = {e: _bf16(m, device) for e, m in D.expert_weights(w, "down")}
    wgu = P.quantize_weights(gu.items(), w.E, 2 * w.I, w.H, device)
    wd = P.quantize_weights(down.items(), w.E, w.H, w.I, device)
    head = torch.randn((w.H, vocab), generator=gen, device=device) * (2.0 / w.H ** 0.5)

    def logits(y: torch.Tensor) -> torch.Tensor:
        y = x.float() + y.float()
        return (y * y.square().mean(1, keepdim=True).add(1e-6).rsqrt()) @ head

    rt = L.moe_route(lg, w.topk)

    def forward(weight) -> torch.Tensor:
        """The trainer's forward, expert by expert."""
        y = torch.zeros((w.T, w.H), device=device)
        for e in range(w.E):
            t, s = torch.nonzero(rt.topk_ids == e, as_tuple=True)
            g = x[t].float() @ weight(gu[e]).T.contiguous()
            h = torch.nn.functional.silu(g[:, :w.I]) * g[:, w.I:]
            h = h @ weight(down[e]).T.contiguous()
            y.index_add_(0, t, rt.topk_weights[t, s, None] * h)
        return logits(y)

    trainer = forward(lambda m: L.nvfp4_qdq(m, out_dtype=torch.float32))
    args = (x, lg, wgu, wd, w.topk)
    rollouts = {
        "naive W4A4": lambda: P.moe_block(*args, None, None, out_dtype=torch.float32)["out"],
        "W4A4 + RAC": lambda: P.moe_block(*args, w.n_select_x, w.n_select_h,
                                          out_dtype=torch.float32)["out"],
        "decode-step layer": lambda: P.moe_decode(*args).out,
    }
    if int8:
        w8gu = P.int8_quantize_weights(gu.items(), w.E, 2 * w.I, w.H, device)
        w8d = P.int8_quantize_weights(down.items(), w.E, w.H, w.I, device)
        plain = forward(lambda m: m.float())
        rollouts["INT8 W8A8"] = lambda: P.int8_moe_block(x, lg, w8gu, w8d, w.topk,
                                                         out_dtype=torch.float32)["out"]
    for name, layer in rollouts.items():
        z = logits(layer())
        tokens = torch.multinomial(torch.softmax(z, 1), 1, generator=gen)[:, 0]
        roll = L.token_logprobs(z, tokens)
        against = plain if name == "INT8 W8A8" else trainer
        gap = (roll.logprobs - L.token_logprobs(against, tokens).logprobs).abs()
        yield name, dict(mean=float(gap.mean()), max=float(gap.max()),
                         entropy=float(roll.entropy.mean()))


def router(seed: int = 1, device: str = "cuda:0") -> Dict[str, float]:
    """Balance loss (1 where every expert gets as much), z-loss, and the fullest
    and emptiest expert's share of the mean, of the layer's router."""
    w = D.small_moe(seed, T=64, E=16, topk=4, H=512, I=256, n_outliers=8)
    lg = torch.from_numpy(D.router_logits(w)).to(device)
    b = P.moe_balance_loss(lg, L.moe_route(lg, w.topk).topk_ids)
    share = b.counts.float() / (w.T * w.topk / w.E)
    return dict(balance=float(b.losses[0]), z=float(b.losses[1]), fullest=float(share.max()),
                emptiest=float(share.min()))


def main() -> None:
    seed = int(sys.argv[1]) if len(sys.argv) > 1 else 1
    for name, f in gaps(seed, int8=True):
        print(f"{name:20s} |log-prob gap| mean {f['mean']:.5f}  max {f['max']:.5f}  "
              f"entropy {f['entropy']:.3f}  trainer on "
              f"{'plain' if name == 'INT8 W8A8' else 'fake-quantized'} weights")
    print("The two trainers' gaps do not compare: INT8's holds the rounding of its weights, the "
          "others' do not.")
    r = router(seed)
    print(f"router: balance loss {r['balance']:.4f}, z-loss {r['z']:.3f}, experts from "
          f"{r['emptiest']:.2f} to {r['fullest']:.2f} of the mean load")


if __name__ == "__main__":
    main()
