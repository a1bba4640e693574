"""The rollout-trainer log-prob gap of one MoE layer, by how the rollout
computes it.

    python -m nvfp4_w4a4_moe_quant_amd.logprob_gap [seed]

The QUADS pages judge a rollout by the gap between the log-probabilities that
it sampled with and the trainer's (blog post, section "What it buys").  Here,
on a small seeded layer and vocabulary head: the trainer's forward takes the
fake-quantized weights (nvfp4_qdq) and unquantized activations; the rollout
is naive W4A4, W4A4 with RAC, or the decode-step layer, which leaves the
activations alone too.  Prints, per rollout, the mean and largest absolute
difference of the sampled tokens' log-probabilities and the mean entropy.
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


def gaps(seed: int = 1, vocab: int = 32000, device: str = "cuda:0"
         ) -> Iterator[Tuple[str, Dict[str, float]]]:
    """(rollout, figures) for the three rollouts of one seeded layer."""
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
    y = torch.zeros((w.T, w.H), device=device)
    for e in range(w.E):  # the trainer's forward, expert by expert
        t, s = torch.nonzero(rt.topk_ids == e, as_tuple=True)
        g = x[t].float() @ L.nvfp4_qdq(gu[e], out_dtype=torch.float32).T.contiguous()
        h = torch.nn.functional.silu(g[:, :w.I]) * g[:, w.I:]
        h = h @ L.nvfp4_qdq(down[e], out_dtype=torch.float32).T.contiguous()
        y.index_add_(0, t, rt.topk_weights[t, s, None] * h)
    trainer = logits(y)
    args = (x, lg, wgu, wd, w.topk)
    rollouts = {
        "naive W4A4": lambda: P.moe_block(*args, None, None, out_dtype=torch.float32)["out"],
        "W4A4 + RAC": lambda: P.moe_block(*args, w.n_select_x, w.n_select_h,
                                          out_dtype=torch.float32)["out"],
        "decode-step layer": lambda: P.moe_decode(*args).out,
    }
    for name, layer in rollouts.items():
        z = logits(layer())
        tokens = torch.multinomial(torch.softmax(z, 1), 1, generator=gen)[:, 0]
        roll = L.token_logprobs(z, tokens)
        gap = (roll.logprobs - L.token_logprobs(trainer, tokens).logprobs).abs()
        yield name, dict(mean=float(gap.mean()), max=float(gap.max()),
                         entropy=float(roll.entropy.mean()))


def main() -> None:
    seed = int(sys.argv[1]) if len(sys.argv) > 1 else 1
    for name, f in gaps(seed):
        print(f"{name:20s} |log-prob gap| mean {f['mean']:.5f}  max {f['max']:.5f}  "
              f"entropy {f['entropy']:.3f}")


if __name__ == "__main__":
    main()
