"""Trains a small stack of MoE blocks, then serves it from e4m3 and e2m1 weights.

    python examples/moe_block.py [--tokens 512] [--steps 20] [--state-bits 8]

A block is norm -> router -> experts -> norm with a gate per token and the
residual; a block's exit norm and the next one's entry norm are one pass.  The
optimiser takes all parameters in one launch.  After training, the experts'
weights become e4m3 codes with a scale per 128 x 128 block, or e2m1 codes with a
scale per 32 of a row, and the same blocks run for inference, for the whole batch
and for single tokens (those of the latter through router and layer in two launches).
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import combine_topk_multihot_gb300 as moe  # noqa: E402


class Stack:
    def __init__(self, blocks: int, H: int, E: int, K: int, I: int, seed: int = 0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rnd = lambda *s, std: torch.randn(*s, generator=g, device="cuda") * std  # noqa: E731
        self.K = K
        self.entry = torch.ones(H, device="cuda", requires_grad=True)
        self.blocks = []
        for _ in range(blocks):
            b = dict(router=rnd(E, H, std=H ** -0.5).bfloat16(), W1=rnd(E, 2 * I, H, std=H ** -0.5).bfloat16(),
                     W2=rnd(E, H, I, std=I ** -0.5).bfloat16(), exit=torch.ones(H, device="cuda"),
                     gate=torch.zeros(H, 1, device="cuda"), next=torch.ones(H, device="cuda"))
            self.blocks.append({k: v.requires_grad_(True) for k, v in b.items()})
        self.blocks[-1].pop("next")
        self.fp8 = self.fp4 = None

    def parameters(self):
        return [self.entry] + [p for b in self.blocks for p in b.values()]

    def to_fp8(self):
        """The experts' weights as codes and scales, for inference."""
        self.fp8 = [(moe.moe_quantize_fp8_block(b["W1"].detach(), 128), moe.moe_quantize_fp8_block(b["W2"].detach(), 128))
                    for b in self.blocks]

    def to_fp4(self):
        """The same in 4 bits."""
        self.fp8, self.fp4 = None, [(moe.moe_quantize_fp4_block(b["W1"].detach()), moe.moe_quantize_fp4_block(b["W2"].detach()))
                                    for b in self.blocks]

    def __call__(self, x):
        normed, _ = torch.ops.moe_gb300.norm_in(x, self.entry, 1e-6, 0.0)
        for i, b in enumerate(self.blocks):
            W1, W2, kept = b["W1"], b["W2"], {}
            if self.fp8 is not None or self.fp4 is not None:
                (W1, s1), (W2, s2) = (self.fp8 or self.fp4)[i]
                kept = {"fp8" if self.fp8 is not None else "fp4": (s1, s2)}
            gate = (normed.float() @ b["gate"]).squeeze(1)
            x, normed = moe.moe_block(x, normed, b["router"], self.K, W1, W2, b["exit"], gate=gate,
                                      next_weight=b.get("next"), few=self.fp4 is not None, **kept)
        return x


def train(stack, x, target, steps: int, lr: float, state_bits: int):
    """Returns the losses."""
    params = stack.parameters()
    opt = moe.AdamWState([p.detach() for p in params], state_bits=state_bits, master=True)
    decay = [0.01 if p.dim() == 3 else 0.0 for p in params]     # the experts' matrices alone
    losses = []
    for _ in range(steps):
        loss = (stack(x).float() - target).square().mean()
        grads = torch.autograd.grad(loss, params)
        moe.moe_adamw_step(opt, grads, lr, beta2=0.95, weight_decay=decay)
        losses.append(loss.detach())
    return torch.stack(losses).tolist()


def serve(stack, x):
    """How far, by the norm, the outputs from e4m3 and e2m1 weights are from those from bf16, and those of the first four
    tokens one at a time from those in the batch."""
    with torch.no_grad():
        out = dict(bf16=stack(x))
        for kind, convert in (("fp8", stack.to_fp8), ("fp4", stack.to_fp4)):
            convert()
            out[kind] = stack(x)
            out[kind + " one"] = torch.cat([stack(x[i:i + 1]) for i in range(4)])
    rel = lambda p, q: float((out[p].float() - q.float()).norm() / q.float().norm())  # noqa: E731
    return {"fp8": rel("fp8", out["bf16"]), "fp8 one": rel("fp8 one", out["fp8"][:4]),
            "fp4": rel("fp4", out["bf16"]), "fp4 one": rel("fp4 one", out["fp4"][:4])}


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--tokens", type=int, default=512)
    ap.add_argument("--blocks", type=int, default=2)
    ap.add_argument("--hidden", type=int, default=512)
    ap.add_argument("--experts", type=int, default=16)
    ap.add_argument("--top-k", type=int, default=4)
    ap.add_argument("--intermediate", type=int, default=256)
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--lr", type=float, default=2e-3)
    ap.add_argument("--state-bits", type=int, choices=(8, 32), default=8)
    a = ap.parse_args(argv)
    stack = Stack(a.blocks, a.hidden, a.experts, a.top_k, a.intermediate)
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(a.tokens, a.hidden, generator=g, device="cuda").bfloat16()
    target = torch.randn(a.tokens, a.hidden, generator=g, device="cuda") + x.float()
    losses = train(stack, x, target, a.steps, a.lr, a.state_bits)
    off = serve(stack, x)
    print(f"loss {losses[0]:.4f} -> {losses[-1]:.4f} in {a.steps} steps with {a.state_bits}-bit states; "
          f"e4m3 experts against bf16: {off['fp8']:.4f}; one token at a time: {off['fp8 one']:.4f}; "
          f"e2m1 experts against bf16: {off['fp4']:.4f}; one token at a time: {off['fp4 one']:.4f}")
    return losses, off["fp8"], off["fp8 one"]


if __name__ == "__main__":
    main()
