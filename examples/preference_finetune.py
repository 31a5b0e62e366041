"""Fine-tunes the LoRA adapters of a small frozen model on preference pairs, on rollouts with
advantages, or on a teacher's record: logits -> loss with its gradient -> adapter gradients -> AdamW.

  python examples/preference_finetune.py [--loss preference|policy|distill] [--steps 30] [--state-bits 8|32]
                                          [--entropy-bonus 0.001]

The model is a frozen random embedding, a hidden layer and an output layer, both of the latter
with an adapter (lora_linear).  The reference model is the same with the adapters off; the teacher
the same with adapters of its own, of which the record holds the 32 most probable tokens of each
row and the mass of the rest.  Inputs are random sequences made from a seed.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from lora_rank_adapter_gb300 import torch_ops  # noqa: E402

VOCAB, WIDTH, RANK, SCALE = 1000, 256, 16, 2.0


class Model:
    def __init__(self, device, gen):
        def randn(*shape, std):
            return (torch.randn(*shape, generator=gen, device=device) * std).bfloat16()

        self.embed = randn(VOCAB, WIDTH, std=1.0)
        self.hidden, self.out = randn(WIDTH, WIDTH, std=WIDTH ** -0.5), randn(WIDTH, VOCAB, std=WIDTH ** -0.5)
        self.adapters = []
        for wide in (WIDTH, VOCAB):          # A random, B zero: the adapter starts as no change
            A, B = randn(WIDTH, RANK, std=WIDTH ** -0.5), torch.zeros(RANK, wide, device=device).bfloat16()
            self.adapters.append((A.requires_grad_(), B.requires_grad_()))

    def parameters(self):
        return [p for pair in self.adapters for p in pair]

    def logits(self, ids, adapters=True):
        x = self.embed[ids]
        for W, (A, B) in zip((self.hidden, self.out), self.adapters):
            base = x @ W
            y = torch_ops.lora_linear(x, A, B, base, SCALE) if adapters else base
            x = torch.tanh(y) if W is self.hidden else y
        return x


def batch(gen, device, sequences, longest=40, prompt=6):
    """Packed random sequences: inputs, labels moved by one with the prompts ignored, and offsets."""
    lens = torch.randint(prompt + 4, longest, (sequences,), generator=gen, device=device)
    cu = torch.zeros(sequences + 1, dtype=torch.int32, device=device)
    cu[1:] = lens.cumsum(0)
    T = int(cu[-1])
    ids = torch.randint(0, VOCAB, (T,), generator=gen, device=device)
    labels = ids.roll(-1)
    place = torch.arange(T, device=device) - cu[:-1].long().repeat_interleave(lens)
    last = place == lens.repeat_interleave(lens) - 1
    labels[(place < prompt - 1) | last] = -100
    return ids, labels, cu, lens


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--loss", choices=("preference", "policy", "distill"), default="preference")
    ap.add_argument("--steps", type=int, default=30)
    ap.add_argument("--state-bits", type=int, choices=(8, 32), default=8)
    ap.add_argument("--entropy-bonus", type=float, default=0.0, help="of the policy loss")
    ap.add_argument("--seed", type=int, default=0)
    args = ap.parse_args(argv)
    device = "cuda:0"
    gen = torch.Generator(device).manual_seed(args.seed)
    model = Model(device, gen)
    opt = torch_ops.AdamW(model.parameters(), lr=2e-3, weight_decay=0.0, state_bits=args.state_bits, masters=True,
                          max_norm=1.0)
    ids, labels, cu, lens = batch(gen, device, 8)
    with torch.no_grad():                    # the reference model: the adapters off
        before = model.logits(ids, adapters=False)
        ref_seq = torch_ops.preference_loss(before, labels, cu)[2]
        ref_tok = torch_ops.token_logps(before, labels)
    counted = (labels >= 0).float()
    of = torch.arange(8, device=device).repeat_interleave(lens)
    advantages = torch.randn(8, generator=gen, device=device)[of]
    per_sequence = torch.zeros(8, device=device).index_add_(0, of, counted)
    weights = 1.0 / (8 * per_sequence.clamp(min=1))[of]
    if args.loss == "distill":               # the teacher: other adapters on the same frozen weights
        teacher = Model(device, torch.Generator(device).manual_seed(args.seed))
        with torch.no_grad():
            for _, B in teacher.adapters:
                B.normal_(0.0, 0.3, generator=gen)
            record = torch_ops.top_logps(teacher.logits(ids), 32)
        weights = counted / counted.sum()
    losses = []
    for step in range(args.steps):
        logits = model.logits(ids)
        if args.loss == "preference":
            loss, _, _ = torch_ops.preference_loss(logits, labels, cu, ref_seq, beta=0.1)
        elif args.loss == "policy":
            loss, _, _ = torch_ops.policy_loss(logits, labels, ref_tok, advantages, weights, ref_logps=ref_tok,
                                               clip_high=0.28, kl_beta=0.02)
            if args.entropy_bonus:
                loss = loss - args.entropy_bonus * (weights * torch_ops.top_logps(logits, 0, labels).entropy).sum()
        else:
            loss, _ = torch_ops.distill_loss(logits, record.ids, record.logps, record.rest, weights)
        opt.zero_grad()
        loss.backward()
        opt.step()
        losses.append(float(loss.detach()))
        if step % 10 == 0 or step == args.steps - 1:
            print(f"step {step:3d}  loss {losses[-1]:.5f}  gradient norm {float(opt.norm[0]):.4f}")
    return losses


if __name__ == "__main__":
    main()
