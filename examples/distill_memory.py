"""Train a small n-gram memory against a teacher's top logits, then decode with it.

The memory hashes the last ids of every position to rows of a table, reads the
rows (engram_lookup), mixes them along the sequence with a gated linear
recurrence and projects the states to logits.  Its loss is the distance from a
teacher of which only the largest logits of each position are kept
(engram_distill); the gradients go back through the recurrence
(engram_recurrence_grad) to the table's rows (engram_lookup_grad_rows), of which
a step touches few.  The dense projections are torch products.

Decoding runs the same operators one position at a time: engram_hash_step,
engram_lookup and engram_recurrence_step.

    python examples/distill_memory.py
"""
from __future__ import annotations

import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import hashed_gram_conditional_gb300 as eg  # noqa: E402

ROW_DIM, WIDTH, TOP, TAU = 32, 256, 16, 2.0


class Memory:
    """Table, gates and projections of the memory, and one training step of them."""

    def __init__(self, vocab: int, base_rows: int = 4099, seed: int = 0, device="cuda"):
        gen = torch.Generator(device=device).manual_seed(seed)

        def weight(rows, cols):
            w = torch.empty((rows, cols), dtype=torch.bfloat16, device=device)
            return w.normal_(0.0, rows ** -0.5, generator=gen)

        self.vocab = vocab
        self.layout = eg.build_layout(vocab, base_rows, [1], max_ngram=3, n_heads=4)
        self.token_map = torch.arange(vocab, dtype=torch.int32, device=device)
        rows, cols = self.layout.total_rows(0), self.layout.n_cols
        self.table = torch.empty((rows, ROW_DIM), dtype=torch.float32, device=device).normal_(0.0, 1.0, generator=gen)
        self.scale = 1.0 / math.sqrt(cols)
        self.w_x, self.w_g = weight(cols * ROW_DIM, WIDTH), weight(cols * ROW_DIM, WIDTH)
        self.w_out = weight(WIDTH, vocab)
        self.status = eg.new_status(device)

    def rows_of(self, raw_ids, cu):
        """The row ids of every position; image positions (DEAD) have none."""
        ids, mask = eg.engram_hash(self.layout, 0, raw_ids, cu, self.token_map, status=self.status)
        return ids.masked_fill_((mask != 0)[:, None], eg.DEAD), mask

    def forward(self, raw_ids, cu, carry=None):
        ids, mask = self.rows_of(raw_ids, cu)
        e = eg.engram_lookup(self.table, ids, self.scale, status=self.status).bfloat16()
        x, g = e @ self.w_x, e @ self.w_g
        y = eg.engram_recurrence(x, g, cu, mask=mask, carry=carry, status=self.status)
        return ids, mask, e, x, g, y, y @ self.w_out

    def step(self, raw_ids, cu, teacher_ids, teacher_logits, lr: float = 0.05) -> float:
        """One step of gradient descent, each weight moved by the fraction lr of its size; returns the mean loss."""
        T = raw_ids.numel()
        carry = eg.recurrence_carry(T, WIDTH, raw_ids.device)
        ids, mask, e, x, g, y, logits = self.forward(raw_ids, cu, carry)
        weight = (mask == 0).float() / T  # image positions teach nothing
        loss = eg.engram_distill(logits, teacher_ids, teacher_logits, TAU, weight=weight, dlogits=logits,
                                 status=self.status)  # the gradient takes the logits' place
        dy = logits @ self.w_out.t()
        dx, dg = eg.engram_recurrence_grad(dy, x, g, carry, cu, mask=mask, status=self.status)
        de = dx @ self.w_x.t() + dg @ self.w_g.t()
        rows, grad, count = eg.engram_lookup_grad_rows(de, ids, self.table.shape[0], self.scale, status=self.status)
        for w, a, d in ((self.w_out, y, logits), (self.w_x, e, dx), (self.w_g, e, dg)):
            d = (a.t() @ d).float()
            w.copy_(w.float() - d * (lr * w.float().norm() / d.norm().clamp_min(1e-20)))
        # the rows past the count are -1 with zero gradients: they add nothing to row 0
        grad *= -lr * self.table.norm() / grad.norm().clamp_min(1e-20)
        self.table.index_add_(0, rows.clamp_min(0).long(), grad)
        return loss.sum().item()

    def decode(self, raw_ids):
        """Logits of one sequence, position by position with carried states."""
        dev = raw_ids.device
        hist = torch.full((1, self.layout.max_ngram - 1), self.layout.pad_id, dtype=torch.int32, device=dev)
        state = torch.zeros((1, WIDTH), device=dev)
        slot = torch.zeros(1, dtype=torch.int32, device=dev)
        out = []
        for t in range(raw_ids.numel()):
            ids, mask = eg.engram_hash_step(self.layout, 0, raw_ids[t:t + 1], slot, self.token_map, hist,
                                            status=self.status)
            image = mask != 0  # no rows and no slot: the state stays, and y is 0
            e = eg.engram_lookup(self.table, ids.masked_fill_(image[:, None], eg.DEAD), self.scale,
                                 status=self.status).bfloat16()
            y = eg.engram_recurrence_step(e @ self.w_x, e @ self.w_g, slot.masked_fill(image, -1), state,
                                          status=self.status)
            out.append(y @ self.w_out)
        return torch.cat(out)


def batch(vocab: int, tokens: int, seqs: int, seed: int, device="cuda"):
    """Token ids of packed sequences, and a teacher's top logits that depend on the last two of them."""
    gen = torch.Generator(device=device).manual_seed(seed)
    ids = torch.randint(0, vocab, (tokens,), generator=gen, device=device, dtype=torch.int32)
    ids = torch.where(torch.rand(tokens, generator=gen, device=device) < 0.6, ids % 7, ids)  # some are frequent
    cu = torch.linspace(0, tokens, seqs + 1, device=device).long()
    pair = ids.long() * 31 + torch.cat([ids[:1], ids[:-1]]).long()
    k = torch.arange(TOP, device=device)
    teacher_ids = ((pair[:, None] * 2654435761 + k * (vocab // TOP)) % vocab).to(torch.int32)
    teacher_logits = (6.0 - 0.5 * k.float()).expand(tokens, TOP).contiguous()
    return ids, cu, teacher_ids, teacher_logits


def main(steps: int = 60, vocab: int = 1000, tokens: int = 2048) -> list:
    memory = Memory(vocab)
    data = batch(vocab, tokens, 8, 1)
    losses = [memory.step(*data) for _ in range(steps)]
    assert memory.status.item() == 0
    return losses


if __name__ == "__main__":
    found = main()
    for i in range(0, len(found), 10):
        print(f"step {i:3d}  loss {found[i]:.4f}")
    print(f"step {len(found) - 1:3d}  loss {found[-1]:.4f}")
