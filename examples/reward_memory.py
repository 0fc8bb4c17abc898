"""Train a memory block on rewards of sampled tokens, then decode with it.

The block reads rows of an n-gram table (engram_lookup) as its residual stream,
and from the stream's norm (engram_norm_add) queries, keys, values and gates for
a matrix-valued memory in each head (engram_delta).  What the memory answers is
normalised by heads, gated and added to the stream, whose norm gives the logits:
all of that is one more engram_norm_add.  Its loss is the clipped policy loss of
tokens that were sampled earlier, with a KL term towards the weights it began with
(engram_policy).  The gradients go back through engram_norm_add_grad,
engram_delta_grad and engram_lookup_grad_rows.  The dense projections are torch
products.

Decoding runs the same operators one position at a time, with engram_delta_step.

    python examples/reward_memory.py
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import hashed_gram_conditional_gb300 as eg  # noqa: E402

KEYS, HEADS, DIM = 2, 4, 32  # key heads, value heads, the width of each
WIDTH = HEADS * DIM


class Block:
    """Table, projections and norms of the block, and one training step of them."""

    def __init__(self, vocab: int, base_rows: int = 1021, seed: int = 0, device="cuda", dtype=torch.bfloat16):
        gen = torch.Generator(device=device).manual_seed(seed)

        def weight(cols):
            w = torch.empty((WIDTH, cols), dtype=dtype, device=device)
            return w.normal_(0.0, WIDTH ** -0.5, generator=gen)

        self.vocab, self.dtype = vocab, dtype
        self.layout = eg.build_layout(vocab, base_rows, [1], max_ngram=3, n_heads=2)
        self.token_map = torch.arange(vocab, dtype=torch.int32, device=device)
        rows, self.cols = self.layout.total_rows(0), self.layout.n_cols
        self.table = torch.empty((rows, WIDTH // self.cols), dtype=dtype, device=device).normal_(0.0, 1.0, generator=gen)
        self.proj = dict(q=weight(KEYS * DIM), k=weight(KEYS * DIM), v=weight(WIDTH), z=weight(WIDTH), g=weight(HEADS),
                         b=weight(HEADS), out=weight(vocab))
        one = lambda n, x=1.0: torch.full((n,), x, device=device)  # noqa: E731
        # norms: of the stream, of a head's answers, of the stream behind the block; the residual scale
        self.norm = dict(first=one(WIDTH), head=one(DIM), scale=one(WIDTH, 0.5), last=one(WIDTH))
        self.unit = one(DIM, DIM ** -0.5)  # a key's norm is 1
        self.status = eg.new_status(device)

    def rows_of(self, raw_ids, cu):
        """The row ids of every position; image positions (DEAD) have none."""
        ids, mask = eg.engram_hash(self.layout, 0, raw_ids, cu, self.token_map, status=self.status)
        return ids.masked_fill_((mask != 0)[:, None], eg.DEAD), mask

    def _inputs(self, ids):
        s = dict(h0=eg.engram_lookup(self.table, ids, status=self.status))
        s["x0"], _ = eg.engram_norm_add(s["h0"], self.norm["first"])
        for n in ("q", "k", "v", "z", "g", "b"):
            s[n] = s["x0"] @ self.proj[n]
        for n in ("q", "k"):
            s[n + "n"], _ = eg.engram_norm_add(s[n], self.unit, groups=KEYS)
        return s

    def _outputs(self, s):
        s["h1"], s["x1"] = eg.engram_norm_add(s["y"], self.norm["head"], gate=s["z"], h=s["h0"], scale=self.norm["scale"],
                                              w_next=self.norm["last"], groups=HEADS)
        s["logits"] = s["x1"] @ self.proj["out"]
        return s

    def forward(self, raw_ids, cu, carry=None):
        ids, mask = self.rows_of(raw_ids, cu)
        s = self._inputs(ids)
        s.update(ids=ids, mask=mask)
        s["y"] = eg.engram_delta(s["qn"], s["kn"], s["v"], s["g"], s["b"], cu, KEYS, mask=mask, carry=carry,
                                 status=self.status)
        return self._outputs(s)

    def logp(self, raw_ids, cu, sampled):
        """The sampled tokens' log-probabilities under the present weights."""
        s = self.forward(raw_ids, cu)
        none = torch.zeros(raw_ids.numel(), device=raw_ids.device)
        return eg.engram_policy(s["logits"], sampled, none, status=self.status)[1]

    def gradients(self, raw_ids, cu, sampled, advantage, old_logp=None, ref_logp=None, kl=0.0):
        """(loss of every position, gradient of every weight by name; the table's as (rows, gradient))."""
        T = raw_ids.numel()
        carry = eg.delta_carry(T, cu.numel() - 1, KEYS, HEADS, DIM, DIM, raw_ids.device)
        s = self.forward(raw_ids, cu, carry)
        weight = (s["mask"] == 0).float() / T
        loss, _ = eg.engram_policy(s["logits"], sampled, advantage, old_logp=old_logp, ref_logp=ref_logp, kl=kl,
                                   weight=weight, dlogits=s["logits"], status=self.status)
        grads = dict(out=s["x1"].t() @ s["logits"])  # the gradient has taken the logits' place
        dx1 = s["logits"] @ self.proj["out"].t()
        dy, dz, dh0, grads["head"], grads["scale"], grads["last"] = eg.engram_norm_add_grad(
            None, s["y"], self.norm["head"], gate=s["z"], scale=self.norm["scale"], h_out=s["h1"], dx=dx1,
            w_next=self.norm["last"], groups=HEADS)
        dqn, dkn, dv, dg, db = eg.engram_delta_grad(dy, s["qn"], s["kn"], s["v"], s["g"], s["b"], carry, cu, KEYS,
                                                    mask=s["mask"], status=self.status)
        dq, dk = (eg.engram_norm_add_grad(d, s[n], self.unit, groups=KEYS, residual=False)[0]
                  for d, n in ((dqn, "q"), (dkn, "k")))
        dx0 = torch.zeros_like(s["x0"])
        for n, d in (("q", dq), ("k", dk), ("v", dv), ("z", dz), ("g", dg), ("b", db)):
            grads[n] = s["x0"].t() @ d
            dx0 += d @ self.proj[n].t()
        d, _, _, grads["first"], _, _ = eg.engram_norm_add_grad(dx0, s["h0"], self.norm["first"], residual=False)
        rows, grad, _ = eg.engram_lookup_grad_rows(d + dh0, s["ids"], self.table.shape[0], status=self.status)
        grads["table"] = (rows, grad)
        return loss, grads

    def step(self, *batch, lr: float = 0.02, **how) -> float:
        """One step of gradient descent, each weight moved by the fraction lr of its size; returns the mean loss."""
        loss, grads = self.gradients(*batch, **how)
        rows, grad = grads.pop("table")
        # the rows past the count are -1 with zero gradients: they add nothing to row 0
        grad = grad * (-lr * self.table.float().norm() / grad.norm().clamp_min(1e-20))
        self.table.copy_(self.table.float().index_add_(0, rows.clamp_min(0).long(), grad))
        for name, d in grads.items():
            w = self.proj.get(name, self.norm.get(name))
            w.copy_(w.float() - d.float() * (lr * w.float().norm() / d.float().norm().clamp_min(1e-20)))
        return loss.sum().item()

    def decode(self, raw_ids):
        """Logits of one sequence, position by position with carried states."""
        dev = raw_ids.device
        hist = torch.full((1, self.layout.max_ngram - 1), self.layout.pad_id, dtype=torch.int32, device=dev)
        state = torch.zeros((1, HEADS, DIM, DIM), device=dev)
        slot = torch.zeros(1, dtype=torch.int32, device=dev)
        out = []
        for t in range(raw_ids.numel()):
            ids, mask = eg.engram_hash_step(self.layout, 0, raw_ids[t:t + 1], slot, self.token_map, hist,
                                            status=self.status)
            image = mask != 0  # no rows and no slot: the state stays, and y is 0
            s = self._inputs(ids.masked_fill_(image[:, None], eg.DEAD))
            s["y"] = eg.engram_delta_step(s["qn"], s["kn"], s["v"], s["g"], s["b"], slot.masked_fill(image, -1), state, KEYS,
                                          status=self.status)
            out.append(self._outputs(s)["logits"])
        return torch.cat(out)


def batch(vocab: int, tokens: int, seqs: int, seed: int, device="cuda"):
    """Token ids of packed sequences with image spans, tokens sampled after them and their advantages: of what follows
    a token's successor, more is better."""
    gen = torch.Generator(device=device).manual_seed(seed)
    ids = torch.randint(0, vocab, (tokens,), generator=gen, device=device, dtype=torch.int32)
    cu = torch.linspace(0, tokens, seqs + 1, device=device).long()
    sampled = torch.randint(0, vocab, (tokens,), generator=gen, device=device, dtype=torch.int32)
    sampled = torch.where(torch.rand(tokens, generator=gen, device=device) < 0.1, -1, sampled)  # prompts
    good = (sampled.long() - ids.long()) % vocab < vocab // 2
    advantage = torch.where(good, 1.0, -1.0) + 0.1 * torch.randn(tokens, generator=gen, device=device)
    return ids, cu, sampled, advantage


def main(steps: int = 20, vocab: int = 500, tokens: int = 1024) -> list:
    block = Block(vocab)
    ids, cu, sampled, advantage = batch(vocab, tokens, 6, 1)
    old = block.logp(ids, cu, sampled)
    losses = [block.step(ids, cu, sampled, advantage, old_logp=old, ref_logp=old, kl=0.05) for _ in range(steps)]
    assert block.status.item() == 0
    return losses


if __name__ == "__main__":
    found = main()
    for i in range(0, len(found), 5):
        print(f"step {i:3d}  loss {found[i]:.4f}")
    print(f"step {len(found) - 1:3d}  loss {found[-1]:.4f}")
