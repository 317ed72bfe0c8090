"""Decode with an 8-bit lm_head: embed, project, draw, embed the drawn token.

The tied table is kept twice: in bf16 for the lookups and as int8 rows with
one scale per vocabulary row for the projection.  No model stands between the
two here; a running mean of the embeddings takes its place.

    python examples/i8_decode.py [--vocab 151936] [--hidden 896] [--batch 4] [--steps 16]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import embedding_lookup_tied_gb300 as lhs  # noqa: E402


class Decoder:
    """One batch of sequences.  Everything a step writes is allocated here."""

    def __init__(self, table: torch.Tensor, batch: int, temperature=0.8, top_k=50, top_p=0.95, min_p=0.02):
        dev, (vocab, hidden) = table.device, table.shape
        self.embed = lhs.lhs_table_init(table, vocab, hidden, lhs.LHS_BF16)
        self.err = torch.zeros(1, dtype=torch.int32, device=dev)
        self.head, _ = lhs.lhs_i8_quantize(table, err=self.err)
        self.x = torch.zeros((batch, hidden), device=dev)
        self.rows = torch.empty((batch, hidden), device=dev)
        self.logits = torch.empty((batch, vocab), device=dev)
        self.ws = torch.empty(lhs.lhs_i8_workspace(self.head, batch), dtype=torch.uint8, device=dev)
        self.ids = torch.empty(batch, dtype=torch.int32, device=dev)
        self.probs = torch.empty(batch, device=dev)
        full = lambda v, t=torch.float32: torch.full((batch,), v, dtype=t, device=dev)  # noqa: E731
        self.filters = dict(temperature=full(temperature), top_k=full(top_k, torch.int32), top_p=full(top_p),
                            min_p=full(min_p))

    def step(self, ids: torch.Tensor, u: torch.Tensor):
        """The tokens that follow ``ids`` (int32 [batch]), drawn with ``u`` (f32
        [batch] in [0, 1)), and their probabilities."""
        lhs.lhs_embed(self.embed, ids, 1.0, out=self.rows, err=self.err)
        self.x.mul_(0.5).add_(self.rows)
        lhs.lhs_i8_logits(self.head, self.x, out=self.logits, ws=self.ws, err=self.err)
        lhs.lhs_sample(self.logits, u, ids=self.ids, probs=self.probs, err=self.err, **self.filters)
        return self.ids, self.probs


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--vocab", type=int, default=151936)
    ap.add_argument("--hidden", type=int, default=896)
    ap.add_argument("--batch", type=int, default=4)
    ap.add_argument("--steps", type=int, default=16)
    a = ap.parse_args(argv)
    g = torch.Generator(device="cuda").manual_seed(0)
    table = torch.randn((a.vocab, a.hidden), generator=g, device="cuda").to(torch.bfloat16)
    d = Decoder(table, a.batch)
    ids = torch.randint(0, a.vocab, (a.batch,), generator=g, device="cuda", dtype=torch.int32)
    out = []
    for _ in range(a.steps):
        nxt, _ = d.step(ids, torch.rand(a.batch, generator=g, device="cuda"))
        ids = nxt.clone()
        out.append(ids)
    tokens = torch.stack(out, 1).cpu()
    if int(d.err.item()):
        raise RuntimeError(f"error bits {int(d.err.item())}")
    for row in tokens.tolist():
        print(" ".join(map(str, row)))
    return tokens


if __name__ == "__main__":
    main()
