"""A draft layer with its 8-bit cache and the 2-bit head, as a speculative decoder runs them.

Random weights of a small shape (or the sizes given): every sequence's prompt goes
through the layer at once (append, attention of many rows); then `--slots` draft
tokens a sequence, one at a time (append of one token, attention of one row a
sequence, the head's argmax); then the sequences keep a part of their drafts, as
after a verification, and draft again over the rejected tokens' places.  The
projections around the attention are plain torch products.

  python examples/draft_step.py [--seqs 8] [--prompt 700] [--slots 9] [--rounds 2]
"""
import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from bit_quantized_lm_amd import (DraftCache, DraftHead, draft_layer_rope_table,  # noqa: E402
                                  draft_layer_workspace)
from bit_quantized_lm_amd import workload  # noqa: E402


class DraftLayer:
    """Norm, attention over the cache, residual, norm: what turns a token's
    embedding into the head's row."""

    def __init__(self, hidden, hq, hkv, d, vocab, positions, pages, page, dev, seed=0):
        g = torch.Generator(device=dev).manual_seed(seed)

        def weight(*shape):
            return (torch.randn(shape, generator=g, device=dev) / math.sqrt(shape[-1])).to(torch.bfloat16)

        self.hq, self.hkv, self.d = hq, hkv, d
        self.embed = torch.randn((vocab, hidden), generator=g, device=dev).to(torch.bfloat16)
        self.qkv, self.out = weight((hq + 2 * hkv) * d, hidden), weight(hidden, hq * d)
        self.rope = torch.from_numpy(draft_layer_rope_table(positions, d)).to(dev)
        self.cache = DraftCache(pages, hkv, d, page, device=dev)

    @staticmethod
    def norm(x):
        f = x.float()
        return (f * torch.rsqrt(f.square().mean(-1, keepdim=True) + 1e-6)).to(torch.bfloat16)

    def __call__(self, tokens, q_start, kv_len, table, workspace, window=0, sinks=0):
        """Hidden rows of `tokens`, the new tokens of the batch's sequences."""
        x = self.embed[tokens]
        rows = torch.nn.functional.linear(self.norm(x), self.qkv).view(len(tokens), self.hq + 2 * self.hkv, self.d)
        q, k, v = rows.split([self.hq, self.hkv, self.hkv], dim=1)
        q = self.cache.append(q, k, v, self.rope, q_start, kv_len, table)
        o, _ = self.cache.attend(q, q_start, kv_len, table, window=window, sinks=sinks, workspace=workspace)
        return self.norm(x + torch.nn.functional.linear(o.view(len(tokens), -1), self.out))


def run(seqs=8, prompt=700, slots=9, rounds=2, hidden=1024, vocab=16384, hq=10, hkv=2, d=128, page=64, window=0, sinks=0, seed=0,
        say=print):
    """Returns the draft tokens of every round, [rounds][seqs][slots]."""
    dev = torch.device("cuda")
    per_seq = -(-(prompt + rounds * slots) // page)
    layer = DraftLayer(hidden, hq, hkv, d, vocab, per_seq * page, seqs * per_seq, page, dev, seed)
    head = DraftHead.from_weight(workload.gen_weight(vocab, hidden, seed=seed + 1), device=dev)
    rng = torch.Generator().manual_seed(seed)
    lengths = [prompt - i * (prompt // (2 * seqs)) for i in range(seqs)]          # prompts of several lengths
    table = torch.randperm(seqs * per_seq, generator=rng).view(seqs, per_seq).to(torch.int32).to(dev)
    workspace = draft_layer_workspace(sum(lengths), seqs, hq, hkv, d, dev)       # for the prompts, and for every smaller batch

    def ints(x):
        return torch.tensor(x, dtype=torch.int32, device=dev)

    def head_tokens(x):
        return head(x)["out_id"].long()

    # prompts: all rows at once, the last row of each sequence goes on to the head
    starts = [0]
    for n in lengths:
        starts.append(starts[-1] + n)
    tokens = torch.randint(0, vocab, (starts[-1],), generator=rng).to(dev)
    x = layer(tokens, ints(starts), ints(lengths), table, workspace, window, sinks)
    last = head_tokens(x[ints(starts[1:]).long() - 1].contiguous())
    one = ints(list(range(seqs + 1)))
    kept, drafts = ints(lengths), []
    for r in range(rounds):
        got, token = [], last
        for i in range(slots):
            x = layer(token, one, kept + (i + 1), table, workspace, window, sinks)
            token = head_tokens(x)
            got.append(token)
        drafts.append(torch.stack(got, 1))
        # stands for the verification: sequence s keeps s % slots + 1 of its tokens; what follows them
        # in the cache is written over by the next round
        keep = torch.arange(seqs, device=dev) % slots
        last = drafts[-1].gather(1, keep[:, None])[:, 0]
        kept = kept + (keep + 1).to(torch.int32)
        say(f"round {r}: {seqs} sequences, {slots} slots each; kept {(keep + 1).tolist()}; first drafts {drafts[-1][0].tolist()}")
    return torch.stack(drafts)


def main():
    p = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, value in (("seqs", 8), ("prompt", 700), ("slots", 9), ("rounds", 2), ("window", 0), ("sinks", 0), ("seed", 0)):
        p.add_argument("--" + name, type=int, default=value)
    run(**vars(p.parse_args()))


if __name__ == "__main__":
    main()
