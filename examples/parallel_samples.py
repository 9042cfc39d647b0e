"""Several continuations of each of a few prompts, decoded together on one GPU: the pages of the cache are shared.

A model of a few random layers reads every prompt once.  `assign_pages` forks the prompts into samples: whole pages
are shared, the page in which a prompt ends is copied for all samples but one.  Every step each sample gets room
for its next token (`assign_pages` again), its token goes to the caches (`rope_append`), and it looks at a window of
them and at the first tokens (`chunk_attention` with sinks).  The caches are held in 4 bits (`FP4Cache`).  Samples that
have ended give their pages back, and `compact_pages` moves what is left together.

    python examples/parallel_samples.py              # the samples, and how many pages they took
    python examples/parallel_samples.py --bits 16    # caches in bfloat16
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import draft_verification_spec_gb300 as sv  # noqa: E402


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


class Model:
    """A decoder of `layers` layers with random weights over paged caches of its own."""

    def __init__(self, vocab, layers, q_heads, kv_heads, dim, pages, page_size, bits, window, sinks, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        width = q_heads * dim
        shapes = [(vocab, width)] + [(width, (q_heads + 2 * kv_heads) * dim), (width, width)] * layers + [(width, vocab)]
        self.weights = [(torch.randn(*s, generator=g, device="cuda") * s[0] ** -0.5).bfloat16() for s in shapes]
        self.heads, self.dim, self.layers = (q_heads, kv_heads), dim, layers
        self.window, self.sinks = window, sinks
        self.rope = sv.RopePlan(dim)

        def cache():
            if bits == 4:
                return sv.FP4Cache(pages, page_size, kv_heads, dim)
            return torch.zeros(pages, page_size, kv_heads, dim, dtype=torch.bfloat16, device="cuda")

        self.caches = [[cache(), cache()] for _ in range(layers)]

    def __call__(self, tokens, table, kv_lens, cu_q, max_q):
        """Logits [tokens, vocab] of packed new tokens; their keys and values go to the caches."""
        hq, hkv = self.heads
        x = self.weights[0][tokens.long()] * self.weights[0].shape[1] ** 0.5
        for layer, (k_cache, v_cache) in enumerate(self.caches):
            w_in, w_out = self.weights[1 + 2 * layer: 3 + 2 * layer]
            qkv = (torch.nn.functional.rms_norm(x, x.shape[-1:]) @ w_in).view(len(tokens), hq + 2 * hkv, self.dim)
            q = sv.rope_append(qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:], self.rope, k_cache, v_cache, table,
                               kv_lens, cu_q)
            y = sv.chunk_attention(q, k_cache, v_cache, table, kv_lens, cu_q, max_q, window=self.window, sinks=self.sinks)
            x = x + y.view(len(tokens), -1) @ w_out
        return torch.nn.functional.rms_norm(x, x.shape[-1:]) @ self.weights[-1] * 2.0


def decode(prompts=2, samples=3, steps=24, bits=4, window=64, sinks=4, T=0.8, top_p=0.95, seed=0, end=1):
    """Tokens of every sample, and the pages in use: after the prompts, at the end, after the last compaction."""
    vocab, page_size, most = 500, 16, 96
    B = prompts * samples
    lens = [40 + 13 * b for b in range(prompts)]
    model = Model(vocab, 2, 8, 2, 64, pages=B * -(-(most + steps) // page_size), page_size=page_size, bits=bits, window=window,
                  sinks=sinks, seed=seed)
    pool = sv.PagePool([c for layer in model.caches for c in layer])
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    width = -(-(most + steps) // page_size)
    # the prompts, in the first rows of the table
    table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
    need = i32(lens + [0] * (B - prompts))
    table = sv.assign_pages(pool, table, need, page_size, kept=torch.zeros_like(need))
    text = [torch.randint(2, vocab, (n,), generator=g, device="cuda").int() for n in lens]
    cu = i32([0] + [sum(lens[: b + 1]) for b in range(prompts)] + [sum(lens)] * (B - prompts))
    logits = model(torch.cat(text), table, need, cu, max(lens))
    shared = int((table >= 0).sum())
    # forked: sample b goes on from prompt b // samples
    parents = i32([b // samples for b in range(B)])
    kept = need[parents.long()]
    last = logits[(cu[1:prompts + 1].long() - 1)[parents.long()]]
    out, live = [[] for _ in range(B)], torch.ones(B, dtype=torch.bool, device="cuda")
    one = torch.arange(B + 1, dtype=torch.int32, device="cuda")
    for step in range(steps):
        tokens = sv.sample_tokens(last, torch.rand(B, generator=g, device="cuda"), T, 0, top_p).tokens
        for b, x in enumerate(tokens.tolist()):
            if live[b]:
                out[b].append(x)
        live &= tokens != end
        # samples that have ended keep nothing; the others get room for one more token
        kept = torch.where(live, kept, torch.zeros_like(kept))
        now = torch.where(live, kept + 1, torch.zeros_like(kept))
        table = sv.assign_pages(pool, table, now, page_size, kept=kept, parents=parents)
        parents, kept = None, now
        if step % 8 == 7:
            table, used = sv.compact_pages(pool, table)
        last = model(tokens.clamp(min=0), table, now, one, 1)
    held = len(set(table[table >= 0].tolist()))
    table, used = sv.compact_pages(pool, table)
    assert sv.default_workspace().status() == 0
    return out, (shared, held, int(used))


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--bits", type=int, choices=(4, 16), default=4)
    a = ap.parse_args()
    out, (shared, held, used) = decode(bits=a.bits)
    print(f"pages: {shared} of the prompts, {held} held at the end, {used} after the compaction")
    for t in out:
        print(t)


if __name__ == "__main__":
    main()
