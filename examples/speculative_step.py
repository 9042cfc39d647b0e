"""Speculative decoding with the operators of this package, end to end on one GPU.

A target model of a few random layers and a draft model that is the target with noise on its weights
decode a batch of prompts.  One step: the draft proposes K tokens (`rope_append`, `chunk_attention`,
`sample_tokens` per token), the target scores the K + 1 positions in one chunk over its paged cache,
both distributions are truncated by the same filters, and `verify_chain` accepts a prefix and draws the
next token.  A rejected draft needs no undoing: the next step's lengths are shorter and its tokens
overwrite the slots.

    python examples/speculative_step.py            # tokens and the mean accepted length
    python examples/speculative_step.py --check    # at T = 0 the tokens equal plain greedy decoding
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import draft_verification_spec_gb300 as sv  # noqa: E402


class Model:
    """A decoder of `layers` layers with a paged cache per layer; weights are random."""

    def __init__(self, vocab, layers, q_heads, kv_heads, dim, pages, page_size, seed, like=None, noise=0.0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        width = q_heads * dim

        def weight(i, *shape):
            w = torch.randn(*shape, generator=g, device="cuda") * shape[0] ** -0.5
            if like is not None:
                w = like.weights[i].float() + noise * w
            return w.to(torch.bfloat16)

        shapes = [(vocab, width)] + [(width, (q_heads + 2 * kv_heads) * dim), (width, width)] * layers + [(width, vocab)]
        self.weights = [weight(i, *s) for i, s in enumerate(shapes)]
        self.heads, self.dim, self.layers = (q_heads, kv_heads), dim, layers
        self.rope = sv.RopePlan(dim, theta=10000.0)
        self.caches = [[torch.zeros(pages, page_size, kv_heads, dim, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
                       for _ in range(layers)]

    def __call__(self, tokens, table, kv_lens, cu_q, max_q):
        """Logits [tokens, vocab] of packed new tokens; their keys and values go to the caches."""
        hq, hkv = self.heads
        x = self.weights[0][tokens.long()] * self.weights[0].shape[1] ** 0.5
        for layer in range(self.layers):
            w_in, w_out = self.weights[1 + 2 * layer: 3 + 2 * layer]
            y = torch.nn.functional.rms_norm(x, x.shape[-1:])
            qkv = (y @ w_in).view(len(tokens), hq + 2 * hkv, self.dim)
            k_cache, v_cache = self.caches[layer]
            q = sv.rope_append(qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:], self.rope, k_cache, v_cache, table,
                               kv_lens, cu_q)
            x = x + sv.chunk_attention(q, k_cache, v_cache, table, kv_lens, cu_q, max_q).view(len(tokens), -1) @ w_out
        return torch.nn.functional.rms_norm(x, x.shape[-1:]) @ self.weights[-1] * 2.0


class Decoder:
    """State of a batch: per request the tokens so far; all but the last are in both caches."""

    def __init__(self, target, draft, prompts, page_size, max_len, T, top_p, seed):
        self.target, self.draft, self.T, self.top_p = target, draft, T, top_p
        self.tokens = [list(p) for p in prompts]
        B = len(prompts)
        width = -(-max_len // page_size)
        self.table = torch.arange(B * width, dtype=torch.int32, device="cuda").view(B, width)
        self.g = torch.Generator(device="cuda").manual_seed(seed)
        for model in (target, draft):
            self._feed(model, [p[:-1] for p in self.tokens], [len(p) - 1 for p in self.tokens])

    def _feed(self, model, new, lens):
        cu = [0]
        for t in new:
            cu.append(cu[-1] + len(t))
        flat = torch.tensor([x for t in new for x in t], dtype=torch.int32, device="cuda")
        i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
        return model(flat, self.table, i32(lens), i32(cu), max(len(t) for t in new))

    def _uniforms(self, *shape):
        return torch.rand(*shape, generator=self.g, device="cuda")

    def greedy(self):
        """One token per request by the target alone."""
        logits = self._feed(self.target, [t[-1:] for t in self.tokens], [len(t) for t in self.tokens])
        out = sv.sample_tokens(logits, self._uniforms(len(self.tokens)), 0.0)
        for t, x in zip(self.tokens, out.tokens.tolist()):
            t.append(x)

    def step(self, K):
        """K drafts, one verification; returns the accepted drafts per request."""
        B = len(self.tokens)
        lens = [len(t) for t in self.tokens]
        # the draft's cache may lack the last two tokens (all drafts accepted and one more drawn)
        fresh = [t[-2:] for t in self.tokens]
        proposals, rows = [], []
        for k in range(K):
            logits = self._feed(self.draft, fresh, [n + k for n in lens])
            last = torch.tensor([sum(len(f) for f in fresh[:b + 1]) - 1 for b in range(B)], device="cuda")
            s = sv.sample_tokens(logits[last], self._uniforms(B), self.T, 0, self.top_p, want_filtered=True)
            proposals.append(s.tokens)
            rows.append(s.filtered)
            fresh = [[x] for x in s.tokens.tolist()]
        drafts = torch.stack(proposals, 1)
        new = [t[-1:] + d for t, d in zip(self.tokens, drafts.tolist())]
        logits = self._feed(self.target, new, [n + K for n in lens])
        p = sv.sample_tokens(logits, self._uniforms(B * (K + 1)), self.T, 0, self.top_p, want_filtered=True).filtered
        if self.T == 0.0:     # argmax matching reads the logits as they are
            p, rows = logits, [logits.view(B, K + 1, -1)[:, k] for k in range(K)]
        out = sv.verify_chain(p.view(B, K + 1, -1), torch.stack(rows, 1), drafts, self._uniforms(B, K + 1), self.T)
        accepted = out.accepted.tolist()
        for t, n, row in zip(self.tokens, accepted, out.tokens.tolist()):
            t.extend(row[: n + 1])
        return accepted


def decode(steps=12, K=3, B=4, T=0.8, top_p=0.95, speculative=True, seed=0, noise=0.15):
    vocab, page_size, max_len = 2000, 16, 24 + steps * (K + 1) + K + 2
    shape = dict(vocab=vocab, layers=2, q_heads=8, kv_heads=2, dim=64, pages=B * -(-max_len // page_size), page_size=page_size)
    target = Model(seed=seed, **shape)
    draft = Model(seed=seed + 1, like=target, noise=noise, **shape)
    g = torch.Generator().manual_seed(seed)
    prompts = [torch.randint(vocab, (12 + 3 * b,), generator=g).tolist() for b in range(B)]
    d = Decoder(target, draft, prompts, page_size, max_len, T, top_p, seed)
    accepted = []
    for _ in range(steps):
        if speculative:
            accepted += d.step(K)
        else:
            d.greedy()
    assert sv.default_workspace().status() == 0
    return [t[len(p):] for t, p in zip(d.tokens, prompts)], accepted


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--check", action="store_true")
    a = ap.parse_args()
    if a.check:
        got, accepted = decode(T=0.0, top_p=1.0, noise=0.02)
        want, _ = decode(steps=max(len(t) for t in got), speculative=False)
        print("greedy tokens equal:", all(x == y[: len(x)] for x, y in zip(got, want)), "mean accepted", sum(accepted) / len(accepted))
        return
    tokens, accepted = decode()
    print("mean accepted drafts per step: %.2f of 3" % (sum(accepted) / len(accepted)))
    for t in tokens:
        print(t)


if __name__ == "__main__":
    main()
