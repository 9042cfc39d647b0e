"""Plain float64 forms of the step operators (CPU, loops over requests and rows), and error bounds."""
import math

import numpy as np
import torch

NINF = float("-inf")


def positions(cu_q, kv_lens, b):
    n = cu_q[b + 1] - cu_q[b]
    return [kv_lens[b] - n + i for i in range(n)]


def attention(q, k_cache, v_cache, table, kv_lens, cu_q, causal, window, scale):
    """out, lse in float64; and per value sum p |v|, per row max sum |q k| scale, for the bounds."""
    q, kc, vc = (t.cpu().double() for t in (q, k_cache, v_cache))
    table, kv_lens, cu_q = table.cpu().tolist(), kv_lens.cpu().tolist(), cu_q.cpu().tolist()
    n, hq, d = q.shape
    P, hkv = kc.shape[1], kc.shape[2]
    out, lse = torch.zeros(n, hq, d, dtype=torch.float64), torch.full((n, hq), NINF, dtype=torch.float64)
    size, spread = torch.zeros_like(out), torch.zeros_like(lse)
    for b in range(len(kv_lens)):
        L = kv_lens[b]
        if L == 0:
            continue
        K = torch.stack([kc[table[b][t // P], t % P] for t in range(L)])
        V = torch.stack([vc[table[b][t // P], t % P] for t in range(L)])
        t = torch.arange(L)
        for i, pos in enumerate(positions(cu_q, kv_lens, b)):
            see = torch.ones(L, dtype=torch.bool)
            if causal:
                see &= t <= pos
            if window:
                see &= t > pos - window
            if not see.any():
                continue
            for h in range(hq):
                g, row = h // (hq // hkv), q[cu_q[b] + i, h]
                x = K[see, g] @ row * scale
                w = torch.exp(x - x.max())
                at = (cu_q[b] + i, h)
                out[at] = (w / w.sum()) @ V[see, g]
                size[at] = (w / w.sum()) @ V[see, g].abs()
                lse[at] = x.max() + math.log(float(w.sum()))
                spread[at] = float((K[see, g].abs() @ row.abs() * abs(scale)).max())
    return out, lse, size, spread


def attention_bounds(dtype, size, spread, dim):
    """Largest errors of out and lse.  out: the probabilities' rounding and the output's, each at most the
    unit roundoff u of the type (half its eps) times sum p |v|, plus the fp32 part.  The fp32 part: scores are sums of `dim` exact products
    (2^-24 each of their size; log2 e and the scale round three times more), and an error e of a score is an
    error e of lse and 2 e of a probability; 2^-21 for the exponentials and the sums."""
    u = torch.finfo(dtype).eps / 2
    score = spread * (dim + 4) * 2.0 ** -24 + 2.0 ** -21
    tiny = 2.0 ** -24 if dtype == torch.float16 else 0.0   # half precision's smallest step
    return size * (2.02 * u + 2 * score.unsqueeze(-1)) + tiny, score


def rope(x, pos, freqs, factor, rotary, layout):
    """Rotated x [heads, dim] (float64) of one token."""
    y = x.clone()
    for j, f in enumerate(freqs):
        a, b = (2 * j, 2 * j + 1) if layout == "interleaved" else (j, j + rotary // 2)
        c, s = math.cos(pos * f) * factor, math.sin(pos * f) * factor
        y[:, a], y[:, b] = x[:, a] * c - x[:, b] * s, x[:, b] * c + x[:, a] * s
    return y


def sample(row, u, T, top_k, top_p, min_p):
    """(token, prob, kept, indices kept) of one row, float64."""
    z = np.where(np.isnan(row), -np.inf, row).astype(np.float64)
    order = np.argsort(-z, kind="stable")
    order = order[z[order] > -np.inf]
    if len(order) == 0:
        return -1, 0.0, 0, order
    f = lambda v: float(np.float32(v))  # noqa: E731
    T, top_p, min_p = f(T), f(top_p), f(min_p)
    if not T > 0:
        T, top_k = 1.0, 1
    with np.errstate(invalid="ignore"):
        d = z[order] - z[order[0]]
    w = np.exp(np.where(np.isnan(d), 0.0, d) / T)
    n = min(len(w), top_k) if top_k > 0 else len(w)
    before = np.cumsum(w) - w
    n_p = max(1, int((before[:n] < top_p * w[:n].sum()).sum())) if top_p < 1 else n
    n_m = max(1, int((w >= min_p).sum())) if min_p > 0 else n
    n = min(n, n_p, n_m)
    total = w[:n].sum()
    at = min(int((np.cumsum(w[:n]) <= f(u) * total).sum()), n - 1)
    while w[at] == 0:
        at -= 1
    return int(order[at]), w[at] / total, n, order[:n]
