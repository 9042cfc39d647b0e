"""Plain float64 forms of the attention with first tokens kept, of caches in 4 bits and of their pages (CPU)."""
import math

import torch

NINF = float("-inf")
CODES = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def e4m3(byte):
    """An e4m3 number (no infinities) from its bits."""
    s, e, m = byte >> 7, (byte >> 3) & 15, byte & 7
    if e == 15 and m == 7:
        return math.nan
    v = m / 8.0 * 2.0 ** -6 if e == 0 else (1 + m / 8.0) * 2.0 ** (e - 7)
    return -v if s else v


SCALES = [e4m3(b) for b in range(127)]     # the finite ones, rising


def nearest(values, x):
    """Index of the value nearest to x in a rising list; of two equally near ones the even index."""
    i = min(range(len(values)), key=lambda j: abs(values[j] - x))
    for j in (i - 1, i + 1):
        if 0 <= j < len(values) and abs(values[j] - x) == abs(values[i] - x) and j % 2 == 0:
            return j
    return i


def quantize(x, unit=1.0):
    """A block of 16 floats: (scale byte, 16 codes)."""
    if any(math.isnan(v) for v in x):
        return 127, None
    top = max(abs(v) for v in x) / 6.0 / unit
    b = nearest(SCALES, min(max(top, 2.0 ** -9), 448.0))
    s = SCALES[b] * unit
    return b, [nearest(CODES, min(abs(v) / s, 6.0)) + (8 if math.copysign(1.0, v) < 0 else 0) for v in x]


def values(codes, scales, unit=1.0):
    """float64 values of codes [..., d / 2] (uint8) and scales [..., d / 16] (bytes)."""
    table = torch.tensor(CODES + [-c for c in CODES], dtype=torch.float64)
    numbers = torch.tensor([e4m3(b) for b in range(256)], dtype=torch.float64)
    codes, scales = codes.cpu().long(), scales.cpu().view(torch.uint8).long()
    y = torch.stack([table[codes & 15], table[codes >> 4]], -1).flatten(-2)
    return y * numbers[scales].repeat_interleave(16, -1) * unit


def attention(q, kc, vc, table, kv_lens, cu_q, causal, window, sinks, scale):
    """out, lse in float64 over float64 caches [pages, page_size, heads, dim]; per value sum p |v|; per row the largest
    sum |q k| |scale|, the largest sum |k| max|q| |scale| and the largest |v|."""
    q, table, kv_lens, cu_q = q.cpu().double(), table.cpu().tolist(), kv_lens.cpu().tolist(), cu_q.cpu().tolist()
    n, hq, d = q.shape
    P, hkv = kc.shape[1], kc.shape[2]
    out, lse = torch.zeros(n, hq, d, dtype=torch.float64), torch.full((n, hq), NINF, dtype=torch.float64)
    size, spread, reach, top = torch.zeros_like(out), torch.zeros_like(lse), torch.zeros_like(lse), torch.zeros_like(lse)
    for b in range(len(kv_lens)):
        L, new = kv_lens[b], cu_q[b + 1] - cu_q[b]
        t = torch.arange(L)
        for i in range(new):
            pos = L - new + i
            see = torch.ones(L, dtype=torch.bool)
            if causal:
                see &= t <= pos
            if window:
                see &= (t > pos - window) | (t < sinks)
            at = t[see].tolist()
            if not at:
                continue
            K = torch.stack([kc[table[b][j // P], j % P] for j in at])
            V = torch.stack([vc[table[b][j // P], j % P] for j in at])
            for h in range(hq):
                g, row, o = h // (hq // hkv), q[cu_q[b] + i, h], (cu_q[b] + i, h)
                x = K[:, g] @ row * scale
                w = torch.exp(x - x.max())
                w, total = w / w.sum(), w.sum()
                out[o], size[o] = w @ V[:, g], w @ V[:, g].abs()
                lse[o] = x.max() + math.log(float(total))
                spread[o] = (K[:, g].abs() @ row.abs()).max() * abs(scale)
                reach[o] = K[:, g].abs().sum(1).max() * row.abs().max() * abs(scale)
                top[o] = V[:, g].abs().max()
    return out, lse, size, spread, reach, top


def bounds(dtype, size, spread, reach, top, keys, dim, bits):
    """Largest errors of out and lse.  Scores: sums of `dim` exact products in fp32 (2^-24 each of their size, three more
    for the factors), 2^-21 for exponentials and sums, and over 4 bits the bf16 queries' 2^-25 of the row's largest.  An
    error e of a score is one of e in lse and 2 e in a probability.  Probabilities are rounded to the operands' type (over 4
    bits half precision, u = 2^-11; the smallest ones to a step of 2^-24 beside a largest of 1 at least), the
    output to its own, each half a unit."""
    u = torch.finfo(dtype).eps / 2
    up = 2.0 ** -11 if bits == 4 else u
    score = spread * (dim + 4) * 2.0 ** -24 + 2.0 ** -21
    if bits == 4 and dtype == torch.bfloat16:
        score = score + reach * 2.0 ** -25
    tiny = 2.0 ** -24 if dtype == torch.float16 else 0.0
    small = keys * 2.0 ** -25 * top if bits == 4 or dtype == torch.float16 else torch.zeros_like(top)
    return size * (1.01 * (u + up) + 2 * score.unsqueeze(-1)) + small.unsqueeze(-1) + tiny, score


def assign(table, lens, page_size, pages, kept, parents=None):
    """New table (lists; -1 none), copies [(src, dst)] and whether everything was found."""
    B, W = len(table), len(table[0]) if table else 0
    parents = list(range(B)) if parents is None else parents
    ok, new, writers, readers = True, [[-1] * W for _ in range(B)], {}, set()
    need, full, part = [], [], []
    for b in range(B):
        n = max(lens[b], 0)
        if n > W * page_size:
            ok, n = False, W * page_size
        k = min(max(kept[b], 0), n)
        if not 0 <= parents[b] < B:
            k = 0
        need.append(-(-n // page_size))
        full.append(k // page_size)
        part.append(k % page_size > 0)
    def have(b, j):
        return table[parents[b]][j]
    for b in range(B):
        for j in range(full[b]):
            readers.add(have(b, j))
        if part[b]:
            writers.setdefault(have(b, full[b]), []).append(b)
    held = {p for p in readers | set(writers) if 0 <= p < pages}
    free = [p for p in range(pages) if p not in held]
    copies = []
    for b in range(B):
        for j in range(need[b]):
            if j < full[b] or (j == full[b] and part[b]):
                p = have(b, j)
                if not 0 <= p < pages:
                    ok = False
                    continue
                if j < full[b] or (p not in readers and writers[p][0] == b):
                    new[b][j] = p
                    continue
            else:
                p = None
            if not free:
                ok = False
                continue
            new[b][j] = free.pop(0)
            if p is not None:
                copies.append((p, new[b][j]))
    return new, copies, ok


def compact(table, pages):
    """New table, used pages, copies."""
    held = sorted({p for row in table for p in row if 0 <= p < pages})
    u = len(held)
    src = [p for p in held if p >= u]
    dst = [p for p in range(u) if p not in set(held)]
    to = dict(zip(src, dst))
    return [[to.get(p, p) if 0 <= p < pages else -1 for p in row] for row in table], u, list(zip(src, dst))
