"""More operators of a speculative decoding step: their cases, inputs and plain forms.

Four operators: ``chunk_attention`` with a window and a few first tokens that stay visible, ``chunk_attention`` over a
cache held in 4 bits, ``rope_append`` into such a cache, and the pages of a cache: ``assign_pages`` (fork, grow, shrink,
free, with copies of the pages that two requests would write to) and ``compact_pages``.

Four bits: values in blocks of 16 along a head; a value is unit * scale * code, the code one of 0, 0.5, 1, 1.5, 2, 3, 4, 6
with a sign (two to a byte, the even one low), the scale an e4m3 number, the unit a power of two of the whole cache.
"""
import math
import random

import torch

own = False

ATTENTION = dict(op="attention", bits=16, dtype="bf16", B=1, nq=1, kv=1024, ragged=False, hq=32, hkv=8, d=128, page=16,
                 causal=True, window=0, sinks=0)
APPEND = dict(op="append", dtype="bf16", B=1, nq=1, past=1000, hq=32, hkv=8, d=128, rotary=128, layout="half",
              theta=10000.0, page=16)
PAGES = dict(op="assign", kind="step", B=64, kv=16384, page=16, caches=2, hkv=8, d=128, dtype="bf16", group=1, load=0.8)


def listed():
    return [
        # one user far into a conversation, a window and 4 first tokens: the latency of a plain decoding step
        dict(ATTENTION, name="sinks decode 1", kv=20000, window=1024, sinks=4),
        # a serving batch of single tokens over long caches, of which a window and 16 first tokens are looked at
        dict(ATTENTION, name="sinks decode 64", B=64, kv=32768, ragged=True, window=4096, sinks=16, page=32),
        # chunked prefill: 2048 tokens of two prompts behind 14336 that are cached, within a window
        dict(ATTENTION, name="sinks prompt chunk", B=2, nq=2048, kv=16384, page=128, window=4096, sinks=64),
        # one user, one token over a conversation held in 4 bits
        dict(ATTENTION, name="4-bit decode 1", bits=4, kv=4096),
        # a serving batch of single tokens over caches of ragged length, one slot of the batch idle
        dict(ATTENTION, name="4-bit decode 64", bits=4, B=64, kv=16384, ragged=True),
        # verification of a block of 16 drafts over long contexts, 8 query heads a key head, fp16
        dict(ATTENTION, name="4-bit verify block", bits=4, dtype="f16", B=32, nq=17, kv=16384, ragged=True, hq=64, page=64),
        # chunked prefill over a cache in 4 bits, pages of 24
        dict(ATTENTION, name="4-bit prompt chunk", bits=4, B=1, nq=2048, kv=16384, page=24),
        # one token of one request
        dict(APPEND, name="4-bit append 1"),
        # chunks of four prompts far into long contexts
        dict(APPEND, name="4-bit append chunk", B=4, nq=2048, past=120000, theta=500000.0, page=64),
        # between two steps: every request drops its rejected drafts and gets room for the next ones
        dict(PAGES, name="pages step"),
        # 8 prompts forked into 8 samples each: the pages that hold the prompts' last tokens are copied in 32 caches
        dict(PAGES, name="pages fork", kind="fork", kv=8000, group=8, caches=32),
        # a pool that is 60 % full is moved together, in 8 caches
        dict(PAGES, name="pages compact", op="compact", kv=4096, page=32, caches=8, load=0.6),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["sinks", "sinks", "4-bit", "4-bit", "4-bit", "append", "pages", "pages"])
    if op in ("sinks", "4-bit"):
        c = dict(ATTENTION, bits=16 if op == "sinks" else 4, dtype=rng.choice(["bf16", "bf16", "f16"]), B=_log(rng, 1, 64),
                 ragged=rng.random() < 0.7, hkv=rng.choice([1, 2, 4, 8]), d=rng.choice([64, 80, 128, 128, 256]),
                 page=rng.choice([1, 8, 16, 24, 32, 64, 128, 256]), causal=rng.random() < 0.75)
        if op == "sinks" or rng.random() < 0.3:
            c["window"], c["sinks"] = _log(rng, 16, 4096), _log(rng, 1, 256)
        c["hq"] = c["hkv"] * rng.choice([1, 2, 4, 7, 8, 16])
        kind = rng.choice(["token", "verify", "prompt"])
        c["nq"] = 1 if kind == "token" else _log(rng, 2, 32) if kind == "verify" else _log(rng, 33, 2048)
        c["kv"] = _log(rng, 1, 32768)
        while c["B"] * c["kv"] * c["hkv"] * c["d"] > 2 ** 29 or c["B"] * c["hq"] * c["nq"] * c["kv"] * max(128, c["d"]) > 2 ** 37:
            c["B"], c["kv"] = max(1, c["B"] * 2 // 3), max(1, int(c["kv"] * 0.8))
        return c
    if op == "append":
        c = dict(APPEND, dtype=rng.choice(["bf16", "f16"]), B=_log(rng, 1, 64), hkv=rng.choice([1, 2, 4, 8]),
                 d=rng.choice([64, 80, 128, 128, 256]), layout=rng.choice(["half", "interleaved"]), past=_log(rng, 1, 200000),
                 theta=rng.choice([10000.0, 500000.0]), page=rng.choice([1, 8, 16, 24, 64, 128]))
        c["hq"] = c["hkv"] * rng.choice([1, 2, 4, 7, 8])
        c["rotary"] = rng.choice([c["d"], c["d"], c["d"] // 2])
        c["nq"] = _log(rng, 1, max(1, min(2048, 2 ** 25 // (c["B"] * (c["hq"] + 2 * c["hkv"]) * c["d"]))))
        return c
    c = dict(PAGES, op=rng.choice(["assign", "assign", "compact"]), kind=rng.choice(["step", "fork"]), B=_log(rng, 1, 256),
             kv=_log(rng, 1, 16384), page=rng.choice([1, 8, 16, 24, 32, 64, 128, 256]), caches=_log(rng, 1, 32),
             hkv=rng.choice([1, 2, 4, 8]), d=rng.choice([64, 80, 128, 256]), dtype=rng.choice(["bf16", "f16", "f32"]),
             group=rng.choice([2, 3, 4, 8, 16]), load=rng.uniform(0.3, 0.98))
    while c["B"] * (c["kv"] + c["page"]) * c["hkv"] * c["d"] * c["caches"] * _size(c) > 2 ** 32 * c["load"]:
        c["caches"], c["kv"], c["B"] = max(1, c["caches"] // 2), max(1, c["kv"] * 2 // 3), max(1, c["B"] * 5 // 6)
    return c


DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def _size(case):
    return {"bf16": 2, "f16": 2, "f32": 4}[case["dtype"]]


def _rng(case):
    """A case's lengths and places are its own, whatever the seed."""
    return random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))


# --------------------------------------------------------------------------------------------- sizes

def _lengths(case):
    """Cache lengths of every request, the new tokens included."""
    rng, B, nq = _rng(case), case["B"], case["nq"]
    kv = [rng.randint(max(1, case["kv"] // 8), case["kv"]) if case["ragged"] and b else case["kv"] for b in range(B)]
    kv = [max(nq, k) for k in kv]
    if case["ragged"] and B >= 8:
        kv[-1] = 0  # an idle slot of the batch: its rows see no key
    return kv


def _seen(case):
    """(query, key) pairs of one head that the mask leaves, and keys that some query of their request sees."""
    pairs = keys = 0
    n, W, S = case["nq"], case["window"], case["sinks"]
    for k in _lengths(case):
        for i in range(n):
            pos = k - n + i
            hi = max(0, min(k, pos + 1) if case["causal"] else k)
            lo = min(hi, max(0, pos - W + 1)) if W else 0
            pairs += hi - lo + min(S if W else 0, lo)
        lo = min(k, max(0, k - n - W + 1)) if W else 0
        keys += k - lo + min(S if W else 0, lo)
    return pairs, keys


def _plan(case):
    """A pool's pages: how many, the lengths before, what every request keeps, from whom, and its length afterwards."""
    rng, B, P = _rng(case), case["B"], case["page"]
    before = [rng.randint(max(1, case["kv"] // 4), case["kv"]) for _ in range(B)]
    if case["op"] == "assign" and case["kind"] == "fork":
        parents = [b - b % case["group"] for b in range(B)]
        before = [n if b == parents[b] else 0 for b, n in enumerate(before)]
        kept = [before[p] for p in parents]
    else:
        parents = list(range(B))
        kept = [max(0, n - rng.randint(0, 8)) for n in before]
    lens = [n + rng.randint(1, 9) for n in kept]
    need = [-(-n // P) for n in before]
    after = [-(-n // P) for n in lens]
    more = sum(n - k // P for n, k in zip(after, kept)) if case["op"] == "assign" else 0
    pages = max(sum(need) + more, int(sum(need) / case["load"])) + 1
    ids = rng.sample(range(pages), sum(need))
    return dict(pages=pages, ids=ids, before=before, need=need, parents=parents, kept=kept, lens=lens,
                width=max(need + after) + 1)


def work(case):
    e = _size(case)
    if case["op"] == "attention":
        pairs, keys = _seen(case)
        n, pages = case["B"] * case["nq"], -(-keys // case["page"])
        row = 2 * e * case["d"] if case["bits"] == 16 else 2 * (case["d"] // 2 + case["d"] // 16)
        rows = 2 * n * case["hq"] * case["d"] * e + 4 * n * case["hq"]
        return {"bytes": rows + keys * case["hkv"] * row + 4 * pages + 8 * case["B"], "flops": 4 * case["d"] * case["hq"] * pairs}
    if case["op"] == "append":
        n = case["B"] * case["nq"]
        stored = n * 2 * case["hkv"] * (case["d"] // 2 + case["d"] // 16)
        moved = n * (2 * case["hq"] + 2 * case["hkv"]) * case["d"] * e + stored
        first = [case["past"] + b for b in range(case["B"])]
        pages = sum(-(-(f + case["nq"]) // case["page"]) - f // case["page"] for f in first) + 3
        held = pages * case["page"] * 2 * case["hkv"]   # rows of the cache, whose values are read back
        return {"bytes": moved + held * (case["d"] // 2 + case["d"] // 16 + 2 * case["d"]),
                "flops": 3 * n * (case["hq"] + case["hkv"]) * case["rotary"] + held * case["d"]}
    p = _plan(case)
    page = case["page"] * case["hkv"] * case["d"] * e * case["caches"]
    if case["op"] == "compact":
        copies = sum(i >= len(p["ids"]) for i in p["ids"])
    else:
        sharers = {}
        for b, (q, k) in enumerate(zip(p["parents"], p["kept"])):
            if k % case["page"]:
                sharers.setdefault((q, k // case["page"]), []).append(b)
        copies = sum(len(s) - 1 for s in sharers.values())
    return {"bytes": 8 * case["B"] * p["width"] + 2 * copies * page, "flops": 0}


# -------------------------------------------------------------------------------------------- inputs

CODES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _quantize(x):
    """x [..., d] in 4 bits: bytes of two codes [..., d / 2] and e4m3 scales [..., d / 16], for a unit of 1."""
    blocks = x.float().unflatten(-1, (-1, 16))
    scale = (blocks.abs().amax(-1) / 6.0).clamp(2.0 ** -9, 448.0).to(torch.float8_e4m3fn)
    y = blocks / scale.float()[..., None]
    a = y.abs()
    code = torch.zeros(a.shape, dtype=torch.uint8, device=x.device)
    for i, tie_up in enumerate((False, True, False, True, False, True, False)):  # to the nearest, ties to the even code
        border = (CODES[i] + CODES[i + 1]) / 2.0
        code += (a >= border) if tie_up else (a > border)
    code = (code + 8 * (y < 0).to(torch.uint8)).flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), scale


def _values(codes, scales):
    """What the 4 bits stand for, in 32 bits (exact)."""
    table = torch.tensor(CODES + tuple(-c for c in CODES), device=codes.device)
    y = torch.stack([table[(codes & 15).int()], table[(codes >> 4).int()]], -1).flatten(-2)
    return (y.unflatten(-1, (-1, 16)) * scales.float()[..., None]).flatten(-2)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dev, dt = "cuda", DTYPES[case["dtype"]]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=dev)

    def i32(v):
        return torch.tensor(v, dtype=torch.int32, device=dev)

    s = {"case": case}
    if case["op"] in ("assign", "compact"):
        return _prepare_pages(case, s, g, i32)
    B, n, hq, hkv, d, P = (case[k] for k in ("B", "nq", "hq", "hkv", "d", "page"))
    kv = _lengths(case) if case["op"] == "attention" else [case["past"] + b + n for b in range(B)]
    first = [0] * B if case["op"] == "attention" else [(k - n) // P for k in kv]  # the first page that holds something
    used = [-(-k // P) - f for k, f in zip(kv, first)]
    pages = sum(used) + 3
    width = max(1, max(u + f for u, f in zip(used, first)))
    order = torch.randperm(pages, generator=g, device=dev).to(torch.int32)
    # page j of request b: the pool's pages in a random order; -1 where a request has none
    cols = torch.arange(width, device=dev)
    at = torch.tensor([sum(used[:b]) - first[b] for b in range(B)], device=dev)[:, None] + cols
    has = (cols >= i32(first)[:, None]) & (cols < i32([u + f for u, f in zip(used, first)])[:, None])
    s["table"] = torch.where(has, order[at.clamp(0, pages - 1)], torch.full_like(order[:1], -1)).contiguous()
    s["cu_q"] = torch.arange(B + 1, dtype=torch.int32, device=dev) * n
    s["kv_lens"] = i32(kv)
    s["max_q"], s["max_kv"] = n, max(kv)
    if case["op"] == "append":
        s["q"], s["k"], s["v"] = (normal(B * n, h, d).to(dt) for h in (hq, hkv, hkv))
        s["k"][..., :: max(1, d // 8)] *= 6.0  # some channels of keys are much larger than others
    else:
        s["q"] = normal(B * n, hq, d).mul_(1.5).to(dt)  # scores of a spread that makes some keys stand out
        if case["bits"] == 16:
            s["k_cache"], s["v_cache"] = (normal(pages, P, hkv, d).to(dt) for _ in range(2))
            return s
    # in 4 bits: pages of [heads, tokens, dim] in memory, as [pages, tokens, heads, dim]
    for x in "kv":
        codes = torch.empty(pages, hkv, P, d // 2, dtype=torch.uint8, device=dev)
        scales = torch.empty(pages, hkv, P, d // 16, dtype=torch.float8_e4m3fn, device=dev)
        step = max(1, 2 ** 26 // (hkv * P * d))
        for i in range(0, pages, step):
            codes[i:i + step], scales[i:i + step] = _quantize(normal(min(step, pages - i), hkv, P, d))
        s[x + "_codes"], s[x + "_scales"] = codes.transpose(1, 2), scales.transpose(1, 2)
    if own:
        import draft_verification_spec_gb300 as sv

        for x in "kv":
            s[x + "_cache"] = sv.FP4Cache.of(s[x + "_codes"], s[x + "_scales"])
    if case["op"] == "append":
        if own:
            s["rope"] = sv.RopePlan(d, rotary_dim=case["rotary"], theta=case["theta"], layout=case["layout"])
        else:
            s["freq"] = _frequencies(case)
    return s


def _prepare_pages(case, s, g, i32):
    p, dev = _plan(case), "cuda"
    ids = torch.tensor(p["ids"], dtype=torch.int32, device=dev)
    ids = ids[torch.randperm(len(ids), generator=g, device=dev)]
    cols, need = torch.arange(p["width"], device=dev), i32(p["need"])[:, None]
    at = torch.tensor([sum(p["need"][:b]) for b in range(case["B"])], device=dev)[:, None] + cols
    s["table"] = torch.where(cols < need, ids[at.clamp(max=len(ids) - 1)], torch.full_like(ids[:1], -1)).contiguous()
    s["pages"], s["page"] = p["pages"], case["page"]
    s["parents"], s["kept"], s["lens"] = (i32(p[k]) for k in ("parents", "kept", "lens"))
    shape = (p["pages"], case["page"], case["hkv"], case["d"])
    s["caches"] = [torch.randn(shape, generator=g, device=dev, dtype=DTYPES[case["dtype"]]) for _ in range(case["caches"])]
    if own:
        import draft_verification_spec_gb300 as sv

        s["pool"] = sv.PagePool(s["caches"])
    return s


# ----------------------------------------------------------------------------------------------- run

def run(s):
    case = s["case"]
    if not own:
        return {"attention": _plain_attention, "append": _plain_append, "assign": _plain_assign, "compact": _plain_compact}[case["op"]](s)
    import draft_verification_spec_gb300 as sv

    if case["op"] == "attention":
        return sv.chunk_attention(s["q"], s["k_cache"], s["v_cache"], s["table"], s["kv_lens"], s["cu_q"], s["max_q"],
                                  causal=case["causal"], window=case["window"], sinks=case["sinks"], want_lse=True)
    if case["op"] == "append":
        q = sv.rope_append(s["q"], s["k"], s["v"], s["rope"], s["k_cache"], s["v_cache"], s["table"], s["kv_lens"], s["cu_q"])
        return q, s["k_cache"].values(), s["v_cache"].values()
    if case["op"] == "assign":
        return sv.assign_pages(s["pool"], s["table"], s["lens"], s["page"], kept=s["kept"], parents=s["parents"]), s["caches"]
    table, used = sv.compact_pages(s["pool"], s["table"])
    return table, used, s["caches"]


def _plain_attention(s):
    case = s["case"]
    q, table, dt = s["q"], s["table"], s["q"].dtype
    kv, B, P, hkv, n = s["kv_lens"].long(), case["B"], case["page"], case["hkv"], case["nq"]
    _, hq, d = q.shape
    i, t = torch.arange(n, device=q.device), torch.arange(s["max_kv"], device=q.device)
    page, slot = table[:, t // P].clamp(min=0).long(), t % P
    if case["bits"] == 16:
        keys, values = (c[page, slot].float().transpose(1, 2) for c in (s["k_cache"], s["v_cache"]))  # [B, hkv, kv, d]
    else:
        keys, values = (_values(s[x + "_codes"][page, slot], s[x + "_scales"].view(torch.uint8)[page, slot].view(torch.float8_e4m3fn))
                        .transpose(1, 2) for x in "kv")
    queries = q.float().view(B, n, hkv, hq // hkv, d).permute(0, 2, 3, 1, 4).reshape(B, hkv, -1, d)
    scores = (queries @ keys.transpose(2, 3) * (1.0 / math.sqrt(d))).view(B, hq, n, len(t))
    pos = (kv - n)[:, None] + i  # the place of each query in its request
    seen = (t < kv[:, None, None]).expand(-1, n, -1)
    if case["causal"]:
        seen = seen & (t <= pos[:, :, None])
    if case["window"]:
        seen = seen & ((t > pos[:, :, None] - case["window"]) | (t < case["sinks"]))
    scores = scores.masked_fill_(~seen[:, None], float("-inf"))
    top = scores.amax(3, keepdim=True)
    top = torch.where(top == float("-inf"), torch.zeros_like(top), top)
    w = scores.sub_(top).exp_()
    total = w.sum(3, keepdim=True)
    out = (w.view(B, hkv, -1, len(t)) @ values).view(B, hq, n, d)
    out = torch.where(total > 0, out / total, torch.zeros_like(out))
    lse = (top + total.log()).squeeze(3)
    return out.transpose(1, 2).reshape(q.shape).to(dt), lse.transpose(1, 2).reshape(q.shape[:2])


def _frequencies(case):
    """Radians a position of every pair, in 64 bits."""
    r = case["rotary"]
    return case["theta"] ** (-2.0 * torch.arange(r // 2, dtype=torch.float64, device="cuda") / r)


def _plain_append(s):
    """Angles and rotated values are in 64 bits: a code is a whole number, and must not hang on a rounding."""
    case = s["case"]
    cu, kv = s["cu_q"].long(), s["kv_lens"].long()
    n, r, P = s["q"].shape[0], case["rotary"], case["page"]
    b = torch.arange(n, device=cu.device) // case["nq"]
    pos = torch.arange(n, device=cu.device) - cu[b + 1] + kv[b]
    angle = pos.double()[:, None] * s["freq"]
    cos, sin = torch.cos(angle)[:, None], torch.sin(angle)[:, None]

    def turn(x):
        y = x.double()
        a, c = (y[..., : r // 2], y[..., r // 2: r]) if case["layout"] == "half" else (y[..., 0:r:2], y[..., 1:r:2])
        a, c = a * cos - c * sin, c * cos + a * sin
        y = torch.cat([a, c] if case["layout"] == "half" else [torch.stack([a, c], -1).flatten(-2)], -1)
        return torch.cat([y, x[..., r:].double()], -1).to(x.dtype)

    page, slot = s["table"][b, pos // P].long(), pos % P
    out = [turn(s["q"])]
    for x, new in (("k", turn(s["k"])), ("v", s["v"])):
        codes, scales = _quantize(new)
        s[x + "_codes"][page, slot] = codes
        s[x + "_scales"].view(torch.uint8)[page, slot] = scales.view(torch.uint8)
        out.append(_values(s[x + "_codes"], s[x + "_scales"]).bfloat16())
    return tuple(out)


def _plain_assign(s):
    table, P, pages = s["table"], s["page"], s["pages"]
    B, W = table.shape
    row, col = torch.arange(B, device=table.device)[:, None], torch.arange(W, device=table.device)
    need = -(-s["lens"] // P)[:, None]
    kept = torch.minimum(s["kept"], s["lens"])[:, None]
    have = table[s["parents"].long()].long()
    full, partial = col < kept // P, (col == kept // P) & (kept % P > 0)
    # who keeps a page: requests that only read it, else the first of those that will write behind its last token
    owner = torch.full((pages + 1,), B, device=table.device)
    owner.scatter_reduce_(0, torch.where(full, have, pages).flatten(), torch.full_like(have, -1).flatten(), "amin")
    owner[pages] = B
    owner.scatter_reduce_(0, torch.where(partial, have, pages).flatten(), row.expand(B, W).flatten(), "amin")
    stays = full | (partial & (owner[have.clamp(min=0)] == row))
    fresh = (col < need) & ~stays
    free = torch.nonzero(owner[:pages] == B).flatten()
    new = torch.where(stays, have, torch.where(fresh, free[(fresh.flatten().cumsum(0) - 1).clamp(min=0).view(B, W)], -1))
    copied = partial & fresh
    src, dst = have[copied], new[copied]
    for c in s["caches"]:
        c[dst] = c[src]
    return new.to(torch.int32), s["caches"]


def _plain_compact(s):
    table, pages = s["table"], s["pages"]
    held = torch.zeros(pages + 1, dtype=torch.bool, device=table.device)
    held[torch.where(table >= 0, table, pages).long()] = True
    held = held[:pages]
    used = held.sum()
    at = torch.arange(pages, device=table.device)
    src, dst = torch.nonzero(held & (at >= used)).flatten(), torch.nonzero(~held & (at < used)).flatten()
    at[src] = dst
    for c in s["caches"]:
        c[dst] = c[src]
    return torch.where(table >= 0, at[table.clamp(min=0).long()], -1).to(torch.int32), used.to(torch.int32).view(1), s["caches"]


# --------------------------------------------------------------------------------------------- exact

def exact(case, seed):
    if case["op"] in ("assign", "compact"):
        return None  # whole numbers and copies
    s = prepare(case, seed)
    return (_exact_attention if case["op"] == "attention" else _exact_append)(s)


def _exact_values(codes, scales):
    """The 4-bit values of [..., d / 2] bytes in 64 bits, from the bits of both numbers."""
    c = torch.stack([codes % 16, codes // 16], -1).flatten(-2).long()
    e, m = (c // 2) % 4, (c % 2).double()
    mag = torch.where(e == 0, m * 0.5, (1.0 + m * 0.5) * torch.pow(2.0, (e - 1).double()))
    b = scales.view(torch.uint8).long()
    se, sm = (b // 8) % 16, (b % 8).double() / 8.0
    scale = torch.where(se == 0, sm * 2.0 ** -6, (1.0 + sm) * torch.pow(2.0, (se - 7).double()))
    return torch.where(c >= 8, -mag, mag) * scale.repeat_interleave(16, -1)


def _exact_attention(s):
    case = s["case"]
    kv, table, n = s["kv_lens"].tolist(), s["table"], case["nq"]
    g, P, d, W, S = case["hq"] // case["hkv"], case["page"], case["d"], case["window"], case["sinks"]
    outs, lses = [], []
    for b in range(case["B"]):
        q = s["q"][b * n:(b + 1) * n].double()
        length = kv[b]
        out, lse = torch.zeros_like(q), torch.full(q.shape[:2], float("-inf"), dtype=torch.float64, device=q.device)
        if length:
            pages = table[b, : -(-length // P)].long()
            if case["bits"] == 16:
                K, V = (c[pages].flatten(0, 1)[:length].double() for c in (s["k_cache"], s["v_cache"]))
            else:
                K, V = (_exact_values(s[x + "_codes"][pages].flatten(0, 1)[:length],
                                      s[x + "_scales"].view(torch.uint8)[pages].flatten(0, 1)[:length]) for x in "kv")
            t = torch.arange(length, device=q.device)[None]
            back = (length - n + torch.arange(n, device=q.device)[:, None]) - t  # how far behind the query
            mask = torch.zeros(n, length, dtype=torch.float64, device=q.device)
            if W:
                mask.masked_fill_((back >= W) & (t >= S), float("-inf"))
            if case["causal"]:
                mask.masked_fill_(back < 0, float("-inf"))
            some = (mask == 0).any(1)
            for h in range(case["hq"]):
                x = q[:, h] @ K[:, h // g].T / math.sqrt(d) + mask
                lse[:, h] = torch.logsumexp(x, 1)
                out[:, h] = torch.where(some[:, None], torch.exp(x - lse[:, h, None]) @ V[:, h // g], out[:, h])
        outs.append(out)
        lses.append(lse)
    return torch.cat(outs), torch.cat(lses)


def _exact_append(s):
    case = s["case"]
    freq, n, r, P = _frequencies(case), case["nq"], case["rotary"], case["page"]
    first, second = (list(range(r // 2)), list(range(r // 2, r))) if case["layout"] == "half" else (list(range(0, r, 2)), list(range(1, r, 2)))
    q, k, v = (s[x].double() for x in "qkv")
    pos = torch.cat([torch.arange(m - n, m, device=q.device) for m in s["kv_lens"].tolist()])
    z = torch.polar(torch.ones_like(freq).expand(len(pos), -1).contiguous(), pos.double()[:, None] * freq)[:, None]

    def turned(x):
        x = x.clone()
        y = torch.complex(x[..., first], x[..., second]) * z
        x[..., first], x[..., second] = y.real, y.imag
        return x

    codes = torch.tensor(CODES, dtype=torch.float64, device=q.device)
    borders = (codes[1:] + codes[:-1]) / 2
    page = s["table"][torch.arange(len(pos), device=q.device) // n, pos // P].long()
    out = [turned(q)]
    for x, new in (("k", turned(k).to(s["k"].dtype)), ("v", v)):  # the key that is held is the rotated one, in its type
        y = new.double().unflatten(-1, (-1, 16))
        scale = (y.abs().amax(-1) / 6).clamp(2.0 ** -9, 448.0).float().to(torch.float8_e4m3fn).double()[..., None]
        a = y.abs() / scale
        at = torch.bucketize(a, borders)  # a border belongs to the code below it, and to the one above where that is even
        up = (a == borders[at.clamp(max=6)]) & (at % 2 == 1)
        held = _exact_values(s[x + "_codes"], s[x + "_scales"].view(torch.uint8))
        held[page, pos % P] = (torch.sign(y) * codes[at + up] * scale).flatten(-2)
        out.append(held)
    return tuple(out)
