"""The operators of a speculative decoding step around the verification: their cases, inputs and plain forms.

Three operators: ``rope_append`` (rotary positions of new tokens and the write of keys and values into a paged cache),
``chunk_attention`` (attention of the new tokens over that cache) and ``sample_tokens`` (temperature, top-k, top-p and
min-p sampling from given uniforms, with the truncated logits that the verification then reads).
"""
import math
import random

import torch

own = False

ATTENTION = dict(op="attention", dtype="bf16", B=1, nq=1, mixed=False, kv=1024, ragged=False, hq=32, hkv=8, d=128,
                 page=16, causal=True, window=0)
ROPE = dict(op="rope", dtype="bf16", B=1, nq=1, past=1000, hq=32, hkv=8, d=128, rotary=128, layout="half",
            scaling="none", theta=10000.0, page=16)
SAMPLE = dict(op="sample", dtype="bf16", R=1, V=128000, shape="zipf", params="fixed", temperature=0.9, top_k=0,
              top_p=0.95, min_p=0.0, filtered=False)


def listed():
    return [
        # one user, one token over a short conversation: the latency of a plain decoding step
        dict(ATTENTION, name="attention decode 1"),
        # a serving batch of single tokens over caches of ragged length, one slot of the batch idle
        dict(ATTENTION, name="attention decode 64", B=64, kv=8192, ragged=True),
        # verification of an MTP chain of 3 drafts: 4 new tokens for each of 64 requests
        dict(ATTENTION, name="attention verify chain", B=64, nq=4, kv=4096, ragged=True, page=32),
        # verification of a block of 16 drafts over long contexts, 8 query heads a key head
        dict(ATTENTION, name="attention verify block", B=32, nq=17, kv=16384, ragged=True, hq=64, page=64),
        # a block-diffusion draft: 16 tokens that see each other both ways; 7 heads a key head, pages of 24, fp16
        dict(ATTENTION, name="attention draft block", dtype="f16", B=5, nq=16, kv=1999, ragged=True, hq=14, hkv=2, d=64,
             page=24, causal=False),
        # chunked prefill: 2048 tokens of two prompts behind 14336 that are cached
        dict(ATTENTION, name="attention prompt chunk", B=2, nq=2048, kv=16384, page=128),
        # one token of one request
        dict(ROPE, name="rope 1"),
        # the 17 positions of 64 requests under verification, interleaved pairs over half of the head, fp16
        dict(ROPE, name="rope verify block", dtype="f16", B=64, nq=17, past=5000, layout="interleaved", rotary=64),
        # chunks of four prompts far into long contexts, positions scaled
        dict(ROPE, name="rope prompt chunk", B=4, nq=2048, past=120000, scaling="yarn", theta=500000.0, page=64),
        # one row: the draft's next token of one request
        dict(SAMPLE, name="sample 1"),
        # 64 requests with settings of their own (greedy ones among them), fp32 logits, an odd vocabulary
        dict(SAMPLE, name="sample 64", dtype="f32", R=64, V=100003, params="mixed"),
        # the target's rows of 64 requests x 17 positions, truncated for the verification and sampled
        dict(SAMPLE, name="sample verify rows", R=1088, params="mixed", filtered=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["attention", "attention", "rope", "sample"])
    if op == "attention":
        c = dict(ATTENTION, dtype=rng.choice(["bf16", "bf16", "f16"]), B=_log(rng, 1, 64), ragged=rng.random() < 0.7,
                 hkv=rng.choice([1, 2, 4, 8]), d=rng.choice([64, 80, 128, 128, 256]),
                 page=rng.choice([1, 8, 16, 24, 32, 64, 128, 256]), causal=rng.random() < 0.75,
                 window=rng.choice([0, 0, 0, _log(rng, 16, 4096)]))
        c["hq"] = c["hkv"] * rng.choice([1, 2, 4, 7, 8, 16])
        kind = rng.choice(["token", "verify", "prompt"])
        c["nq"] = 1 if kind == "token" else _log(rng, 2, 32) if kind == "verify" else _log(rng, 33, 2048)
        c["mixed"] = kind == "prompt" and rng.random() < 0.5
        c["kv"] = _log(rng, 1, 32768)
        while c["B"] * c["kv"] * c["hkv"] * c["d"] > 2 ** 29 or c["B"] * c["hq"] * c["nq"] * c["kv"] * max(128, c["d"]) > 2 ** 38:
            c["B"], c["kv"] = max(1, c["B"] * 2 // 3), max(1, int(c["kv"] * 0.8))
        return c
    if op == "rope":
        c = dict(ROPE, dtype=rng.choice(["bf16", "bf16", "f16", "f32"]), B=_log(rng, 1, 64),
                 hkv=rng.choice([1, 2, 4, 8]), d=rng.choice([64, 80, 128, 128, 256]),
                 layout=rng.choice(["half", "interleaved"]), scaling=rng.choice(["none", "linear", "ntk", "yarn"]),
                 past=_log(rng, 1, 1000000), theta=rng.choice([10000.0, 500000.0]), page=rng.choice([1, 8, 16, 24, 64, 128]))
        c["hq"] = c["hkv"] * rng.choice([1, 2, 4, 7, 8])
        c["rotary"] = rng.choice([c["d"], c["d"], c["d"] // 2])
        c["nq"] = _log(rng, 1, max(1, min(2048, 2 ** 25 // (c["B"] * (c["hq"] + 2 * c["hkv"]) * c["d"]))))
        return c
    c = dict(SAMPLE, dtype=rng.choice(["bf16", "f32"]), V=_log(rng, 1000, 131072), shape=rng.choice(["zipf", "zipf", "normal"]),
             params=rng.choice(["fixed", "mixed"]), temperature=rng.choice([0.0, 0.6, 0.9, 1.0, 1.4]),
             top_k=rng.choice([0, 0, 1, 50, 1000]), top_p=rng.choice([1.0, 0.95, 0.8]), min_p=rng.choice([0.0, 0.0, 0.02, 0.1]),
             filtered=rng.random() < 0.5)
    c["R"] = _log(rng, 1, min(1088, 2 ** 26 // c["V"]))
    return c


DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def _size(case):
    return {"bf16": 2, "f16": 2, "f32": 4}[case["dtype"]]


def _lengths(case):
    """New tokens and cache lengths (the new tokens included) of every request: the case's own, whatever the seed."""
    rng = random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))
    B, nq = case["B"], case["nq"]
    new = [nq if b == 0 or not case["mixed"] else 1 for b in range(B)]
    kv = [rng.randint(max(1, case["kv"] // 8), case["kv"]) if case["ragged"] and b else case["kv"] for b in range(B)]
    kv = [max(n, k) for n, k in zip(new, kv)]
    if case["ragged"] and B >= 8:
        kv[-1] = 0  # an idle slot of the batch: its rows see no key
    return new, kv


def _visible(case, new, kv):
    """How many (query, key) pairs of one head the mask leaves."""
    pairs = 0
    for n, k in zip(new, kv):
        for i in range(n):
            pos = k - n + i
            hi = min(k, pos + 1) if case["causal"] else k
            lo = max(0, pos - case["window"] + 1) if case["window"] else 0
            pairs += max(0, hi - lo)
    return pairs


def _keys_seen(case, new, kv):
    """How many keys of one head some query of their request sees."""
    total = 0
    for n, k in zip(new, kv):
        lo = max(0, k - n - case["window"] + 1) if case["window"] else 0
        total += max(0, k - lo)
    return total


def work(case):
    e = _size(case)
    if case["op"] == "attention":
        new, kv = _lengths(case)
        n, pages = sum(new), sum(-(-k // case["page"]) for k in kv)
        rows = 2 * n * case["hq"] * case["d"] * e + 4 * n * case["hq"]
        cache = 2 * _keys_seen(case, new, kv) * case["hkv"] * case["d"] * e
        return {"bytes": rows + cache + 4 * pages + 8 * case["B"], "flops": 4 * case["d"] * case["hq"] * _visible(case, new, kv)}
    if case["op"] == "rope":
        n = case["B"] * case["nq"]
        values = n * (case["hq"] + 2 * case["hkv"]) * case["d"]
        return {"bytes": 2 * values * e + 4 * n, "flops": 3 * n * (case["hq"] + case["hkv"]) * case["rotary"]}
    n = case["R"] * case["V"]
    return {"bytes": n * e * (2 if case["filtered"] else 1) + 32 * case["R"], "flops": 4 * n}


def _scaling(case):
    return {"none": None, "linear": {"type": "linear", "factor": 4.0}, "ntk": {"type": "ntk", "factor": 4.0},
            "yarn": {"type": "yarn", "factor": 16.0, "original": 8192, "beta_fast": 32.0, "beta_slow": 1.0}}[case["scaling"]]


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dev, dt = "cuda", DTYPES[case["dtype"]]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=dev)

    s = {"case": case}
    if case["op"] == "sample":
        R, V = case["R"], case["V"]
        if case["shape"] == "zipf":  # logits of a language model's shape: -1.1 ln(rank), with noise
            z = torch.log1p(torch.rand(R, V, generator=g, device=dev) * V).mul_(-1.1).add_(normal(R, V).mul_(0.5))
        else:
            z = normal(R, V).mul_(3.0)
        s["logits"] = z.to(dt)
        s["uniforms"] = torch.rand(R, generator=g, device=dev)
        if case["params"] == "fixed":
            s.update({k: case[k] for k in ("temperature", "top_k", "top_p", "min_p")})
        else:  # every request has settings of its own
            pick = lambda v: torch.tensor(v, device=dev)[torch.randint(len(v), (R,), generator=g, device=dev)]  # noqa: E731
            s["temperature"] = pick([0.0, 0.5, 0.7, 0.9, 1.0, 1.3])
            s["top_k"] = pick([0, 1, 20, 50, 400, 5000]).to(torch.int32)
            s["top_p"] = pick([1.0, 0.99, 0.95, 0.9, 0.5])
            s["min_p"] = pick([0.0, 0.0, 0.01, 0.1])
        return s
    B, hq, hkv, d, P = case["B"], case["hq"], case["hkv"], case["d"], case["page"]
    if case["op"] == "attention":
        new, kv = _lengths(case)
    else:
        new, kv = [case["nq"]] * B, [case["past"] + b + case["nq"] for b in range(B)]
    n = sum(new)
    starts = [sum(new[:b]) for b in range(B + 1)]
    first = [0] * B if case["op"] == "attention" else [(k - m) // P for m, k in zip(new, kv)]  # the first page that holds something
    used = [-(-k // P) - f for k, f in zip(kv, first)]
    pages = sum(used) + 3
    width = max(1, max(u + f for u, f in zip(used, first)))
    order = torch.randperm(pages, generator=g, device=dev).to(torch.int32)
    # page j of request b: the pool's pages in a random order; -1 where a request has none
    cols = torch.arange(width, device=dev)
    at = torch.tensor([sum(used[:b]) - first[b] for b in range(B)], device=dev)[:, None] + cols
    has = (cols >= torch.tensor(first, device=dev)[:, None]) & (cols < torch.tensor([u + f for u, f in zip(used, first)], device=dev)[:, None])
    s["table"] = torch.where(has, order[at.clamp(0, pages - 1)], torch.full_like(order[:1], -1)).contiguous()
    s["cu_q"] = torch.tensor(starts, dtype=torch.int32, device=dev)
    s["kv_lens"] = torch.tensor(kv, dtype=torch.int32, device=dev)
    s["max_q"] = max(new)
    s["max_kv"] = max(kv)
    if case["op"] == "attention":
        s["q"] = normal(n, hq, d).mul_(1.5).to(dt)  # scores of a spread that makes some keys stand out
        s["k_cache"], s["v_cache"] = (normal(pages, P, hkv, d).to(dt) for _ in range(2))
        return s
    s["q"], s["k"], s["v"] = (normal(n, h, d).to(dt) for h in (hq, hkv, hkv))
    s["k_cache"], s["v_cache"] = (normal(pages, P, hkv, d).to(dt) for _ in range(2))
    if own:
        import draft_verification_spec_gb300 as sv

        s["rope"] = sv.RopePlan(d, rotary_dim=case["rotary"], theta=case["theta"], layout=case["layout"], scaling=_scaling(case))
    else:
        s["freq"], s["factor"] = _frequencies(case)
    return s


def run(s):
    case = s["case"]
    if own:
        import draft_verification_spec_gb300 as sv

        if case["op"] == "attention":
            return sv.chunk_attention(s["q"], s["k_cache"], s["v_cache"], s["table"], s["kv_lens"], s["cu_q"], s["max_q"],
                                      causal=case["causal"], window=case["window"], want_lse=True)
        if case["op"] == "rope":
            q = sv.rope_append(s["q"], s["k"], s["v"], s["rope"], s["k_cache"], s["v_cache"], s["table"], s["kv_lens"], s["cu_q"])
            return q, s["k_cache"], s["v_cache"]
        r = sv.sample_tokens(s["logits"], s["uniforms"], s["temperature"], s["top_k"], s["top_p"], s["min_p"],
                             want_filtered=case["filtered"])
        return r.tokens, r.probs, r.kept, r.filtered
    return {"attention": _plain_attention, "rope": _plain_rope, "sample": _plain_sample}[case["op"]](s)


def _plain_attention(s):
    case = s["case"]
    q, table, dt = s["q"], s["table"], s["q"].dtype
    cu, kv = s["cu_q"].long(), s["kv_lens"].long()
    n, hq, d = q.shape
    hkv, P, B = case["hkv"], case["page"], case["B"]
    new = cu[1:] - cu[:-1]
    i, t = torch.arange(s["max_q"], device=q.device), torch.arange(s["max_kv"], device=q.device)
    page = table[:, t // P].clamp(min=0).long()
    keys, values = (c[page, t % P].float().transpose(1, 2) for c in (s["k_cache"], s["v_cache"]))  # [B, hkv, kv, d]
    queries = q[(cu[:-1, None] + i).clamp(max=n - 1)].float()  # [B, nq, hq, d]
    queries = queries.view(B, len(i), hkv, hq // hkv, d).permute(0, 2, 3, 1, 4).reshape(B, hkv, -1, d)
    scores = (queries @ keys.transpose(2, 3) * (1.0 / math.sqrt(d))).view(B, hq, len(i), len(t))
    pos = (kv - new)[:, None] + i  # the place of each query in its request
    seen = (t < kv[:, None, None]) & (i[:, None] < new[:, None, None])
    if case["causal"]:
        seen = seen & (t <= pos[:, :, None])
    if case["window"]:
        seen = seen & (t > pos[:, :, None] - case["window"])
    scores = scores.masked_fill_(~seen[:, None], float("-inf"))
    top = scores.amax(3, keepdim=True)
    top = torch.where(top == float("-inf"), torch.zeros_like(top), top)
    w = scores.sub_(top).exp_()
    total = w.sum(3, keepdim=True)
    out = (w.view(B, hkv, -1, len(t)) @ values).view(B, hq, len(i), d)
    out = torch.where(total > 0, out / total, torch.zeros_like(out))
    lse = (top + total.log()).squeeze(3)
    b = torch.repeat_interleave(torch.arange(B, device=q.device), new, output_size=n)
    j = torch.arange(n, device=q.device) - cu[b]
    return out[b, :, j].to(dt), lse[b, :, j]


def _frequencies(case):
    """Radians a position of every pair, in 64 bits (a position of 10^5 leaves 32 bits no digits behind the turn), and the
    factor of YaRN on the rotated values."""
    r, theta, sc = case["rotary"], case["theta"], _scaling(case)
    j = torch.arange(r // 2, dtype=torch.float64, device="cuda")
    if sc is None:
        return theta ** (-2.0 * j / r), 1.0
    if sc["type"] == "linear":
        return theta ** (-2.0 * j / r) / sc["factor"], 1.0
    if sc["type"] == "ntk":
        return (theta * sc["factor"] ** (r / (r - 2.0))) ** (-2.0 * j / r), 1.0
    turns = lambda b: r * math.log(sc["original"] / (b * 2.0 * math.pi)) / (2.0 * math.log(theta))  # noqa: E731
    lo, hi = max(0, math.floor(turns(sc["beta_fast"]))), min(r - 1, math.ceil(turns(sc["beta_slow"])))
    ramp = ((j - lo) / max(hi - lo, 1e-3)).clamp(0.0, 1.0)
    f = theta ** (-2.0 * j / r)
    return f / sc["factor"] * ramp + f * (1.0 - ramp), 0.1 * math.log(sc["factor"]) + 1.0


def _plain_rope(s):
    case = s["case"]
    cu, kv = s["cu_q"].long(), s["kv_lens"].long()
    n, r, P = s["q"].shape[0], case["rotary"], case["page"]
    b = torch.repeat_interleave(torch.arange(case["B"], device=cu.device), cu[1:] - cu[:-1], output_size=n)
    pos = torch.arange(n, device=cu.device) - cu[b + 1] + kv[b]
    angle = pos.double()[:, None] * s["freq"]
    cos, sin = (torch.cos(angle) * s["factor"]).float()[:, None], (torch.sin(angle) * s["factor"]).float()[:, None]

    def turn(x):
        y = x.float()
        a, c = (y[..., : r // 2], y[..., r // 2: r]) if case["layout"] == "half" else (y[..., 0:r:2], y[..., 1:r:2])
        a, c = a * cos - c * sin, c * cos + a * sin
        y = torch.cat([a, c] if case["layout"] == "half" else [torch.stack([a, c], -1).flatten(-2)], -1)
        return torch.cat([y, x[..., r:].float()], -1).to(x.dtype)

    page = s["table"][b, pos // P].long()
    s["k_cache"][page, pos % P] = turn(s["k"])
    s["v_cache"][page, pos % P] = s["v"]
    return turn(s["q"]), s["k_cache"], s["v_cache"]


def _rows(v, R, dtype):
    return v.to(dtype)[:, None] if isinstance(v, torch.Tensor) else torch.full((R, 1), v, dtype=dtype, device="cuda")


def _plain_sample(s):
    """Masses and their sums are in 64 bits: the token and the cut are whole numbers, and must not hang on a rounding."""
    z, u = s["logits"], s["uniforms"]
    R, V = z.shape
    f32 = lambda v: _rows(v, R, torch.float32).double()  # noqa: E731 (what the settings are as 32-bit numbers)
    T, k, top_p, min_p = f32(s["temperature"]), _rows(s["top_k"], R, torch.int64), f32(s["top_p"]), f32(s["min_p"])
    v, order = torch.sort(z.float(), dim=1, descending=True, stable=True)
    j = torch.arange(V, device=z.device)
    w = (v.double() - v[:, :1].double()).div_(torch.where(T > 0, T, torch.ones_like(T))).exp_()
    w = torch.where(T > 0, w, (j == 0).double())
    in_k = (j < k) | (k <= 0)
    mass = w * in_k
    keep = in_k & (mass.cumsum(1) - mass < top_p * mass.sum(1, keepdim=True)) & (w >= min_p) & ((T > 0) | (j == 0))
    keep = (keep | (j == 0)) & (v > float("-inf"))
    mass = w * keep
    kept, total, upto = keep.sum(1), mass.sum(1), mass.cumsum(1)
    at = torch.minimum((upto <= u.double()[:, None] * total[:, None]).sum(1), kept - 1)[:, None]
    tokens = order.gather(1, at)[:, 0].to(torch.int32)
    probs = (mass.gather(1, at)[:, 0] / total).float()
    filtered = None
    if s["case"]["filtered"]:
        filtered = torch.full_like(v, float("-inf")).scatter_(1, order, torch.where(keep, v, torch.full_like(v, float("-inf")))).to(z.dtype)
    return tokens, probs, kept.to(torch.int32), filtered


def exact(case, seed):
    s = prepare(case, seed)
    return {"attention": _exact_attention, "rope": _exact_rope, "sample": _exact_sample}[case["op"]](s)


def _exact_attention(s):
    case = s["case"]
    cu, kv, table = s["cu_q"].tolist(), s["kv_lens"].tolist(), s["table"]
    g, P, d = case["hq"] // case["hkv"], case["page"], case["d"]
    outs, lses = [], []
    for b in range(case["B"]):
        q = s["q"][cu[b]:cu[b + 1]].double()
        n, length = q.shape[0], kv[b]
        out, lse = torch.zeros_like(q), torch.full(q.shape[:2], float("-inf"), dtype=torch.float64, device=q.device)
        if length:
            pages = table[b, : -(-length // P)].long()
            K, V = (c[pages].flatten(0, 1)[:length].double() for c in (s["k_cache"], s["v_cache"]))
            where = torch.arange(length, device=q.device)[None] - (length - n + torch.arange(n, device=q.device)[:, None])
            mask = torch.zeros(n, length, dtype=torch.float64, device=q.device)
            if case["causal"]:
                mask.masked_fill_(where > 0, float("-inf"))
            if case["window"]:
                mask.masked_fill_(where <= -case["window"], float("-inf"))
            some = (mask == 0).any(1)
            for h in range(case["hq"]):
                x = q[:, h] @ K[:, h // g].T / math.sqrt(d) + mask
                lse[:, h] = torch.logsumexp(x, 1)
                out[:, h] = torch.where(some[:, None], torch.exp(x - lse[:, h, None]) @ V[:, h // g], out[:, h])
        outs.append(out)
        lses.append(lse)
    return torch.cat(outs), torch.cat(lses)


def _exact_rope(s):
    case = s["case"]
    freq, factor = _frequencies(case)
    cu, kv, r, P = s["cu_q"].tolist(), s["kv_lens"].tolist(), case["rotary"], case["page"]
    first, second = (list(range(r // 2)), list(range(r // 2, r))) if case["layout"] == "half" else (list(range(0, r, 2)), list(range(1, r, 2)))
    q, k, v = (s[x].double() for x in "qkv")
    kc, vc = s["k_cache"].double(), s["v_cache"].double()
    q_out = q.clone()
    for b in range(case["B"]):
        at = slice(cu[b], cu[b + 1])
        pos = torch.arange(kv[b] - (cu[b + 1] - cu[b]), kv[b], device=q.device)
        z = torch.polar(torch.full_like(freq, factor).expand(len(pos), -1).contiguous(), pos.double()[:, None] * freq)[:, None]

        def turned(x):
            x = x.clone()
            y = torch.complex(x[..., first], x[..., second]) * z
            x[..., first], x[..., second] = y.real, y.imag
            return x

        page = s["table"][b, (pos // P)].long()
        q_out[at] = turned(q[at])
        kc[page, pos % P], vc[page, pos % P] = turned(k[at]), v[at]
    return q_out, kc, vc


def _exact_sample(s):
    R, V = s["logits"].shape
    at = lambda v, i: float(v[i]) if isinstance(v, (list, tuple)) else float(torch.tensor(v, dtype=torch.float32))  # noqa: E731
    T, k, top_p, min_p = (x.tolist() if isinstance(x, torch.Tensor) else x for x in (s["temperature"], s["top_k"], s["top_p"], s["min_p"]))
    u, probs, filtered = s["uniforms"].tolist(), [], []
    for i in range(R):
        z = s["logits"][i].double()
        place = torch.argsort(-z, stable=True)  # the tokens from the most likely on, the lowest first among equals
        n = V if at(T, i) > 0 else 1
        n = min(n, int(at(k, i))) if at(k, i) > 0 else n
        w = torch.exp((z[place[:n]] - z.max()) / (at(T, i) or 1.0))
        share = torch.cumsum(w / w.sum(), 0)
        n_p = 1 + int((share[:-1] < at(top_p, i)).sum())
        n_m = int((w >= at(min_p, i)).sum())
        n = max(1, min(n, n_p, n_m, int((z > float("-inf")).sum())))
        w = w[:n] / w[:n].sum()
        probs.append(w[min(int((torch.cumsum(w, 0) <= u[i]).sum()), n - 1)])
        if s["case"]["filtered"]:
            row = torch.full_like(z, float("-inf"))
            row[place[:n]] = z[place[:n]]
            filtered.append(row.float())
    return None, torch.stack(probs), None, torch.stack(filtered) if filtered else None
