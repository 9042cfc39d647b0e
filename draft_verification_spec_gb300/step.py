"""The operators of a speculative decoding step around its verification.

    from draft_verification_spec_gb300 import RopePlan, chunk_attention, rope_append, sample_tokens
    rope = RopePlan(head_dim, theta=10000.0)
    q = rope_append(q, k, v, rope, k_cache, v_cache, page_table, kv_lens, cu_q)
    out = chunk_attention(q, k_cache, v_cache, page_table, kv_lens, cu_q, max_q)
    s = sample_tokens(logits, uniforms, temperature=0.8, top_p=0.95, want_filtered=True)

A batch is packed: tokens ``cu_q[b]:cu_q[b+1]`` are the new ones of request b, the last of its
``kv_lens[b]`` tokens; its token t is slot ``t % page_size`` of page ``page_table[b, t // page_size]``
of caches [pages, page_size, kv_heads, dim].  Lengths stay on the device.  With ``stream=`` a call runs
on that stream: it waits for nothing on the current one (the caller orders the two), and its tensors'
memory is kept until it is done.  As in the rest of the package, this file checks arguments, allocates
outputs and passes pointers; the contracts are in include/spec_verify.h.
"""
from __future__ import annotations

import math
import struct
from dataclasses import dataclass
from typing import Optional

import torch

_CODES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}
_device = torch.cuda.current_device
_current_stream = torch._C._cuda_getCurrentRawStream   # torch.cuda.current_stream(), without the object around it


# the ABI's structures, packed in one go (a ctypes field costs as much as a check): native alignment
_BATCH = struct.Struct("@PPqqqqqqiiiiPqiiPPi4x")     # spec_paged_batch_t
_ROPE = struct.Struct("@PPPPPqqqqqqqqqq")            # spec_rope_tensors_t
_SAMPLING = struct.Struct("@fiffPPPP")               # spec_sampling_t


_lib = None
_workspace = None


def _bind():
    """The package's library and workspaces (looked up once: this module is imported by the package)."""
    global _lib, _workspace
    import draft_verification_spec_gb300 as m
    _lib, _workspace = m.lib(), m._workspace_of
    return _lib


def _check(code, where):
    import draft_verification_spec_gb300 as m
    m._check(code, where)


def _raw_stream(stream, index):
    return _current_stream(index) if stream is None else stream.cuda_stream


def _where(t, name, index):
    return ValueError(f"{name} must be on the current device cuda:{index}, it is on {t.device}")


def _int(v):
    """A bound or count for a C int: what is beyond it stands for as much as the largest one (a refused one stays refused)."""
    return v if -0x80000000 <= v <= 0x7fffffff else 0x7fffffff if v > 0 else -0x80000000


def _step_buffer(workspace, index, raw, need, stream):
    """The workspace's buffer (None: the default workspace of the stream) of `need` bytes at least."""
    if workspace is None:
        workspace = _workspace(index, raw)
    elif workspace.device.type != "cuda" or workspace.device.index != index:
        raise ValueError(f"workspace must be on the current device cuda:{index}, it is on {workspace.device}")
    return workspace.get_step(need, stream)


def _fresh(stream, shape, dtype, device):
    """An output.  With a stream it is that stream's memory, for the current stream to read: the current stream's free memory
    may still be read by work that is queued there, which the kernel on `stream` would not wait for."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    here = torch.cuda.current_stream()
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=device)
    t.record_stream(here)
    return t


def _used_on(stream, *tensors):
    """Memory of the caller's tensors is not handed out again before the work queued on `stream` is done with it."""
    for t in tensors:
        if isinstance(t, torch.Tensor):
            t.record_stream(stream)


def _heads(t, name, index, n=None, dim=None):
    """Strides of a [tokens, heads, dim] tensor on the current device whose heads are contiguous."""
    if t.get_device() != index:
        raise _where(t, name, index)
    s = t.shape
    if len(s) != 3 or (n is not None and s[0] != n) or (dim is not None and s[2] != dim):
        raise ValueError(f"{name} must be [tokens, heads, dim], got {tuple(s)}")
    st = t.stride()
    if st[2] != 1 and s[2] > 1 and s[0] and s[1]:
        raise ValueError(f"{name}: the values of a head must be contiguous")
    return st


def _batch(k_cache, v_cache, page_table, kv_lens, cu_q, tokens, kv_heads, dim, dtype, index):
    """spec_paged_batch_t of checked tensors."""
    if kv_lens.dtype != torch.int32 or cu_q.dtype != torch.int32:
        raise TypeError(f"kv_lens and cu_q must be torch.int32, got {kv_lens.dtype} and {cu_q.dtype}")
    if kv_lens.get_device() != index or cu_q.get_device() != index:
        raise _where(cu_q if kv_lens.get_device() == index else kv_lens, "kv_lens and cu_q", index)
    ls, cs = kv_lens.shape, cu_q.shape
    if len(ls) != 1 or len(cs) != 1 or cs[0] != ls[0] + 1 or not (kv_lens.is_contiguous() and cu_q.is_contiguous()):
        raise ValueError(f"kv_lens and cu_q must be contiguous, of B and B + 1 entries, got {tuple(ls)} and {tuple(cs)}")
    B = ls[0]
    if k_cache is None:
        return _BATCH.pack(0, 0, 0, 0, 0, 0, 0, 0, 0, 0, kv_heads, dim, 0, 0, 0, B, kv_lens.data_ptr(), cu_q.data_ptr(), tokens)
    if k_cache.get_device() != index or v_cache.get_device() != index or page_table.get_device() != index:
        bad = next(t for t in (k_cache, v_cache, page_table) if t.get_device() != index)
        raise _where(bad, "k_cache, v_cache and page_table", index)
    if k_cache.dtype != dtype or v_cache.dtype != dtype:
        raise TypeError(f"k_cache and v_cache must be {dtype}, got {k_cache.dtype} and {v_cache.dtype}")
    s = k_cache.shape
    if len(s) != 4 or v_cache.shape != s or s[2] != kv_heads or s[3] != dim:
        raise ValueError(f"k_cache and v_cache must be [pages, page_size, {kv_heads}, {dim}], got {tuple(s)} and "
                         f"{tuple(v_cache.shape)}")
    k0, k1, k2, k3 = k_cache.stride()
    v0, v1, v2, v3 = v_cache.stride()
    if (k3 != 1 or v3 != 1) and dim > 1:
        raise ValueError("k_cache and v_cache: the values of a head must be contiguous")
    if page_table.dtype != torch.int32:
        raise TypeError(f"page_table must be torch.int32, got {page_table.dtype}")
    if page_table.dim() != 2 or page_table.shape[0] != B:
        raise ValueError(f"page_table must be [{B}, pages of a request], got {tuple(page_table.shape)}")
    width = page_table.shape[1]
    row, col = page_table.stride()
    if (width > 1 and col != 1) or (B > 1 and row < width):
        raise ValueError("page_table must have contiguous rows that do not overlap")
    return _BATCH.pack(k_cache.data_ptr(), v_cache.data_ptr(), k0, k1, k2, v0, v1, v2, s[0], s[1], kv_heads, dim,
                       page_table.data_ptr(), row if row > width else width, width, B, kv_lens.data_ptr(), cu_q.data_ptr(),
                       tokens)


_ws_bytes: dict = {}


def chunk_attention(q, k_cache, v_cache, page_table, kv_lens, cu_q, max_q: int, *, causal: bool = True,
                    window: int = 0, scale: Optional[float] = None, want_lse: bool = False, out=None, stream=None,
                    workspace=None, tuning=None):
    """Attention of the new tokens q [tokens, q_heads, dim] over the paged cache (spec_chunk_attention).

    ``max_q`` bounds the new tokens of a request.  ``causal``: a token sees the keys up to its own;
    otherwise all of its request.  ``window`` > 0: only keys within that many positions back, its
    own included (pages wholly behind it may be gone).  ``scale`` defaults to dim ** -0.5.  Returns
    out [tokens, q_heads, dim], with ``want_lse`` (out, lse [tokens, q_heads] float32); a row that
    sees no key gives 0 and -inf, rows of tokens that no request has stay unwritten.
    ``tuning``: a Tuning, of which the wait limit counts here (spec_chunk_attention_tuned).
    """
    lib = _lib or _bind()
    dtype = q.dtype
    code = _CODES.get(dtype)
    if code != 1 and code != 2:
        raise TypeError(f"q must be bfloat16 or float16, got {dtype}")
    index = _device()
    max_q, window = _int(max_q), _int(window)
    q_token, q_head, _ = _heads(q, "q", index)
    n, hq, d = q.shape
    if k_cache.dim() != 4:
        raise ValueError("k_cache must be [pages, page_size, kv_heads, dim]")
    hkv = k_cache.shape[2]
    c = _batch(k_cache, v_cache, page_table, kv_lens, cu_q, n, hkv, d, dtype, index)
    if out is None:
        out = _fresh(stream, (n, hq, d), dtype, q.device)
    elif out.shape != q.shape or out.dtype != dtype or out.get_device() != index or not out.is_contiguous():
        raise ValueError("out must be a contiguous tensor of q's shape, dtype and device")
    lse = _fresh(stream, (n, hq), torch.float32, q.device) if want_lse else None
    key = (index, code, hq, hkv, d, max_q if max_q < 129 else 129)   # more than 128 rows are all alike
    need = _ws_bytes.get(key)
    if need is None:
        need = _ws_bytes[key] = lib.spec_attention_workspace_bytes(code, hq, hkv, d, max_q)
    raw = _raw_stream(stream, index)
    buf = _step_buffer(workspace, index, raw, need, stream)
    args = (q.data_ptr(), q_token, q_head, code, hq, c, max_q, d ** -0.5 if scale is None else scale, causal, window,
            out.data_ptr(), None if lse is None else lse.data_ptr(), buf.data_ptr(), buf.numel(), raw)
    if stream is not None:
        _used_on(stream, q, k_cache, v_cache, page_table, kv_lens, cu_q, out)
    err = lib.spec_chunk_attention(*args) if tuning is None else lib.spec_chunk_attention_tuned(*args, tuning.ref())
    if err:
        _check(err, "spec_chunk_attention")
    return (out, lse) if want_lse else out


class RopePlan:
    """Rotation frequencies of the rotary positions: theta^(-2j/r) turns of 2 pi a position for the r/2 pairs
    of the first r = ``rotary_dim`` values of a head, as 64-bit fractions of a turn on the device.

    layout: "half" pairs (j, j + r/2), "interleaved" pairs (2j, 2j + 1).
    scaling (for contexts longer than the trained one):
      {"type": "linear", "factor": s}  every frequency / s;
      {"type": "ntk", "factor": s}     theta s^(r / (r - 2)), which divides the slowest frequency by s and
                                       keeps the fastest;
      {"type": "yarn", "factor": s, "original": L, "beta_fast": 32, "beta_slow": 1, "attention_factor": None}
        frequencies with more than beta_fast turns over the trained length L stay, those with less than
        beta_slow are divided by s, a ramp over the pairs' index between; rotated values are multiplied by
        attention_factor (0.1 ln s + 1).
    """

    def __init__(self, head_dim: int, rotary_dim: Optional[int] = None, theta: float = 10000.0, layout: str = "half",
                 scaling: Optional[dict] = None, device=None):
        r = head_dim if rotary_dim is None else int(rotary_dim)
        if r < 2 or r % 2 or r > head_dim:
            raise ValueError(f"rotary_dim must be even, in [2, {head_dim}], got {r}")
        if layout not in ("half", "interleaved"):
            raise ValueError(f"layout must be 'half' or 'interleaved', got {layout!r}")
        if not theta > 0:
            raise ValueError("theta must be positive")
        self.head_dim, self.rotary_dim, self.theta, self.layout = int(head_dim), r, float(theta), layout
        self.interleaved = int(layout == "interleaved")
        self.frequencies, self.factor = self._frequencies(r, float(theta), scaling)
        turns = [int(round(f / (2.0 * math.pi) * 2.0 ** 64)) % 2 ** 64 for f in self.frequencies]
        signed = [t - 2 ** 64 if t >= 2 ** 63 else t for t in turns]
        device = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
        self.turns = torch.tensor(signed, dtype=torch.int64, device=device)

    @staticmethod
    def _frequencies(r, theta, scaling):
        base = [theta ** (-2.0 * j / r) for j in range(r // 2)]
        if scaling is None:
            return base, 1.0
        kind, s = scaling.get("type"), float(scaling.get("factor", 0.0))
        if not s > 0:
            raise ValueError("scaling needs a positive factor")
        if kind == "linear":
            return [f / s for f in base], 1.0
        if kind == "ntk":
            if r < 4:
                raise ValueError("ntk scaling needs rotary_dim >= 4")
            t = theta * s ** (r / (r - 2.0))
            return [t ** (-2.0 * j / r) for j in range(r // 2)], 1.0
        if kind == "yarn":
            L = float(scaling["original"])

            def pair(turns):   # the (fractional) pair that makes this many turns over L positions
                return r * math.log(L / (turns * 2.0 * math.pi)) / (2.0 * math.log(theta))

            lo = max(0, math.floor(pair(float(scaling.get("beta_fast", 32.0)))))
            hi = min(r - 1, math.ceil(pair(float(scaling.get("beta_slow", 1.0)))))
            out = []
            for j, f in enumerate(base):
                ramp = min(max((j - lo) / max(hi - lo, 1e-3), 0.0), 1.0)
                out.append(f / s * ramp + f * (1.0 - ramp))
            m = scaling.get("attention_factor")
            return out, (0.1 * math.log(s) + 1.0 if s > 1 else 1.0) if m is None else float(m)
        raise ValueError(f"unknown scaling type {kind!r}")


def rope_append(q, k, v, rope: RopePlan, k_cache, v_cache, page_table, kv_lens, cu_q, *, q_out=None, k_out=None,
                stream=None, workspace=None):
    """Rotary positions of the new tokens and the write of rotated keys and values into the paged cache
    (spec_rope_append).

    q [tokens, q_heads, dim], k and v [tokens, kv_heads, dim], float32, bfloat16 or float16.  Returns the
    rotated queries (in ``q_out``, which may be q).  ``k_out`` receives the rotated keys too (may be k);
    it is required where k_cache, v_cache and page_table are None and nothing is stored.  Rows of tokens
    that no request has stay unwritten.
    """
    lib = _lib or _bind()
    dtype = q.dtype
    code = _CODES.get(dtype)
    if code is None:
        raise TypeError(f"q must be float32, bfloat16 or float16, got {dtype}")
    index = _device()
    q0, q1, _ = _heads(q, "q", index)
    n, hq, d = q.shape
    k0, k1, _ = _heads(k, "k", index, n, d)
    hkv = k.shape[1]
    if k.dtype != dtype:
        raise TypeError(f"k must be {dtype}, got {k.dtype}")
    if rope.head_dim != d:
        raise ValueError(f"the plan is for heads of {rope.head_dim}, q has {d}")
    if rope.turns.get_device() != index:
        raise _where(rope.turns, "the plan", index)
    v0 = v1 = vp = o0 = o1 = op = 0
    ws = None
    raw = _raw_stream(stream, index)
    if k_cache is not None:
        v0, v1, _ = _heads(v, "v", index, n, d)
        if v.dtype != dtype or v.shape[1] != hkv:
            raise (TypeError if v.dtype != dtype else ValueError)(f"v must be {dtype} of {hkv} heads, got {v.dtype} of {v.shape[1]}")
        vp = v.data_ptr()
        ws = _step_buffer(workspace, index, raw, 256, stream).data_ptr()
    elif k_out is None:
        raise ValueError("k_out is required where there is no cache")
    c = _batch(k_cache, v_cache, page_table, kv_lens, cu_q, n, hkv, d, dtype, index)
    if q_out is None:
        q_out = _fresh(stream, (n, hq, d), dtype, q.device)
        w0, w1 = hq * d, d
    else:
        w0, w1, _ = _heads(q_out, "q_out", index, n, d)
        if q_out.shape[1] != hq or q_out.dtype != dtype:
            raise ValueError("q_out must have q's shape and dtype")
    if k_out is not None:
        o0, o1, _ = _heads(k_out, "k_out", index, n, d)
        if k_out.shape[1] != hkv or k_out.dtype != dtype:
            raise ValueError("k_out must have k's shape and dtype")
        op = k_out.data_ptr()
    r = _ROPE.pack(q.data_ptr(), k.data_ptr(), vp, q_out.data_ptr(), op, q0, q1, k0, k1, v0, v1, w0, w1, o0, o1)
    if stream is not None:
        _used_on(stream, q, k, v, rope.turns, k_cache, v_cache, page_table, kv_lens, cu_q, q_out, k_out)
    err = lib.spec_rope_append(r, code, hq, c, rope.turns.data_ptr(), rope.rotary_dim, rope.factor, rope.interleaved, ws, raw)
    if err:
        _check(err, "spec_rope_append")
    return q_out


@dataclass
class SampleOutput:
    tokens: torch.Tensor                     # [rows] int32; -1 for a row without a logit above -inf
    probs: torch.Tensor                      # [rows] float32: the token's probability among the kept ones
    kept: torch.Tensor                       # [rows] int32: how many tokens the filters keep
    filtered: Optional[torch.Tensor] = None  # [rows, V]: the kept tokens' logits, -inf elsewhere


def _overlap(a, b):
    """Whether two [rows, V] tensors of one type and shape, values of a row contiguous, share memory."""
    (rows, V), size = a.shape, a.element_size()
    sa, sb = (t.stride(0) if rows > 1 else V for t in (a, b))
    gap = (b.data_ptr() - a.data_ptr()) // size
    if rows == 0 or gap >= (rows - 1) * sa + V or -gap >= (rows - 1) * sb + V:
        return False
    return sa != sb or not V <= gap % sa <= sa - V     # rows side by side in one buffer are apart


def _setting(name, value, dtype, rows, index):
    """(number, pointer) of a setting that is a number or a tensor of one per row."""
    if not isinstance(value, torch.Tensor):
        return (_int(value) if dtype == torch.int32 else value), 0
    if value.get_device() != index:
        raise ValueError(f"{name} must be a number or on the current device cuda:{index}, it is on {value.device}")
    if value.dtype != dtype or tuple(value.shape) != (rows,) or not value.is_contiguous():
        raise ValueError(f"{name} must be a number or a contiguous {dtype} tensor of {rows}")
    return 0, value.data_ptr()


def sample_tokens(logits, uniforms, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0, *, want_filtered: bool = False,
                  stream=None, out: Optional[SampleOutput] = None) -> SampleOutput:
    """Temperature, top-k, top-p and min-p sampling from given uniforms (spec_sample_tokens).

    logits [rows, V] bfloat16 or float32 (rows may be strided), uniforms [rows] float32.  Each setting is
    a number or a tensor of one per row (float32, top_k int32); top_k <= 0, top_p >= 1 and min_p <= 0 keep
    all, temperature 0 is greedy.  With ``want_filtered`` the truncated logits come too: what
    verify_chain / verify_block take as the distribution that the token was drawn from (their
    ``temperature`` is one for the batch, so rows sampled at others are not theirs to verify).
    """
    lib = _lib or _bind()
    if logits.dim() != 2:
        raise ValueError("logits must be [rows, V]")
    dtype = logits.dtype
    code = _CODES.get(dtype)
    if code != 0 and code != 1:
        raise TypeError(f"logits must be bfloat16 or float32, got {dtype}")
    R, V = logits.shape
    index, dev = _device(), logits.device
    if logits.get_device() != index or uniforms.get_device() != index:
        raise _where(uniforms if logits.get_device() == index else logits, "logits and uniforms", index)
    row, col = logits.stride()
    if (V > 1 and col != 1) or (R > 1 and row < V):
        raise ValueError("logits: the values of a row must be contiguous, and rows must not overlap")
    if uniforms.dtype != torch.float32 or tuple(uniforms.shape) != (R,) or not uniforms.is_contiguous():
        raise ValueError(f"uniforms must be a contiguous float32 tensor of {R}")
    t0, t1 = _setting("temperature", temperature, torch.float32, R, index)
    k0, k1 = _setting("top_k", top_k, torch.int32, R, index)
    p0, p1 = _setting("top_p", top_p, torch.float32, R, index)
    m0, m1 = _setting("min_p", min_p, torch.float32, R, index)
    c = _SAMPLING.pack(t0, k0, p0, m0, t1, k1, p1, m1)
    if out is None:
        out = SampleOutput(_fresh(stream, R, torch.int32, dev), _fresh(stream, R, torch.float32, dev),
                           _fresh(stream, R, torch.int32, dev), _fresh(stream, (R, V), dtype, dev) if want_filtered else None)
    else:
        for t, name, kind in ((out.tokens, "tokens", torch.int32), (out.probs, "probs", torch.float32),
                               (out.kept, "kept", torch.int32)):
            if t.dtype != kind or tuple(t.shape) != (R,) or not t.is_contiguous() or t.device != dev:
                raise ValueError(f"out.{name} must be a contiguous {kind} tensor of {R} on {dev}")
        f = out.filtered
        if f is not None and (f.dtype != logits.dtype or f.shape != logits.shape or f.device != dev or
                              (V > 1 and f.stride(1) != 1) or (R > 1 and f.stride(0) < V)):
            raise ValueError("out.filtered must have the shape, dtype and device of logits and contiguous rows")
        if f is not None and _overlap(logits, f):
            raise ValueError("out.filtered must not overlap logits")
    f = out.filtered
    if stream is not None:
        _used_on(stream, logits, uniforms, temperature, top_k, top_p, min_p, out.tokens, out.probs, out.kept, f)
    err = lib.spec_sample_tokens(logits.data_ptr(), row if row > V else V, code, R, V, uniforms.data_ptr(), c,
                                 out.tokens.data_ptr(), out.probs.data_ptr(), out.kept.data_ptr(),
                                 None if f is None else f.data_ptr(), V if f is None else max(f.stride(0), V),
                                 _raw_stream(stream, index))
    if err:
        _check(err, "spec_sample_tokens")
    return out


__all__ = ["RopePlan", "SampleOutput", "chunk_attention", "rope_append", "sample_tokens"]
