"""Host side of the step operators (no device): frequencies of the rotary plans, refusals of the C ABI that
come before any CUDA call."""
import ctypes
import math
import struct

import pytest
import torch


@pytest.fixture(scope="module")
def lib():
    from draft_verification_spec_gb300 import build as B
    B.build(quiet=True)
    from draft_verification_spec_gb300 import _lib
    return _lib.load()


def _plan(**kw):
    import draft_verification_spec_gb300 as sv
    return sv.RopePlan(64, device="cpu", **kw)


def test_rope_plan_plain_and_turns():
    p = _plan(theta=10000.0)
    assert p.factor == 1.0 and len(p.frequencies) == 32
    for j, f in enumerate(p.frequencies):
        assert f == pytest.approx(10000.0 ** (-2 * j / 64), rel=1e-15)
    # the 64-bit fractions of a turn, after a million positions, against the angle in 64 bits
    for f, t in zip(p.frequencies, p.turns.tolist()):
        phase = (t * 1_000_000) % 2 ** 64 / 2.0 ** 64 * 2 * math.pi
        want = math.fmod(f * 1_000_000, 2 * math.pi)
        d = abs(phase - want) % (2 * math.pi)
        assert min(d, 2 * math.pi - d) < 1e-8


def test_rope_plan_scalings():
    base = _plan(theta=500000.0).frequencies
    lin = _plan(theta=500000.0, scaling={"type": "linear", "factor": 4.0}).frequencies
    assert [a * 4 for a in lin] == pytest.approx(base)
    ntk = _plan(theta=500000.0, scaling={"type": "ntk", "factor": 8.0}).frequencies
    assert ntk[0] == pytest.approx(base[0]) and ntk[-1] * 8.0 == pytest.approx(base[-1])
    yarn = _plan(theta=10000.0, scaling={"type": "yarn", "factor": 16.0, "original": 4096})
    plain = _plan(theta=10000.0).frequencies
    turns = [4096 * f / (2 * math.pi) for f in plain]
    for f, g, t in zip(plain, yarn.frequencies, turns):
        if t > 32 * 2:
            assert g == pytest.approx(f)
        elif t < 0.5:
            assert g * 16 == pytest.approx(f)
        else:
            assert f / 16 * 0.999999 <= g <= f * 1.000001
    assert yarn.factor == pytest.approx(0.1 * math.log(16.0) + 1.0)
    assert _plan(scaling={"type": "yarn", "factor": 4.0, "original": 4096, "attention_factor": 1.5}).factor == 1.5


@pytest.mark.parametrize("bad", [dict(rotary_dim=3), dict(rotary_dim=0), dict(rotary_dim=128), dict(layout="pairs"),
                                 dict(theta=0.0), dict(scaling={"type": "linear", "factor": 0.0}),
                                 dict(scaling={"type": "spline", "factor": 2.0})])
def test_rope_plan_refusals(bad):
    with pytest.raises(ValueError):
        _plan(**bad)


def _batch(**kw):
    """A spec_paged_batch_t with made-up pointers (never followed: every call here is refused)."""
    v = dict(k=4096, v=4096, k_page=1024, k_token=64, k_head=64, v_page=1024, v_token=64, v_head=64, pages=2, page_size=16,
             kv_heads=1, dim=64, page_table=4096, table_stride=2, table_width=2, batch=1, kv_lens=4096, cu_q=4096, tokens=1)
    v.update(kw)
    return struct.pack("@PPqqqqqqiiiiPqiiPPi4x", *v.values())


def _attention(lib, batch, dtype=1, q_heads=4, max_q=1, window=0, scale=0.1, q=4096, out=4096, ws=4096, q_token=256):
    return lib.spec_chunk_attention(q, q_token, 64, dtype, q_heads, batch, max_q, scale, 1, window, out, None, ws, 1 << 30, None)


def test_attention_refusals(lib):
    invalid, unsupported, workspace = 1, 2, 6
    assert _attention(lib, None) == invalid
    assert _attention(lib, _batch(), dtype=0) == invalid          # fp32
    assert _attention(lib, _batch(), dtype=7) == invalid
    assert _attention(lib, _batch(), window=-1) == invalid
    assert _attention(lib, _batch(), scale=math.inf) == invalid
    assert _attention(lib, _batch(kv_heads=3)) == invalid         # 4 query heads over 3
    assert _attention(lib, _batch(k=4097)) == invalid             # not 16-byte aligned
    assert _attention(lib, _batch(k_token=63)) == invalid
    assert _attention(lib, _batch(table_stride=1)) == invalid
    assert _attention(lib, _batch(page_size=0)) == invalid
    assert _attention(lib, _batch(page_table=0)) == invalid
    assert _attention(lib, _batch(dim=60)) == unsupported
    assert _attention(lib, _batch(dim=264)) == unsupported
    assert _attention(lib, _batch(), q_token=100) == invalid
    assert _attention(lib, _batch(), q=0) == invalid
    assert _attention(lib, _batch(), ws=0) == workspace
    assert _attention(lib, _batch(), ws=4097) == workspace
    assert _attention(lib, _batch(batch=0, tokens=0)) == 0        # nothing to do
    assert lib.spec_attention_workspace_bytes(0, 4, 1, 64, 1) == 0
    assert lib.spec_attention_workspace_bytes(1, 4, 1, 264, 1) == 0


def test_rope_refusals(lib):
    t = struct.pack("@PPPPPqqqqqqqqqq", 4096, 4096, 4096, 4096, 0, *([64] * 10))
    call = lambda tensors=t, dtype=1, batch=_batch(), freq=4096, r=64, f=1.0, ws=4096: lib.spec_rope_append(  # noqa: E731
        tensors, dtype, 4, batch, freq, r, f, 0, ws, None)
    assert call(tensors=None) == 1
    assert call(dtype=3) == 1
    assert call(r=63) == 1 and call(r=66) == 1 and call(r=-2) == 1
    assert call(f=math.nan) == 1
    assert call(freq=0) == 1
    assert call(ws=0) == 6
    assert call(batch=_batch(dim=2048)) == 2
    assert call(batch=_batch(k=0)) == 1                           # no cache, and nowhere to put the keys
    assert call(batch=_batch(batch=0, tokens=0)) == 0


def test_sampling_refusals(lib):
    how = lambda T=1.0, k=0, p=1.0, m=0.0: struct.pack("@fiffPPPP", T, k, p, m, 0, 0, 0, 0)  # noqa: E731
    call = lambda dtype=0, rows=1, V=100, h=how(), logits=4096, u=4096, tok=4096, stride=100, filt=None, fs=100: \
        lib.spec_sample_tokens(logits, stride, dtype, rows, V, u, h, tok, None, None, filt, fs, None)  # noqa: E731
    assert call(dtype=2) == 1 and call(rows=-1) == 1 and call(V=0) == 1 and call(h=None) == 1
    assert call(h=how(T=-1.0)) == 1 and call(h=how(T=math.nan)) == 1 and call(h=how(p=math.nan)) == 1
    assert call(h=how(m=math.nan)) == 1
    assert call(stride=99) == 1 and call(filt=4096, fs=99) == 1
    assert call(V=262145, stride=262145) == 2
    assert call(logits=None) == 1 and call(u=None) == 1 and call(tok=None) == 1
    assert call(rows=0) == 0


def test_structures_match_the_header():
    """The packed formats of the binding have the sizes that a C compiler gives the header's structures."""
    from draft_verification_spec_gb300 import step

    class B(ctypes.Structure):
        _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p)] + [(n, ctypes.c_longlong) for n in "abcdef"] + \
                   [(n, ctypes.c_int) for n in "ghij"] + [("t", ctypes.c_void_p), ("ts", ctypes.c_longlong), ("tw", ctypes.c_int),
                                                          ("b", ctypes.c_int), ("l", ctypes.c_void_p), ("c", ctypes.c_void_p),
                                                          ("n", ctypes.c_int)]

    class S(ctypes.Structure):
        _fields_ = [("T", ctypes.c_float), ("k", ctypes.c_int), ("p", ctypes.c_float), ("m", ctypes.c_float)] + \
                   [(n, ctypes.c_void_p) for n in "abcd"]

    assert step._BATCH.size == ctypes.sizeof(B)
    assert step._ROPE.size == 15 * 8
    assert step._SAMPLING.size == ctypes.sizeof(S)


def test_cpu_tensors_are_refused():
    import draft_verification_spec_gb300 as sv
    if torch.cuda.is_available():
        pytest.skip("needs a machine without a device for the early part only")
    with pytest.raises(TypeError):
        sv.chunk_attention(torch.zeros(1, 1, 64), None, None, None, None, None, 1)     # float32
    with pytest.raises(TypeError):
        sv.rope_append(torch.zeros(1, 1, 64, dtype=torch.float64), None, None, None, None, None, None, None, None)
    with pytest.raises(ValueError):
        sv.sample_tokens(torch.zeros(5), torch.zeros(5))
