"""Host side of the attention with first tokens kept, of caches in 4 bits and of page pools (no device): refusals of the C
ABI that come before any CUDA call, what is launched, the binding's structures and checks."""
import ctypes
import math
import random
import struct

import pytest
import torch

from tests import more_reference as M
from tests.fake_runtime import with_fake_runtime
from tests.test_step_host import _batch


@pytest.fixture(scope="module")
def lib():
    from draft_verification_spec_gb300 import build as B
    B.build(quiet=True)
    from draft_verification_spec_gb300 import _lib
    return _lib.load()


INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 6


def _scales(**kw):
    v = dict(k=4096, v=4096, k_page=64, k_token=4, k_head=4, v_page=64, v_token=4, v_head=4, k_unit=1.0, v_unit=1.0)
    v.update(kw)
    return struct.pack("@PPqqqqqqff", *v.values())


def _codes(**kw):
    """A batch whose strides count the bytes of 4-bit codes."""
    v = dict(k_page=512, k_token=32, k_head=32, v_page=512, v_token=32, v_head=32)
    v.update(kw)
    return _batch(**v)


def test_sinks_refusals(lib):
    call = lambda batch=_batch(), window=4, sinks=2, ws=4096, scale=0.1: lib.spec_chunk_attention_sinks(  # noqa: E731
        4096, 256, 64, 1, 4, batch, 1, scale, 1, window, sinks, 4096, None, ws, 1 << 30, None, None)
    assert call(sinks=-1) == INVALID and call(sinks=-2 ** 31) == INVALID
    assert call(window=-1) == INVALID and call(batch=None) == INVALID
    assert call(scale=math.nan) == INVALID
    assert call(ws=0) == WORKSPACE
    assert call(batch=_batch(batch=0, tokens=0)) == 0


def test_fp4_refusals(lib):
    call = lambda batch=_codes(), scales=_scales(), dtype=1, sinks=0, scale=0.1, ws=4096, heads=4: lib.spec_chunk_attention_fp4(  # noqa: E731
        4096, 256, 64, dtype, heads, batch, scales, 1, scale, 1, 0, sinks, 4096, None, ws, 1 << 30, None, None)
    assert call(scales=None) == INVALID and call(batch=None) == INVALID
    assert call(dtype=0) == INVALID and call(sinks=-1) == INVALID
    assert call(batch=_codes(kv_heads=3)) == INVALID
    assert call(batch=_codes(k_token=36)) == INVALID and call(batch=_codes(v=4100)) == INVALID
    assert call(batch=_codes(k_page=-8)) == INVALID
    for dim in (8, 72, 264, 272):
        assert call(batch=_codes(dim=dim)) == UNSUPPORTED
    for bad in (dict(k=0), dict(v=0), dict(k_token=-1), dict(k_unit=0.0), dict(k_unit=3.0), dict(v_unit=-1.0), dict(v_unit=math.inf),
                dict(k_unit=math.nan), dict(k_unit=2.0 ** 65), dict(v_unit=2.0 ** -65)):
        assert call(scales=_scales(**bad)) == INVALID, bad
    assert call(ws=0) == WORKSPACE and call(ws=4097) == WORKSPACE
    assert call(batch=_codes(batch=0, tokens=0)) == 0
    assert lib.spec_attention_fp4_workspace_bytes(1, 4, 1, 72, 1) == 0
    assert lib.spec_attention_fp4_workspace_bytes(0, 4, 1, 64, 1) == 0

    t = struct.pack("@PPPPPqqqqqqqqqq", 4096, 4096, 4096, 4096, 0, *([64] * 10))
    rope = lambda tensors=t, dtype=1, batch=_codes(), scales=_scales(), freq=4096, r=64, f=1.0, ws=4096: lib.spec_rope_append_fp4(  # noqa: E731
        tensors, dtype, 4, batch, scales, freq, r, f, 0, ws, None)
    assert rope(tensors=None) == INVALID and rope(scales=None) == INVALID and rope(batch=_codes(k=0)) == INVALID
    assert rope(dtype=0) == INVALID                                   # float32 tokens
    assert rope(r=63) == INVALID and rope(r=66) == INVALID and rope(f=math.inf) == INVALID and rope(freq=0) == INVALID
    assert rope(batch=_codes(dim=72), r=8) == UNSUPPORTED and rope(batch=_codes(dim=512), r=8) == UNSUPPORTED
    assert rope(scales=_scales(v_unit=0.3)) == INVALID
    assert rope(ws=0) == WORKSPACE
    assert rope(batch=_codes(batch=0, tokens=0)) == 0

    values = lambda codes=4096, st=(512, 32, 32), scales=4096, ss=(64, 4, 4), unit=1.0, n=(2, 16, 1, 64), dtype=1, out=4096: \
        lib.spec_fp4_values(codes, *st, scales, *ss, unit, *n, dtype, out, None)  # noqa: E731
    assert values(dtype=3) == INVALID and values(unit=0.7) == INVALID and values(n=(2, 0, 1, 64)) == INVALID
    assert values(n=(2, 16, 1, 40)) == UNSUPPORTED and values(n=(-1, 16, 1, 64)) == INVALID
    assert values(st=(512, 33, 32)) == INVALID and values(ss=(64, -4, 4)) == INVALID
    assert values(codes=0) == INVALID and values(scales=0) == INVALID and values(out=4100) == INVALID
    assert values(n=(0, 16, 1, 64)) == 0


def _pool(**kw):
    v = dict(arrays=4096, n=2, pages=10, most=100)
    v.update(kw)
    return struct.pack("@Piiq", *v.values())


def test_page_refusals(lib):
    assign = lambda pool=_pool(), size=16, table=4096, stride=4, rows=3, width=4, lens=4096, kept=4096, out=4096, ostride=4, ws=4096, \
        n=1 << 20: lib.spec_assign_pages(pool, size, table, stride, rows, width, lens, kept, None, out, ostride, ws, n, None)  # noqa: E731
    assert assign(pool=None) == INVALID and assign(pool=_pool(pages=0)) == INVALID and assign(pool=_pool(arrays=0)) == INVALID
    assert assign(pool=_pool(n=-1)) == INVALID and assign(pool=_pool(most=-1)) == INVALID
    assert assign(size=0) == INVALID and assign(stride=3) == INVALID and assign(ostride=3) == INVALID
    assert assign(rows=-1) == INVALID and assign(width=-1) == INVALID
    assert assign(table=0) == INVALID and assign(out=0) == INVALID and assign(lens=0) == INVALID and assign(kept=0) == INVALID
    assert assign(rows=1 << 20, width=1 << 20, stride=1 << 20, ostride=1 << 20) == UNSUPPORTED
    assert assign(ws=0) == WORKSPACE and assign(ws=4100) == WORKSPACE and assign(n=256) == WORKSPACE
    assert assign(rows=0) == 0 and assign(width=0) == 0
    need = lib.spec_pages_workspace_bytes(10, 3)
    assert need % 256 == 0 and assign(n=need - 256) == WORKSPACE
    assert lib.spec_pages_workspace_bytes(0, 3) == 0 and lib.spec_pages_workspace_bytes(3, -1) == 0
    compact = lambda used=4096, **kw: lib.spec_compact_pages(kw.get("pool", _pool()), 4096, 4, 3, 4, kw.get("out", 4096), 4, used,  # noqa: E731
                                                             kw.get("ws", 4096), 1 << 20, None)
    assert compact(used=0) == INVALID and compact(out=0) == INVALID and compact(pool=None) == INVALID and compact(ws=0) == WORKSPACE


def test_structures_match_the_header():
    from draft_verification_spec_gb300 import step

    class S(ctypes.Structure):
        _fields_ = [(n, ctypes.c_void_p) for n in "kv"] + [(n, ctypes.c_longlong) for n in "abcdef"] + [("x", ctypes.c_float), ("y", ctypes.c_float)]

    class P(ctypes.Structure):
        _fields_ = [("a", ctypes.c_void_p), ("n", ctypes.c_int), ("p", ctypes.c_int), ("m", ctypes.c_longlong)]

    assert step._SCALES.size == ctypes.sizeof(S) and step._POOL.size == ctypes.sizeof(P)


def test_what_is_launched(tmp_path):
    """The kernels that sizes, strides and masks choose."""
    out = with_fake_runtime(tmp_path, """
def scales(**kw):
    v = dict(k=4096, v=4096, k_page=1 << 12, k_token=64, k_head=8, v_page=1 << 12, v_token=64, v_head=8, ku=1.0, vu=1.0)
    v.update(kw)
    return struct.pack("@PPqqqqqqff", *v.values())

def codes(**kw):
    v = dict(k_page=1 << 15, k_token=512, k_head=64, v_page=1 << 15, v_token=512, v_head=64, dim=128)
    v.update(kw)
    return batch(**v)

def name(n, args):
    kind = n[0].split("(")[0]
    return kind[kind.index("attn_"):].replace("(bool)", "") if "attn_" in kind else kind

def sinks(max_q, window, n, **kw):
    fake.fake_clear()
    assert lib.spec_chunk_attention_sinks(4096, 256, 64, 1, 4, batch(tokens=40, **kw), max_q, 0.1, 1, window, n, 4096, None, 4096, 1 << 30, None, None) == 0
    first, second = launches()
    assert "combine" in second[0]
    return first[0]

# without a window, or without first tokens, the kernels that were there
plain = [sinks(q, w, n) for q, w, n in ((1, 0, 0), (1, 0, 5), (1, 7, 0), (40, 0, 5), (40, 7, 0))]
kept = [sinks(q, 7, 5) for q in (1, 40)]
print(len({plain[0], plain[1], plain[2]}) == 1, plain[3] == plain[4], kept[0] != plain[0], kept[1] != plain[3])

def fp4(max_q, c=None, s=None, scale=0.1, heads=4):
    fake.fake_clear()
    st = lib.spec_chunk_attention_fp4(4096, 256, 64, 1, heads, c or codes(tokens=40), s or scales(), max_q, scale, 1, 0, 0, 4096, None, 4096, 1 << 30, None, None)
    assert st == 0, st
    return "tc" if "attn_tc_kernel" in launches()[0][0] else "mma", launches()[0][2][0]

print(fp4(1), fp4(4), fp4(8), fp4(9))
print(fp4(40, scale=-0.1)[0], fp4(40, c=codes(tokens=40, dim=256, k_head=128, v_head=128), s=scales(k_head=16, v_head=16))[0])
print(fp4(40, s=scales(v_token=72))[0], fp4(40, c=codes(tokens=40, k_page=1 << 38, v_page=1 << 38), s=scales(k_page=1 << 35, v_page=1 << 35))[0],
      fp4(40, c=codes(tokens=40, page_size=24))[0])

def rope(**kw):
    fake.fake_clear()
    v = dict(q=4096, r=128, dim=128, out=8192)
    v.update(kw)
    t = struct.pack("@PPPPPqqqqqqqqqq", v["q"], 4096, 4096, v["out"], 0, *([1024, 128] * 5))
    assert lib.spec_rope_append_fp4(t, 1, 4, codes(tokens=3, dim=v["dim"]), scales(), 4096, v["r"], 1.0, 0, 4096, None) == 0
    return "scalar" if "scalar" in launches()[0][0] else "blocks"

print(rope(), rope(r=64), rope(r=48), rope(q=4104), rope(dim=80, r=80), rope(dim=96, r=96), rope(dim=80, r=20), rope(r=48, out=4096), rope(out=4096))

def pages(n_arrays, most, rows=3):
    fake.fake_clear()
    pool = struct.pack("@Piiq", 4096 if n_arrays else 0, n_arrays, 10, most)
    assert lib.spec_assign_pages(pool, 16, 4096, 4, rows, 4, 4096, 4096, None, 4096, 4, 4096, 1 << 20, None) == 0
    return [l[1][0] for l in launches()]

print(pages(0, 0), pages(2, 100), pages(2, 100000), pages(2000, 1 << 20))
""")
    got = out.split("\n")
    assert got[0] == "True True True True"
    assert got[1] == "('mma', 128) ('mma', 128) ('mma', 128) ('tc', 512)"
    assert got[2] == "mma mma"
    assert got[3] == "mma mma tc"
    assert got[4] == "blocks blocks blocks scalar blocks blocks scalar scalar blocks"
    sms = int(got[5].rsplit(" ", 1)[1].rstrip("]")) // 8
    assert got[5] == f"[8] [8, 6] [8, 42] [8, {8 * sms}]"


def test_fp4_cache_and_pool_checks():
    import draft_verification_spec_gb300 as sv
    codes, scales = torch.zeros(3, 4, 2, 32, dtype=torch.uint8), torch.zeros(3, 4, 2, 4, dtype=torch.uint8).view(torch.float8_e4m3fn)
    c = sv.FP4Cache.of(codes, scales, 0.25)
    assert c.shape == (3, 4, 2, 64) and c.dim() == 4 and c.unit == 0.25
    f = sv.FP4Cache(3, 4, 2, 64, device="cpu")
    assert f.codes.shape == codes.shape and f.scales.shape == scales.shape and f.codes.transpose(1, 2).is_contiguous()
    for bad in (dict(unit=0.3), dict(unit=-1.0), dict(unit=0.0), dict(unit=math.inf), dict(codes=codes[0]), dict(scales=scales[:2]),
                dict(codes=codes[..., :31]), dict(codes=codes.transpose(2, 3))):
        a = dict(codes=codes, scales=scales, unit=1.0)
        a.update(bad)
        with pytest.raises(ValueError):
            sv.FP4Cache.of(a["codes"], a["scales"], a["unit"])
    with pytest.raises(TypeError):
        sv.FP4Cache.of(codes.float(), scales)
    with pytest.raises(TypeError):
        sv.FP4Cache.of(codes, scales.view(torch.uint8))
    for dim in (8, 40, 272):
        with pytest.raises(ValueError):
            sv.FP4Cache(3, 4, 2, dim, device="cpu")
    pool = sv.PagePool([c, torch.zeros(3, 5)])
    assert pool.pages == 3 and pool.max_bytes == 4 * 2 * 32
    rows = pool.arrays.tolist()
    assert [r[2] for r in rows] == [256, 32, 20] and [r[1] for r in rows] == [256, 32, 20]
    assert sv.PagePool([torch.zeros(3, 4, 5).transpose(1, 2)]).max_bytes == 80
    for bad in ([], [torch.zeros(3, 4), torch.zeros(2, 4)], [torch.zeros(3, 4, 6)[:, :, :3]], [torch.zeros(1, 4).expand(3, 4)]):
        with pytest.raises(ValueError):
            sv.PagePool(bad)


def test_the_plain_forms_agree_with_the_definitions():
    """The references of the GPU tests: a block's scale and codes are the nearest ones, pages are shared as is said."""
    rng = random.Random(3)
    for _ in range(200):
        x = [float(torch.tensor(rng.gauss(0, 1) * 4 ** rng.randint(-3, 3)).bfloat16()) for _ in range(16)]
        byte, codes = M.quantize(x)
        s = M.e4m3(byte)
        for v, c in zip(x, codes):
            mag = M.CODES[c & 7] * s
            assert all(abs(abs(v) - mag) <= abs(abs(v) - o * s) + 1e-12 for o in M.CODES)
            assert v == 0 or (c >= 8) == (v < 0)
    for seed in range(50):
        rng = random.Random(seed)
        B, W, P, pages = rng.randint(1, 6), rng.randint(1, 5), rng.choice([1, 3, 16]), 40
        ids = rng.sample(range(pages), B * W)
        table = [ids[b * W:(b + 1) * W] for b in range(B)]
        parents = [rng.randrange(B) for _ in range(B)]
        kept = [rng.randint(0, W * P) for _ in range(B)]
        lens = [min(W * P, k + rng.randint(0, 4)) for k in kept]
        new, copies, ok = M.assign(table, lens, P, pages, kept, parents)
        written = [new[b][j] for b in range(B) for j in range(kept[b] // P, -(-lens[b] // P)) if lens[b] > kept[b]]
        readers = [new[b][j] for b in range(B) for j in range(kept[b] // P)]
        if ok:      # what a row writes to is its own
            assert len(set(written)) == len(written) and not set(written) & set(readers)
        content = {p: p for p in range(pages)}
        for s, d in copies:
            content[d] = s
        for b in range(B):      # what a row keeps is what it had
            for j in range(-(-min(kept[b], lens[b]) // P)):
                if new[b][j] >= 0:
                    assert content[new[b][j]] == table[parents[b]][j]
