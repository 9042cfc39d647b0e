"""What the operators on pages and caches in 4 bits launch and refuse, seen by a runtime that launches nothing (no device)."""
import pytest

from tests.fake_runtime import with_fake_runtime


def test_append_without_queries(tmp_path):
    """Keys and values alone: null query pointers, or any others and any strides, are no reason for the kernel that takes a head at
    a time; a rotation in place is."""
    out = with_fake_runtime(tmp_path, """
def rope(q=0, out=0, stride=1024, dim=80, k_out=0, heads=0):
    fake.fake_clear()
    t = struct.pack("@PPPPPqqqqqqqqqq", q, 4096, 4096, out, k_out, stride, 128, 1024, 128, 1024, 128, stride, 128, 1024, 128)
    codes = batch(k_page=1 << 15, k_token=512, k_head=64, v_page=1 << 15, v_token=512, v_head=64, dim=dim, tokens=3)
    scales = struct.pack("@PPqqqqqqff", 4096, 4096, 1 << 12, 64, 8, 1 << 12, 64, 8, 1.0, 1.0)
    assert lib.spec_rope_append_fp4(t, 1, heads, codes, scales, 4096, dim, 1.0, 0, 4096, None) == 0
    (name, *_), = launches()
    return "scalar" if "scalar" in name else "blocks"

print(rope(), rope(dim=128), rope(q=4096, out=4096), rope(q=4100, out=4099, stride=-7), rope(k_out=8192), rope(k_out=4096))
print(rope(4096, 4096, heads=4), rope(4096, 8192, heads=4), rope(4100, 8192, heads=4), rope(4096, 8192, stride=1001, heads=4))
""")
    assert out.split("\n")[:2] == ["blocks blocks blocks blocks blocks scalar", "scalar blocks scalar scalar"]


def test_pools_and_tables_beyond_the_kernels_counters(tmp_path):
    """Counters of rows, entries and pages step past the last one by up to 1024: near 2^31 they would start again below zero."""
    out = with_fake_runtime(tmp_path, """
def both(pages, rows, width):
    fake.fake_clear()
    pool = struct.pack("@Piiq", 0, 0, pages, 0)
    table = (4096, max(width, 1), rows, width)
    ws = (4096, 1 << 62, None)
    a = lib.spec_assign_pages(pool, 16, *table, 4096, 4096, None, 4096, max(width, 1), *ws)
    c = lib.spec_compact_pages(pool, *table, 4096, max(width, 1), 4096, *ws)
    return a, c, len(launches()), lib.spec_pages_workspace_bytes(pages, rows) > 0

most = 1 << 30
print(both(most, 3, 4), both(10, most, 1), both(10, 1, most), both(10, 1 << 15, 1 << 15))
print(both(most + 1, 3, 4), both(2 ** 31 - 1, 3, 4), both(10, 2 ** 31 - 1, 1), both(10, most + 1, 0), both(10, 3, 2 ** 29), both(10, 1, 2 ** 31 - 1))
""")
    fine, refused = out.split("\n")[:2]
    assert fine == " ".join(["(0, 0, 2, True)"] * 4)
    big = "(2, 2, 0, False)"
    assert refused == " ".join([big] * 4 + ["(2, 2, 0, True)"] * 2)


def test_a_pool_of_too_many_pages_is_refused():
    import draft_verification_spec_gb300 as sv
    for pages in (2 ** 30 + 1, 2 ** 31, 2 ** 40):
        with pytest.raises(ValueError):
            sv.PagePool([], pages=pages)
