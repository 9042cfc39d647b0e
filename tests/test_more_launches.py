"""What the operators on pages and caches in 4 bits launch and refuse, seen by a runtime that launches nothing (no device)."""
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
