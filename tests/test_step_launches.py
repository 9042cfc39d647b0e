"""What the step operators launch, seen by a runtime that launches nothing (no device)."""
from tests.fake_runtime import with_fake_runtime


def test_rope_of_tokens_too_wide_for_the_quotients(tmp_path):
    """rope_kernel divides a piece's number by the pieces of a token in 32 bits, which is exact up to 65,535 pieces; a wider
    token takes the kernel without such quotients."""
    for pieces in (65537, 76800):       # in integers: the last pieces of such a token would be taken for the next one's
        inverse = 0xffffffff // pieces + 1
        assert any((n * inverse >> 32) != 0 for n in (pieces - 1, pieces - 2))
    assert all((n * (0xffffffff // d + 1) >> 32) == n // d for d in (2, 3, 4097, 65533, 65535) for n in range(d))
    out = with_fake_runtime(tmp_path, """
def kernel(q_heads, kv_heads, dim, dtype):
    fake.fake_clear()
    t = struct.pack("@PPPPPqqqqqqqqqq", 4096, 4096, 4096, 4096, 0, *([1 << 20, 1024] * 5))
    b = batch(kv_heads=kv_heads, dim=dim, k_head=1024, v_head=1024, k_token=1 << 20, v_token=1 << 20, tokens=3)
    assert lib.spec_rope_append(t, dtype, q_heads, b, 4096, dim, 1.0, 0, 4096, None) == 0
    (name, grid, _, _), = launches()
    return "scalar" if "rope_scalar_kernel" in name else "pieces"

print(kernel(32, 8, 128, 1), kernel(155, 50, 1024, 0), kernel(156, 50, 1024, 0), kernel(200, 50, 1024, 0), kernel(500, 50, 1024, 1))
""")
    assert out.split() == ["pieces", "pieces", "scalar", "scalar", "scalar"]


def test_attention_on_a_thread_without_a_context(tmp_path):
    """A thread's first call into CUDA has no current context yet, without which TMA descriptors cannot be made: it gets one,
    and the kernel that every other call of these sizes runs."""
    out = with_fake_runtime(tmp_path, """
import threading

def call():
    b = batch(tokens=20)
    assert lib.spec_chunk_attention(4096, 256, 64, 1, 4, b, 20, 0.1, 1, 0, 4096, None, 4096, 1 << 30, None) == 0

def twice():
    call()
    call()

t = threading.Thread(target=twice)
t.start()
t.join()
print(*["tc" if "attn_tc_kernel" in l[0] else "mma" for l in launches()[::2]])
""")
    assert out.split() == ["tc", "tc"]


def test_attention_launches_its_two_kernels_together(tmp_path):
    """Two threads on one stream and workspace: no call's kernel comes between another's pair, which talk through it."""
    out = with_fake_runtime(tmp_path, """
import threading
fake.fake_delay(30)
b = batch(tokens=4)

def call(max_q):
    assert lib.spec_chunk_attention(4096, 256, 64, 1, 4, b, max_q, 0.1, 1, 0, 4096, None, 4096, 1 << 30, None) == 0

call(4)
fake.fake_clear()
threads = [threading.Thread(target=lambda n=n: [call(n) for _ in range(4)]) for n in (4, 5, 40)]
[t.start() for t in threads]
[t.join() for t in threads]
done = launches()
assert len(done) == 24
for a, c in zip(done[::2], done[1::2]):
    assert "combine" not in a[0] and "combine" in c[0] and a[3] == c[3], done
print("pairs")
""")
    assert out.split() == ["pairs"]
