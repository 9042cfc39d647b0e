"""Runs host code of the library against a runtime that launches nothing (fake_cudart.cpp), in a process of its own.

    with_fake_runtime(tmp_path, body)   # body: Python source; `lib` is the library, `launches()` what it launched

The process never loads torch or the real runtime, so pointers may be made up: nothing follows them.
"""
import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)

PRELUDE = """
import ctypes, struct, sys
fake = ctypes.CDLL({fake!r})
sys.modules["torch"] = type(sys)("torch")      # _lib.load() wants it only for the real runtime
import importlib.util
spec = importlib.util.spec_from_file_location("_lib", {lib_py!r})
_lib = importlib.util.module_from_spec(spec)
spec.loader.exec_module(_lib)
lib = _lib.load()

def launches():
    out, name, sizes, thread = [], ctypes.create_string_buffer(400), (ctypes.c_uint * 6)(), ctypes.c_size_t()
    for i in range(fake.fake_count()):
        fake.fake_get(i, name, 400, sizes, ctypes.byref(thread))
        out.append((name.value.decode(), tuple(sizes[:3]), tuple(sizes[3:]), thread.value))
    return out

def batch(**kw):
    v = dict(k=4096, v=4096, k_page=1 << 16, k_token=4096, k_head=64, v_page=1 << 16, v_token=4096, v_head=64, pages=2,
             page_size=16, kv_heads=1, dim=64, page_table=4096, table_stride=2, table_width=2, batch=1, kv_lens=4096,
             cu_q=4096, tokens=1)
    v.update(kw)
    return struct.pack("@PPqqqqqqiiiiPqiiPPi4x", *v.values())
"""


def with_fake_runtime(tmp_path, body):
    from draft_verification_spec_gb300 import build as B
    B.build(quiet=True)
    so, versions = os.path.join(tmp_path, "libcudart.so.13"), os.path.join(tmp_path, "versions")
    with open(versions, "w") as f:
        f.write("libcudart.so.13 { global: *; };\n")
    subprocess.run(["g++", "-std=c++17", "-shared", "-fPIC", "-pthread", "-o", so, os.path.join(HERE, "fake_cudart.cpp"),
                    "-Wl,-soname,libcudart.so.13", f"-Wl,--version-script={versions}"], check=True)
    program = PRELUDE.format(fake=so, lib_py=os.path.join(ROOT, "draft_verification_spec_gb300", "_lib.py")) + body
    r = subprocess.run([sys.executable, "-c", program], capture_output=True, text=True, timeout=120,
                       env={**os.environ, "LD_LIBRARY_PATH": str(tmp_path)})
    assert r.returncode == 0, r.stdout + r.stderr
    return r.stdout
