"""csa_kv4_decode from several host threads at once (tests/c/kv4_threads.c:
threads that no interpreter lock keeps apart)."""
import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest

from tests.gpu_common import ensure_built

pytestmark = pytest.mark.gpu


def test_threads_with_different_numbers_of_tokens(tmp_path):
    # one kernel instance, but another amount of shared memory for each T:
    # every call goes through and gives what it gives alone
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ensure_built()
    import certified_sparse_attention_gb300 as csa
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    cc = shutil.which("cc") or shutil.which("gcc")
    if not cc:
        pytest.skip("no C compiler")
    lib, libdir = str(tmp_path / "threads.so"), os.path.dirname(csa.LIB_PATH)
    subprocess.run([cc, "-std=c11", "-Wall", "-Werror", "-fPIC", "-shared",
                    "-I", os.path.join(root, "include"),
                    os.path.join(root, "tests", "c", "kv4_threads.c"),
                    "-L", libdir, "-lcsa", "-lpthread",
                    f"-Wl,-rpath,{libdir}", "-o", lib], check=True)

    class Call(ctypes.Structure):
        _fields_ = [("shape", ctypes.POINTER(csa.csa_shape)),
                    ("cache", ctypes.POINTER(csa.csa_kv4)),
                    ("T", ctypes.c_int), ("repeat", ctypes.c_int),
                    ("q", ctypes.c_void_p),
                    ("qs", ctypes.POINTER(csa.csa_strides)),
                    ("len", ctypes.c_void_p), ("o", ctypes.c_void_p),
                    ("workspace", ctypes.c_void_p),
                    ("workspace_bytes", ctypes.c_size_t),
                    ("stream", ctypes.c_void_p), ("status", ctypes.c_int)]

    dev = torch.device("cuda:0")
    rng = np.random.default_rng(1)
    n, G, d = 700, 4, 128
    s = csa.make_shape(1, G, 1, d, n, "bf16")

    def bf16(*size):
        return torch.from_numpy(rng.normal(size=size).astype(np.float32)).to(dev).bfloat16()
    cache = csa.KV4Cache(s, dev)
    ln = torch.tensor([n], dtype=torch.int64, device=dev)
    cache.append(bf16(1, n, 1, d), bf16(1, n, 1, d), ln)
    tokens = (3, 6, 9, 16)
    calls, keep = (Call * len(tokens))(), []
    for c, T in zip(calls, tokens):
        q, op, st = bf16(1, T, G, d), csa.KV4Decode(s, dev, T), torch.cuda.Stream(dev)
        want = op(q, cache, ln).clone()
        qs = csa.csa_strides(*q.stride()[:3])
        keep.append((q, op, st, want, qs))
        c.shape, c.cache, c.T, c.repeat = ctypes.pointer(s), ctypes.pointer(cache.desc), T, 3000
        c.q, c.qs, c.len = q.data_ptr(), ctypes.pointer(qs), ln.data_ptr()
        c.o, c.workspace = op.o.data_ptr(), op.ws.data_ptr()
        c.workspace_bytes, c.stream = op.ws_bytes, st.cuda_stream
    torch.cuda.synchronize()
    assert ctypes.CDLL(lib).run_calls(calls, len(tokens)) == csa.CSA_OK
    torch.cuda.synchronize()
    for q, op, st, want, qs in keep:
        assert csa.csa_check(op.ws) == 0 and torch.equal(op.o, want)
