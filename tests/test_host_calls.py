"""The entry points on the host, over a CUDA runtime without a device
(``tests/harness/host/fake_runtime.cpp``): what a failed launch leaves behind."""
import ctypes
import os
import subprocess
import tempfile

import pytest

from product_vq_kv_gb300 import build as lib_build
import product_vq_kv_gb300._binding as bind

HERE = os.path.dirname(os.path.abspath(__file__))
FAKE = os.path.join(HERE, "harness", "host", "fake_runtime.cpp")
LIB = os.path.join(HERE, "harness", "_build", "libfake_calls.so")
OK, CUDA = 0, 3
P = 0x10000  # an address that is never used


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(LIB) or any(os.path.getmtime(p) > os.path.getmtime(LIB) for p in [FAKE] + lib_build.DEPENDS):
        os.makedirs(os.path.dirname(LIB), exist_ok=True)
        arch = ["-gencode", "arch=compute_103a,code=compute_103a"]  # the kernels are not run
        flags = ["-O1", "-std=c++17", "--fmad=false", "-Xcompiler", "-fPIC", "-I", lib_build.CSRC,
                 "-I", os.path.join(lib_build.ROOT, "include")]
        with tempfile.TemporaryDirectory(dir=os.path.dirname(LIB)) as tmp:
            jobs = []
            for src in [FAKE] + lib_build.SOURCES:
                obj = os.path.join(tmp, os.path.basename(src) + ".o")
                jobs.append((obj, subprocess.Popen([lib_build.nvcc(), *arch, *flags, "-c", "-o", obj, src])))
            assert all(proc.wait() == 0 for _, proc in jobs)
            out = os.path.join(tmp, "lib.so")
            subprocess.run([lib_build.nvcc(), *arch, "--cudart", "none", "-Xlinker", "-Bsymbolic", "-shared", "-o", out,
                            *(obj for obj, _ in jobs)], check=True)
            os.replace(out, LIB)
    return bind._configure(ctypes.CDLL(LIB))


def reserve(lib, requests=4):
    return lib.vq_paged_reserve(P, P, requests, P, P, 10, P, 8, 16, 5, P, P, P, P, None)


def trim(lib, requests=4):
    return lib.vq_paged_trim(P, P, requests, P, 8, 16, P, P, 10, P, P, None)


def append(lib, n_c=256, dtype=0, smooth=None, sub=8):
    return lib.vq_paged_append(P, P, 256, 256, P, 4, 2, 128, sub, n_c, P, P, smooth, P, P, 4, 16, 2 * 16 * (128 // sub),
                               dtype, None)


def attend(lib, requests=2, tokens=300, max_new=200, dtype=0, dim=128, sub=8):
    ws = lib.vq_paged_attention_workspace_bytes(requests, tokens, max_new, 4, 2, dim, sub, 256, 16)
    return lib.vq_paged_attention(P, 4 * dim, P, P, requests, tokens, max_new, P, 80, P, P, 4, 16, 32 * (dim // sub), P, P,
                                  4, 2, dim, sub, 256, 0, 0.0, dtype, P, P, P, ws, None)


def encode(lib, n_c=256, dtype=0, n=100000, sub=4):
    return lib.vq_encode_grouped(P, P, 2, n, n_c, sub, dtype, P, None)


def decode_attention(lib, hkv=2, sub=8):
    ws = lib.vq_attention_workspace_bytes(2, 8, hkv, 3000, 128, sub, 256, 0)
    return lib.vq_attention_decode(P, P, P, P, P, 2, 8, hkv, 3000, 128, sub, 256, 0, 0.0, 0, P, P, ws, None)


CALLS = {
    "reserve": reserve, "reserve of many": lambda lib: reserve(lib, 8192), "trim": trim, "append": append,
    "append, general": lambda lib: append(lib, sub=16), "append, smoothed": lambda lib: append(lib, smooth=P),
    "attention of chunks": attend, "attention of few rows": lambda lib: attend(lib, 2, 2, 1),
    "attention, general": lambda lib: attend(lib, dtype=2), "encode": encode,
    "encode, small codebook": lambda lib: encode(lib, n_c=16), "encode, general": lambda lib: encode(lib, sub=3),
    "decode attention": decode_attention,
}


@pytest.mark.parametrize("name", CALLS)
def test_a_failed_launch_is_reported_once(lib, name):
    """The launch that fails is that call's error and no later one's."""
    call = CALLS[name]
    before = lib.fake_launches()
    assert call(lib) == OK and lib.fake_launches() > before
    for n in range(1, lib.fake_launches() - before + 1):
        lib.fake_fail_in(n)
        assert call(lib) == CUDA
        assert lib.fake_last_error() == 0
    assert call(lib) == OK


def test_a_kernel_has_one_limit_of_shared_memory(lib):
    """The limit is the kernel's: calls of other sizes, in other threads, must not lower
    it under a launch.  So every call of a kernel sets the same one."""
    for requests in (5, 4100, 6000, 8192):
        assert reserve(lib, requests) == trim(lib, requests) == OK
    for n_c in (64, 100, 256):
        for dtype in (0, 1, 2):
            assert append(lib, n_c, dtype) == append(lib, n_c, dtype, smooth=P) == append(lib, n_c, dtype, sub=4) == OK
            assert encode(lib, n_c, dtype) == encode(lib, n_c, dtype, sub=8) == OK
    for n_c in (1000, 1500, 2000, 4096):
        assert encode(lib, n_c) == encode(lib, n_c, sub=8) == OK
    for shape in (dict(), dict(sub=4), dict(hkv=4), dict(hkv=8), dict(hkv=1), dict(hkv=1, sub=4)):
        assert decode_attention(lib, **shape) == OK
    assert lib.fake_most_limits() == 1


def test_calls_of_several_threads(lib):
    """Large and small calls of the same kernels side by side: none finds its limit
    lowered."""
    import threading

    wrong = []

    def work(requests, n_c):
        for _ in range(3000):
            if reserve(lib, requests) or trim(lib, requests) or append(lib, n_c):
                wrong.append(requests)

    threads = [threading.Thread(target=work, args=a) for a in ((8192, 256), (4100, 64), (5000, 128), (8000, 200))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong
