"""Every kernel variant that the plan of the 16-bit feed-forward products picks has a
shape in the GPU tests: a refit of the plan's constants that moves a variant out of
their reach fails here. The plan's own source is compiled for the host
(ffn_plan_query.cpp) and asked for 60000 shapes."""
import ctypes as C
import math
import os
import random
import subprocess

import pytest

import test_ffn_gpu as base
import test_ffn_variants_gpu as variants

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")


@pytest.fixture(scope="module")
def query(tmp_path_factory):
    lib = str(tmp_path_factory.mktemp("plan") / "libplan.so")
    out = subprocess.run(
        [HIPCC, "-x", "hip", "--offload-host-only", "-std=c++17", "-O2", "-fPIC", "-shared",
         "-I", os.path.join(ROOT, "include"),
         "-I", os.path.join(ROOT, "bit_quantized_matmul_col_amd", "csrc"),
         os.path.join(ROOT, "tests", "ffn_plan_query.cpp"), "-o", lib],
        capture_output=True, text=True, timeout=300)
    assert out.returncode == 0, out.stderr
    L = C.CDLL(lib)
    buf = (C.c_int * 9)()
    for f in (L.query_forward, L.query_backward):
        f.argtypes, f.restype = [C.c_int, C.c_int64, C.c_int64, C.c_int64, C.c_void_p], None

    def forward(M, K, N):
        """The variants of a product and a gated product."""
        keys = set()
        for gated in (0, 1):
            L.query_forward(gated, M, K, N, buf)
            keys.add(("gated" if gated else "forward", *buf[:3]))
        return keys

    def backward(M, K, N):
        """The variants of dX alone, dW alone and both, of a product and a gated product."""
        keys = set()
        for grads in (1, 2):
            L.query_backward(grads, M, K, N, buf)
            keys |= {(kind, grads, *buf[3 * i:3 * i + 3])
                     for i, kind in enumerate(("dX", "dW", "both"))}
        return keys
    return forward, backward


def test_the_gpu_tests_reach_every_variant(query):
    forward, backward = query
    held = set().union(*(forward(*s) for s in base.SHAPES + variants.FORWARD),
                       *(backward(*s) for s in base.BACK + variants.BACKWARD))
    rng = random.Random(5)

    def size(lo, hi, mult):
        v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
        return max(mult, int(v / mult + 0.5) * mult)
    missing = {}
    for _ in range(60000):
        s = (size(1, 8192, 1), size(8, 28672, 8), size(8, 28672, 8))
        for key in (forward(*s) | backward(*s)) - held:
            missing.setdefault(key, s)
    assert not missing, missing
