"""Every kernel variant that the plans of the experts' products and of the block-scaled FP8
product pick has a shape in the GPU tests: a refit of a plan's constants that moves a
variant out of their reach fails here. The plans' own sources are compiled for the host
(routed_plan_query.cpp) and asked for thousands of shapes."""
import ctypes as C
import math
import os
import random
import subprocess

import pytest

import test_experts_calls_gpu as calls
import test_experts_gpu as experts
import test_fp8_block_gpu as fp8

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "bit_quantized_matmul_col_amd", "csrc")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")


@pytest.fixture(scope="module")
def plans(tmp_path_factory):
    lib = str(tmp_path_factory.mktemp("plan") / "libplan.so")
    out = subprocess.run(
        [HIPCC, "-x", "hip", "--offload-host-only", "-std=c++17", "-O2", "-fPIC", "-shared",
         "-I", os.path.join(ROOT, "include"), "-I", CSRC,
         os.path.join(ROOT, "tests", "routed_plan_query.cpp"),
         *(os.path.join(CSRC, f) for f in ("experts_plan.hip", "blockwise_plan.hip")), "-o", lib],
        capture_output=True, text=True, timeout=300)
    assert out.returncode == 0, out.stderr
    L = C.CDLL(lib)
    L.query_experts.argtypes = [C.c_int, C.c_int64, C.c_int, C.c_int64, C.c_int64, C.c_void_p]
    L.query_fp8.argtypes = [C.c_int64, C.c_int64, C.c_int64, C.c_void_p]
    L.query_experts.restype = L.query_fp8.restype = None
    buf = (C.c_int * 6)()

    def of_experts(M, K, N, E, k):
        keys = set()
        for name, kind, n, d in (("second", 0, K, N), ("gated", 1, N, K), ("dX", 2, K, 2 * N),
                                 ("dH", 2, N, K)):
            L.query_experts(kind, M * k, E, n, d, buf)
            keys.add((name, *buf[:4]))
        return keys

    def of_fp8(M, K, N):
        L.query_fp8(M, K, N, buf)
        return {tuple(buf)}
    return of_experts, of_fp8


def size(rng, lo, hi, mult):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(mult, int(v / mult + 0.5) * mult)


def test_the_gpu_tests_reach_every_variant_of_the_experts(plans):
    held = set().union(*(plans[0](*s[:5]) for s in experts.EXPERTS + calls.EXPERTS))
    rng, missing = random.Random(5), {}
    for _ in range(40000):
        E = size(rng, 1, 512, 1)
        s = (size(rng, 1, 16384, 1), size(rng, 8, 11008, 8), size(rng, 8, 11008, 8), E,
             rng.randint(1, min(E, 8)))
        for key in plans[0](*s) - held:
            missing.setdefault(key, s)
    assert not missing, missing


def test_the_gpu_tests_reach_every_variant_of_the_block_scaled_product(plans):
    held = set().union(*(plans[1](*s) for s in fp8.PRODUCTS + calls.FP8))
    rng, missing = random.Random(6), {}
    for _ in range(40000):
        s = (size(rng, 1, 8192, 1), size(rng, 16, 28672, 16), size(rng, 8, 28672, 8))
        for key in plans[1](*s) - held:
            missing.setdefault(key, s)
    assert not missing, missing
