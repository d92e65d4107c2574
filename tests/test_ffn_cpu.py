"""The 16-bit feed-forward operators without a GPU: every refusal of the C calls (in a
child process with the GPUs hidden, so that a wrongly accepted call could not reach one),
the workspace queries, the binding's own checks, and the 64-bit definitions that the GPU
tests use against differences and against themselves."""
import json
import os
import subprocess
import sys

import pytest
import torch

import ffn_oracle as fo

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "bit_quantized_matmul_col_amd", "libllmint8.so")


@pytest.fixture(autouse=True)
def _library(built_library):
    return built_library


CHILD = r"""
import ctypes as C, json, sys
L = C.CDLL(sys.argv[1])
p, i64, i, sz = C.c_void_p, C.c_int64, C.c_int, C.c_size_t
class Saved(C.Structure):
    _fields_ = [("data", p), ("ld", i64), ("scales", p), ("ld_scales", i64)]
class Opts(C.Structure):
    _fields_ = [("struct_size", sz), ("activation", i), ("bias", p), ("residual", p), ("ldr", i64),
                ("Z", p), ("ldz", i64)]
L.llmint8_checkpoint_pack.argtypes = [p, i64, i64, i64, i, p, p]
L.llmint8_checkpoint_unpack.argtypes = [p, i64, i64, i, p, i64, p]
L.llmint8_matmul.argtypes = [p, i64, i64, i64, p, i64, i64, i, p, i64, p, p, sz, p]
L.llmint8_matmul_backward.argtypes = [p, i64, i64, i64, p, i64, p, i64, p, i64, i, i, p, i64, p,
                                      i64, p, p, sz, p]
L.llmint8_gated.argtypes = [p, i64, i64, i64, p, p, i64, i64, i, i, p, i64, p, p, p, sz, p]
L.llmint8_gated_backward.argtypes = [p, i64, i64, i64, p, i64, p, p, i64, p, p, i, i, p, i64, p, p,
                                     i64, p, sz, p]
for n in ("matmul", "matmul_backward", "gated", "gated_backward"):
    f = getattr(L, "llmint8_%s_workspace_size" % n)
    f.argtypes, f.restype = [i64, i64, i64], sz
A, B, MIS, N0, BIG = 0x100000, 0x200000, 0x300008, None, 1 << 50
res = {}
def ref(s):
    return C.byref(s) if s is not None else None
def saved(data=A, ld=64, scales=N0, lds=2):
    return Saved(data, ld, scales, lds)
Q = lambda **k: saved(**{"ld": 64, "scales": B, **k})
def pack(name, X=A, M=4, K=64, ldx=64, dt=0, out=0):
    out = Q() if out == 0 else out
    res[name] = L.llmint8_checkpoint_pack(X, M, K, ldx, dt, ref(out), None)
def unpack(name, inp=0, M=4, K=64, dt=0, X=A, ldx=64):
    inp = Q() if inp == 0 else inp
    res[name] = L.llmint8_checkpoint_unpack(ref(inp), M, K, dt, X, ldx, None)
def mm(name, X=A, M=300, K=64, ldx=64, W=A, ldw=64, N=64, dt=0, Y=B, ldy=64, size=C.sizeof(Opts),
       act=0, bias=N0, R=N0, ldr=64, Z=N0, ldz=64, ws=A, wsb=BIG):
    o = Opts(size, act, bias, R, ldr, Z, ldz)
    res[name] = L.llmint8_matmul(X, M, K, ldx, W, ldw, N, dt, Y, ldy, C.byref(o), ws, wsb, None)
def mb(name, dY=A, M=300, N=64, lddy=64, X=0, K=64, W=A, ldw=64, Z=A, ldz=64, act=4, dt=0, dX=B,
       lddx=64, dW=B, lddw=64, db=N0, ws=A, wsb=BIG):
    X = saved() if X == 0 else X
    res[name] = L.llmint8_matmul_backward(dY, M, N, lddy, ref(X), K, W, ldw, Z, ldz, act, dt, dX,
                                          lddx, dW, lddw, db, ws, wsb, None)
def gt(name, X=A, M=300, K=64, ldx=64, Wg=A, Wu=A, ldw=64, N=64, act=4, dt=0, H=B, ldh=64, G=N0,
       U=N0, ws=A, wsb=BIG):
    res[name] = L.llmint8_gated(X, M, K, ldx, Wg, Wu, ldw, N, act, dt, H, ldh, ref(G), ref(U), ws,
                                wsb, None)
def gb(name, dH=A, M=300, N=64, lddh=64, X=0, K=64, Wg=A, Wu=A, ldw=64, G=0, U=0, act=4, dt=0,
       dX=B, lddx=64, dWg=B, dWu=B, lddw=64, ws=A, wsb=BIG):
    X, G, U = (saved() if t == 0 else t for t in (X, G, U))
    res[name] = L.llmint8_gated_backward(dH, M, N, lddh, ref(X), K, Wg, Wu, ldw, ref(G), ref(U),
                                         act, dt, dX, lddx, dWg, dWu, lddw, ws, wsb, None)
pack("pack_null_X", X=N0); pack("pack_M0", M=0); pack("pack_K0", K=0); pack("pack_ld", ldx=56)
pack("pack_dtype", dt=2); pack("pack_null_out", out=None); pack("pack_no_scales", out=saved())
pack("pack_null_codes", out=Q(data=N0)); pack("pack_ldc_short", out=Q(ld=48))
pack("pack_lds_short", out=Q(lds=1)); pack("pack_mis_X", X=MIS); pack("pack_K_not_mult8", K=60)
pack("pack_ldx_not_mult8", ldx=68); pack("pack_ldc_not_mult16", out=Q(ld=72))
pack("pack_mis_codes", out=Q(data=MIS))
unpack("unpack_null", inp=None); unpack("unpack_no_scales", inp=saved()); unpack("unpack_null_X", X=N0)
unpack("unpack_mis", X=MIS); unpack("unpack_ld", ldx=32); unpack("unpack_neg", M=-1)
mm("mm_null_X", X=N0); mm("mm_null_W", W=N0); mm("mm_null_Y", Y=N0); mm("mm_M0", M=0)
mm("mm_N0", N=0); mm("mm_K0", K=0); mm("mm_dtype", dt=-1); mm("mm_act", act=5)
mm("mm_act_neg", act=-1); mm("mm_struct", size=8); mm("mm_ldx", ldx=56); mm("mm_ldw", ldw=56)
mm("mm_ldy", ldy=56); mm("mm_ldr", R=A, ldr=56); mm("mm_ldz", Z=A, ldz=56)
mm("mm_ld_huge", ldx=1 << 21); mm("mm_M_huge", M=1 << 30)
mm("mm_K_not_mult8", K=60); mm("mm_N_not_mult8", N=60); mm("mm_ldw_not_mult8", ldw=68)
mm("mm_mis_X", X=MIS); mm("mm_mis_W", W=MIS); mm("mm_mis_bias", bias=MIS); mm("mm_mis_R", R=MIS)
mm("mm_mis_Z", Z=MIS); mm("mm_mis_Y", Y=MIS)
mm("mm_ws_null", M=64, K=11008, ldx=11008, ws=N0); mm("mm_ws_small", M=64, K=11008, ldx=11008, wsb=16)
mm("mm_ws_mis", M=64, K=11008, ldx=11008, ws=MIS)
mb("mb_null_dY", dY=N0); mb("mb_no_output", dX=N0, dW=N0); mb("mb_null_X", X=None)
mb("mb_null_W", W=N0); mb("mb_null_Z", Z=N0); mb("mb_act", act=9); mb("mb_dtype", dt=3)
mb("mb_M0", M=0); mb("mb_lddx", lddx=56); mb("mb_lddw", lddw=56); mb("mb_X_ld", X=saved(ld=56))
mb("mb_X_lds", X=Q(lds=1)); mb("mb_X_ldc", X=Q(ld=72)); mb("mb_mis_dX", dX=MIS)
mb("mb_mis_db", db=MIS); mb("mb_N_not_mult8", N=60); mb("mb_ws_null", ws=N0); mb("mb_ws_small", wsb=64)
gt("gt_null_Wu", Wu=N0); gt("gt_null_H", H=N0); gt("gt_G_alone", G=saved()); gt("gt_U_alone", U=saved())
gt("gt_mixed", G=saved(), U=Q()); gt("gt_G_null_data", G=saved(data=N0), U=saved())
gt("gt_ld_differ", G=saved(), U=saved(ld=72)); gt("gt_lds_differ", G=Q(), U=Q(lds=3))
gt("gt_act", act=7); gt("gt_M0", M=0); gt("gt_ldw", ldw=8); gt("gt_mis_Wg", Wg=MIS)
gt("gt_G_mis", G=saved(data=MIS), U=saved()); gt("gt_K_not_mult8", K=12, ldx=64)
gt("gt_ws_null", M=64, K=11008, ldx=11008, ws=N0)
gb("gb_null_dH", dH=N0); gb("gb_null_G", G=None); gb("gb_null_U", U=None); gb("gb_mixed", U=Q())
gb("gb_dWg_alone", dWu=N0); gb("gb_no_output", dX=N0, dWg=N0, dWu=N0); gb("gb_null_X", X=None)
gb("gb_null_Wg", Wg=N0); gb("gb_M0", M=0); gb("gb_lddw", lddw=56); gb("gb_mis_dX", dX=MIS)
gb("gb_ws_null", ws=N0); gb("gb_ws_small", wsb=1024); gb("gb_dtype", dt=2)
W = lambda n, *a: getattr(L, "llmint8_%s_workspace_size" % n)(*a)
res["q_mm"] = W("matmul", 64, 11008, 64); res["q_mm_bad"] = W("matmul", 64, 60, 64)
res["q_mm_large"] = W("matmul", 8192, 8192, 28672)
res["q_mb"] = W("matmul_backward", 300, 64, 64); res["q_mb_bad"] = W("matmul_backward", 0, 64, 64)
res["q_gt_bad"] = W("gated", 4, 64, -8)
res["q_gb"] = W("gated_backward", 2048, 4096, 11008); res["q_gb_bad"] = W("gated_backward", 4, 64, 12)
print(json.dumps(res))
"""

ARG = """pack_null_X pack_M0 pack_K0 pack_ld pack_dtype pack_null_out pack_no_scales pack_null_codes
pack_ldc_short pack_lds_short unpack_null unpack_no_scales unpack_null_X unpack_ld unpack_neg
mm_null_X mm_null_W mm_null_Y mm_M0 mm_N0 mm_K0 mm_dtype mm_act mm_act_neg mm_struct mm_ldx mm_ldw
mm_ldy mm_ldr mm_ldz mm_ld_huge mm_M_huge mb_null_dY mb_no_output mb_null_X mb_null_W mb_null_Z
mb_act mb_dtype mb_M0 mb_lddx mb_lddw mb_X_ld mb_X_lds gt_null_Wu gt_null_H gt_G_alone gt_U_alone
gt_mixed gt_G_null_data gt_ld_differ gt_lds_differ gt_act gt_M0 gt_ldw gb_null_dH gb_null_G
gb_null_U gb_mixed gb_dWg_alone gb_no_output gb_null_X gb_null_Wg gb_M0 gb_lddw gb_dtype""".split()
UNSUPPORTED = """pack_mis_X pack_K_not_mult8 pack_ldx_not_mult8 pack_ldc_not_mult16 pack_mis_codes
unpack_mis mm_K_not_mult8 mm_N_not_mult8 mm_ldw_not_mult8 mm_mis_X mm_mis_W mm_mis_bias mm_mis_R
mm_mis_Z mm_mis_Y mm_ws_mis mb_X_ldc mb_mis_dX mb_mis_db mb_N_not_mult8 gt_mis_Wg gt_G_mis
gt_K_not_mult8 gb_mis_dX""".split()
WORKSPACE = "mm_ws_null mm_ws_small mb_ws_null mb_ws_small gt_ws_null gb_ws_null gb_ws_small".split()


def test_refusals_before_any_hip_call():
    env = dict(os.environ, HIP_VISIBLE_DEVICES="-1", ROCR_VISIBLE_DEVICES="-1",
               CUDA_VISIBLE_DEVICES="-1")
    out = subprocess.run([sys.executable, "-c", CHILD, LIB], capture_output=True, text=True,
                         env=env, timeout=120)
    assert out.returncode == 0, out.stderr
    res = json.loads(out.stdout.strip().splitlines()[-1])
    want = {**{n: 1 for n in ARG}, **{n: 2 for n in UNSUPPORTED}, **{n: 4 for n in WORKSPACE}}
    assert {n: res[n] for n in want} == want
    assert {n for n in res if not n.startswith("q_")} == set(want)
    # partial sums of a split reduction: a whole number of [M x N] fp32 planes
    assert res["q_mm"] > 0 and res["q_mm"] % (64 * 64 * 4) == 0
    assert res["q_mm_large"] == 0 and res["q_mm_bad"] == 0 and res["q_mb_bad"] == 0
    assert res["q_gt_bad"] == 0 and res["q_gb_bad"] == 0
    # dZ in 16 bits and X expanded to 16 bits; dG, dU and X
    assert res["q_mb"] >= 300 * 64 * 2 * 2
    assert res["q_gb"] >= 2048 * 11008 * 2 * 2 + 2048 * 4096 * 2


def test_binding_refuses_before_the_library():
    import bit_quantized_matmul_col_amd as lm
    X = torch.zeros((4, 64), dtype=torch.float16)
    for call in (lambda: lm.llmint8_matmul(X, X.t()), lambda: lm.llmint8_gated(X, X, X),
                 lambda: lm.llmint8_checkpoint_pack(X), lambda: lm.llmint8_matmul_backward(X, X, X),
                 lambda: lm.llmint8_gated_backward(X, X, X, X, X, X),
                 lambda: lm.llmint8_checkpoint_unpack(
                     lm.Checkpoint(torch.zeros((4, 64), dtype=torch.int8),
                                   torch.zeros((4, 2), dtype=torch.uint8)))):
        with pytest.raises(ValueError, match="GPU"):
            call()
    for bad in (X.float(), X.double(), X.to(torch.int16)):
        with pytest.raises(TypeError):
            lm.llmint8_matmul(bad, bad)
        with pytest.raises(TypeError):
            lm.llmint8_checkpoint_pack(bad)
    with pytest.raises(TypeError):
        lm.llmint8_matmul([1.0], X)
    with pytest.raises(TypeError):
        lm.llmint8_checkpoint_unpack(lm.Checkpoint(X, X), torch.float32)
    assert set(fo.ACTS) == set(lm._ACTIVATIONS)


@pytest.mark.parametrize("name", fo.ACTS)
def test_definitions_against_differences(name):
    """act' against central differences of act, away from relu's kink: the quotient's error is
    h^2 / 6 of the third derivative (below 2 for these functions) and 1e-16 / h of rounding."""
    z = torch.linspace(-9, 9, 1801, dtype=torch.float64) + 0.0031
    h = 1e-5
    d = (fo.act(name, z + h) - fo.act(name, z - h)) / (2 * h)
    assert float((d - fo.act_grad(name, z)).abs().max()) < 2 * h * h / 6 + 9e-16 / h * 4


def test_definition_of_the_gated_gradient_against_differences():
    g = torch.Generator().manual_seed(3)
    r = lambda *s: torch.randn(s, generator=g, dtype=torch.float64)
    X, Wg, Wu, D = r(3, 8), r(8, 16), r(8, 16), r(3, 16)
    G, U = X @ Wg, X @ Wu
    grads = [t for t, _ in fo.gated_backward(D, X, Wg, Wu, G, U, "gelu", torch.float16)]
    loss = lambda x, a, b: (D * fo.act("gelu", x @ a) * (x @ b)).sum()
    at, h = [X, Wg, Wu], 1e-5
    for i, grad in enumerate(grads):
        V = r(*at[i].shape)
        up, down = list(at), list(at)
        up[i], down[i] = at[i] + h * V, at[i] - h * V
        d = float((loss(*up) - loss(*down)) / (2 * h))
        assert abs(d - float((grad * V).sum())) < 1e-6 * max(1.0, abs(d))


def test_definition_of_the_checkpoint():
    """Worked values: a block whose largest entry is 12 has the scale 2^(3 - 6) = 1/8."""
    x = torch.zeros((1, 40), dtype=torch.float64)
    x[0, :6] = torch.tensor([12.0, -0.1, 0.0625, 0.1875, -12.0, 3.3])
    x[0, 32] = 2.0 ** -130
    codes, byte = fo.pack(x)
    assert byte.tolist() == [[127 - 3, 0]]
    assert codes[0, :6].tolist() == [96, -1, 0, 2, -96, 26]  # ties at 0.5 and 1.5 to even
    assert codes[0, 32].item() == 0  # 2^-130 is an eighth of the smallest scale 2^-127
    v = fo.unpack(codes, byte)
    assert v[0, :6].tolist() == [12.0, -0.125, 0.0, 0.25, -12.0, 3.25]
    for dt in (torch.float16, torch.bfloat16):
        assert torch.equal(v[:, :32].to(dt).double(), v[:, :32])
    x[0, 7] = 15.99  # rounds to 128 steps, clamped to 127
    codes, byte = fo.pack(x)
    assert codes[0, 7].item() == 127 and byte[0, 0].item() == 124
    x[0, 7] = float("nan")
    codes, byte = fo.pack(x)
    assert byte[0, 0].item() == 255 and not codes[0, :32].any() and byte[0, 1].item() == 0
    assert fo.unpack(codes, byte)[0, :32].isnan().all()
