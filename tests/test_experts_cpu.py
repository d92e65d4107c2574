"""The routed feed-forward operators and the block-scaled FP8 product without a GPU: every refusal
of the C calls (in a child process with the GPUs hidden, so that a wrongly accepted call
could not reach one), the workspace queries, the binding's own checks, and the 64-bit
definitions that the GPU tests use, against differences and against themselves."""
import json
import math
import os
import subprocess
import sys

import pytest
import torch

import experts_oracle as eo
import ffn_oracle as fo
import fp8_block_oracle as bo

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "bit_quantized_matmul_col_amd", "libllmint8.so")


@pytest.fixture(autouse=True)
def _library(built_library):
    return built_library


CHILD = r"""
import ctypes as C, json, sys
L = C.CDLL(sys.argv[1])
p, i64, i, sz, f = C.c_void_p, C.c_int64, C.c_int, C.c_size_t, C.c_float
class Opts(C.Structure):
    _fields_ = [("struct_size", sz), ("scores", i), ("renormalize", i), ("scale", f), ("groups", i),
                ("top_groups", i), ("group_best", i), ("bias", p)]
class Rows(C.Structure):
    _fields_ = [("offsets", p), ("order", p), ("places", p), ("E", i64), ("k", i64)]
L.llmint8_route.argtypes = [p, i64, i64, i64, i, i64, p, p, p, p]
L.llmint8_route_backward.argtypes = [p, p, i64, i64, i64, i, i64, p, p, p, i64, p]
L.llmint8_expert_plan.argtypes = [p, i64, i64, i64, p, p, p, p, sz, p]
L.llmint8_expert_plan_workspace_size.argtypes = [i64] * 3
L.llmint8_expert_plan_workspace_size.restype = sz
L.llmint8_experts_gated.argtypes = [p, i64, i64, i64, p, p, i64, i64, i64, p, p, i, i, p, i64, p, p,
                                    i64, p, sz, p]
L.llmint8_experts_gated_backward.argtypes = [p, i64, i64, i64, p, i64, i64, p, p, i64, i64, p, p,
    i64, p, p, i, i, p, i64, p, p, i64, i64, p, p, sz, p]
L.llmint8_experts_matmul.argtypes = [p, i64, i64, i64, p, i64, i64, i64, p, p, i64, i, p, i64, p, sz,
                                     p]
L.llmint8_experts_matmul_backward.argtypes = [p, i64, i64, i64, p, i64, i64, p, i64, i64, p, i, p,
    i64, p, i64, i64, p, sz, p]
L.llmint8_quantize_blockwise_fp8.argtypes = [p, i64, i64, i64, i, p, p, p]
L.llmint8_quantize_rowblock_fp8.argtypes = [p, i64, i64, i64, i, p, p, i64, p]
L.llmint8_linear_blockwise_fp8.argtypes = [p, i64, i64, i64, p, p, i64, i64, i, p, p, i64, p, sz, p]
L.llmint8_linear_blockwise_fp8_workspace_size.argtypes = [i64, i64, i64]
L.llmint8_linear_blockwise_fp8_workspace_size.restype = sz
for n in ("gated", "gated_backward", "matmul", "matmul_backward"):
    q = getattr(L, "llmint8_experts_%s_workspace_size" % n)
    q.argtypes, q.restype = [i64] * 5, sz
A, B, MIS, ODD, N0, BIG = 0x100000, 0x200000, 0x300008, 0x300001, None, 1 << 50
res = {}
def opts(size=C.sizeof(Opts), scores=0, renorm=0, groups=1, top=1, best=1, bias=N0):
    return Opts(size, scores, renorm, 1.0, groups, top, best, bias)
def route(name, x=A, M=4, E=16, ld=16, dt=0, k=2, ids=B, w=B, **o):
    res["r_" + name] = L.llmint8_route(x, M, E, ld, dt, k, C.byref(opts(**o)), ids, w, None)
def rback(name, d=A, x=A, M=4, E=16, ld=16, dt=0, k=2, ids=A, dx=B, ldd=16, **o):
    res["rb_" + name] = L.llmint8_route_backward(d, x, M, E, ld, dt, k, ids, C.byref(opts(**o)), dx,
                                                 ldd, None)
def plan(name, ids=A, M=4, k=2, E=16, offsets=B, order=B, places=B, ws=A, wsb=BIG):
    res["p_" + name] = L.llmint8_expert_plan(ids, M, k, E, offsets, order, places, ws, wsb, None)
def rows(E=4, k=2, offsets=A, order=A, places=A):
    return Rows(offsets, order, places, E, k)
def ref(r):
    return C.byref(r) if r is not None else None
def gt(name, X=A, M=300, K=64, ldx=64, Wg=A, Wu=A, ldw=64, sw=4096, N=64, r=0, w=N0, act=4, dt=0, H=B,
       ldh=64, G=N0, U=N0, ldz=64, ws=A, wsb=BIG):
    r = rows() if r == 0 else r
    res["g_" + name] = L.llmint8_experts_gated(X, M, K, ldx, Wg, Wu, ldw, sw, N, ref(r), w, act, dt,
                                               H, ldh, G, U, ldz, ws, wsb, None)
def gb(name, dH=A, M=300, N=64, lddh=64, X=A, K=64, ldx=64, Wg=A, Wu=A, ldw=64, sw=4096, G=A, U=A,
       ldz=64, r=0, w=N0, act=4, dt=0, dX=B, lddx=64, dWg=B, dWu=B, lddw=64, sdw=4096, dw=N0, ws=A,
       wsb=BIG):
    r = rows() if r == 0 else r
    res["gb_" + name] = L.llmint8_experts_gated_backward(dH, M, N, lddh, X, K, ldx, Wg, Wu, ldw, sw,
        G, U, ldz, ref(r), w, act, dt, dX, lddx, dWg, dWu, lddw, sdw, dw, ws, wsb, None)
def mm(name, H=A, M=300, N=64, ldh=64, Wd=A, ldw=64, sw=4096, K=64, r=0, R=N0, ldr=64, dt=0, Y=B,
       ldy=64, ws=A, wsb=BIG):
    r = rows() if r == 0 else r
    res["m_" + name] = L.llmint8_experts_matmul(H, M, N, ldh, Wd, ldw, sw, K, ref(r), R, ldr, dt, Y,
                                                ldy, ws, wsb, None)
def mb(name, dY=A, M=300, K=64, lddy=64, H=A, N=64, ldh=64, Wd=A, ldw=64, sw=4096, r=0, dt=0, dH=B,
       lddh=64, dWd=B, lddw=64, sdw=4096, ws=A, wsb=BIG):
    r = rows() if r == 0 else r
    res["mb_" + name] = L.llmint8_experts_matmul_backward(dY, M, K, lddy, H, N, ldh, Wd, ldw, sw,
        ref(r), dt, dH, lddh, dWd, lddw, sdw, ws, wsb, None)
def qw(name, W=A, K=64, N=64, ldw=64, dt=0, q=B, s=B):
    res["qw_" + name] = L.llmint8_quantize_blockwise_fp8(W, K, N, ldw, dt, q, s, None)
def qx(name, X=A, M=4, K=64, ldx=64, dt=0, q=B, s=B, lds=4):
    res["qx_" + name] = L.llmint8_quantize_rowblock_fp8(X, M, K, ldx, dt, q, s, lds, None)
def fl(name, X=A, M=300, K=64, ldx=64, q=A, s=A, lds=1, N=64, dt=0, b=N0, Y=B, ldy=64, ws=A, wsb=BIG):
    res["f_" + name] = L.llmint8_linear_blockwise_fp8(X, M, K, ldx, q, s, lds, N, dt, b, Y, ldy, ws,
                                                      wsb, None)
route("null_x", x=N0); route("null_ids", ids=N0); route("null_w", w=N0); route("M0", M=0)
route("E0", E=0); route("E_large", E=1025, ld=1025); route("k0", k=0); route("k_over_E", k=17)
route("k_large", E=512, ld=512, k=65); route("ld", ld=15); route("ld_huge", ld=1 << 21)
route("dt", dt=3); route("dt_neg", dt=-1); route("struct", size=8); route("scores", scores=2)
route("renorm", renorm=2); route("groups0", groups=0); route("groups_uneven", groups=3)
route("groups_many", E=130, ld=130, groups=65); route("top0", top=0); route("top_many", top=2)
route("best0", best=0); route("best3", best=3); route("pairs", M=1 << 24); route("M_neg", M=-4)
route("odd_x", x=ODD); route("odd_x32", x=A + 2, dt=2); route("odd_ids", ids=A + 2)
route("odd_w", w=A + 2); route("odd_bias", bias=A + 1)
rback("null_d", d=N0); rback("null_x", x=N0); rback("null_ids", ids=N0); rback("null_dx", dx=N0)
rback("ldd", ldd=15); rback("ldd_huge", ldd=1 << 21); rback("k0", k=0); rback("dt", dt=7)
rback("scores", scores=-1); rback("odd_dx", dx=ODD); rback("odd_dx32", dx=A + 2, dt=2)
rback("odd_d", d=A + 2); rback("struct", size=0)
plan("null_ids", ids=N0); plan("null_offsets", offsets=N0); plan("null_order", order=N0)
plan("null_places", places=N0); plan("M0", M=0); plan("k0", k=0); plan("k65", k=65, E=100)
plan("k_over_E", k=17); plan("E0", E=0); plan("E_large", E=1025); plan("pairs", M=1 << 24)
plan("odd_ids", ids=A + 2); plan("odd_order", order=A + 2); plan("odd_places", places=A + 1)
plan("odd_offsets", offsets=A + 3); plan("k_huge", k=1 << 62, M=8)
plan("ws_null", M=70000, ws=N0); plan("ws_small", M=70000, wsb=64); plan("ws_mis", M=70000, ws=MIS)
def plan_faults(f):
    f("no_plan", r=None); f("E0", r=rows(E=0)); f("E_large", r=rows(E=1025)); f("k0", r=rows(k=0))
    f("k_over_E", r=rows(k=5)); f("null_offsets", r=rows(offsets=N0))
    f("null_order", r=rows(order=N0)); f("null_places", r=rows(places=N0))
    f("odd_places", r=rows(places=A + 2)); f("M0", M=0); f("pairs", M=1 << 24); f("dt", dt=2)
    f("K60", K=60); f("N60", N=60); f("ldw", ldw=56); f("sw_neg", sw=-8); f("sw_huge", sw=1 << 40)
    f("sw_mis", sw=4100)
for f in (gt, gb, mm, mb):
    plan_faults(f)
gt("null_X", X=N0); gt("null_Wg", Wg=N0); gt("null_Wu", Wu=N0); gt("null_H", H=N0); gt("G_alone", G=B)
gt("U_alone", U=B); gt("ldx", ldx=56); gt("ldh", ldh=56); gt("ldz", G=B, U=B, ldz=56)
gt("act", act=5); gt("mis_X", X=MIS); gt("mis_H", H=MIS); gt("mis_G", G=MIS, U=B)
gt("odd_w", w=A + 2); gt("ldx_mis", ldx=68); gt("span", M=4096, ldx=(1 << 19)); gt("ld_huge", ldx=1 << 21)
for f in (gb, mm, mb):
    f("ws_mis", ws=MIS)
gt("ws_mis", M=1 << 24, K=128, ldx=128, r=rows(E=2, k=1), ws=MIS); gt("ws_small", M=1 << 24, K=128, ldx=128, r=rows(E=2, k=1), wsb=64); gt("ws_null", M=1 << 24, K=128, ldx=128, r=rows(E=2, k=1), ws=N0)
gb("null_dH", dH=N0); gb("null_G", G=N0); gb("null_U", U=N0); gb("null_X", X=N0)
gb("null_Wg", Wg=N0); gb("null_Wu", Wu=N0); gb("dWg_alone", dWu=N0); gb("dWu_alone", dWg=N0)
gb("no_output", dX=N0, dWg=N0, dWu=N0); gb("lddh", lddh=56); gb("ldz", ldz=56); gb("lddx", lddx=56)
gb("lddw", lddw=56); gb("sdw_overlap", sdw=4088); gb("act", act=-1); gb("mis_dX", dX=MIS)
gb("mis_dWg", dWg=MIS); gb("odd_dw", dw=A + 2); gb("ws_null", ws=N0); gb("ws_small", wsb=1024)
mm("null_H", H=N0); mm("null_Wd", Wd=N0); mm("null_Y", Y=N0); mm("ldh", ldh=56); mm("ldy", ldy=56)
mm("ldr", R=A, ldr=56); mm("mis_R", R=MIS); mm("mis_Y", Y=MIS); mm("ws_null", ws=N0)
mm("ws_small", wsb=64)
mb("null_dY", dY=N0); mb("null_H", H=N0); mb("null_Wd", Wd=N0); mb("no_output", dH=N0, dWd=N0)
mb("lddy", lddy=56); mb("ldh", ldh=56); mb("lddh", lddh=56); mb("lddw", lddw=56)
mb("sdw_overlap", sdw=0); mb("mis_dH", dH=MIS); mb("mis_dWd", dWd=MIS); mb("ws_null", ws=N0)
mb("ws_small", wsb=64)
qw("null_W", W=N0); qw("null_q", q=N0); qw("null_s", s=N0); qw("K0", K=0); qw("N0", N=0)
qw("K_large", K=131088); qw("ldw", ldw=56); qw("dt", dt=2); qw("K24", K=24); qw("N60", N=60)
qw("mis_W", W=MIS); qw("mis_q", q=MIS)
qx("null_X", X=N0); qx("null_q", q=N0); qx("null_s", s=N0); qx("M0", M=0); qx("K0", K=0)
qx("lds", lds=3); qx("lds_huge", lds=1 << 21); qx("ldx", ldx=56); qx("dt", dt=-1); qx("K24", K=24)
qx("mis_X", X=MIS); qx("mis_q", q=MIS)
fl("null_X", X=N0); fl("null_q", q=N0); fl("null_s", s=N0); fl("null_Y", Y=N0); fl("M0", M=0)
fl("N0", N=0); fl("K0", K=0); fl("K_large", K=131088, ldx=131088, lds=2000); fl("lds", K=256, ldx=256)
fl("ldx", ldx=56); fl("ldy", ldy=56); fl("dt", dt=2); fl("K24", K=24); fl("N60", N=60)
fl("mis_X", X=MIS); fl("mis_q", q=MIS); fl("mis_b", b=MIS); fl("mis_Y", Y=MIS); fl("ws_null", ws=N0)
fl("ws_small", wsb=64); fl("ws_mis", ws=MIS); fl("M_huge", M=(1 << 30) - 1, N=4096, ldy=4096)
W = lambda n, *a: getattr(L, "llmint8_experts_%s_workspace_size" % n)(*a)
q = {}
q["gated_few"] = W("gated", 1, 64, 64, 8, 2)
q["gated_copy"] = W("gated", 1 << 20, 2048, 64, 2, 1)
q["gated_back"] = W("gated_backward", 300, 64, 128, 4, 2)
q["matmul"] = W("matmul", 3000, 64, 128, 4, 2)
q["matmul_back"] = W("matmul_backward", 300, 64, 128, 4, 2)
q["bad"] = [W(n, *a) for n in ("gated", "gated_backward", "matmul", "matmul_backward")
            for a in ((0, 64, 64, 4, 2), (4, 60, 64, 4, 2), (4, 64, 64, 4, 5), (4, 64, 64, 1025, 5),
                      (1 << 24, 64, 64, 4, 2), (4, 64, -64, 4, 2))]
P = L.llmint8_expert_plan_workspace_size
q["plan"] = [P(1, 8, 64), P(8192, 8, 256), P(1 << 21, 8, 256), P(2048, 8, 256), P(70000, 2, 1025), P(1 << 24, 2, 8)]
F = L.llmint8_linear_blockwise_fp8_workspace_size
q["fp8"] = [F(1, 4096, 4096), F(300, 4096, 4096), F(1, 24, 64), F(0, 64, 64), F(4, 131088, 64)]
print(json.dumps([res, q]))
"""

PLAN_ARG = """no_plan E0 E_large k0 k_over_E null_offsets null_order null_places M0 pairs dt ldw
sw_neg sw_huge""".split()
PLAN_UNSUPPORTED = "odd_places K60 N60 sw_mis ws_mis".split()
ARG = [f"{c}_{n}" for c in ("g", "gb", "m", "mb") for n in PLAN_ARG] + """
r_null_x r_null_ids r_null_w r_M0 r_E0 r_E_large r_k0 r_k_over_E r_k_large r_ld r_ld_huge r_dt
r_dt_neg r_struct r_scores r_renorm r_groups0 r_groups_uneven r_groups_many r_top0 r_top_many r_best0
r_best3 r_pairs r_M_neg rb_null_d rb_null_x rb_null_ids rb_null_dx rb_ldd rb_ldd_huge rb_k0 rb_dt
rb_scores rb_struct p_null_ids p_null_offsets p_null_order p_null_places p_M0 p_k0 p_k65 p_k_over_E
p_E0 p_E_large p_pairs p_k_huge g_null_X g_null_Wg g_null_Wu g_null_H g_G_alone g_U_alone g_ldx g_ldh
g_ldz g_act g_ld_huge gb_null_dH gb_null_G gb_null_U gb_null_X gb_null_Wg gb_null_Wu gb_dWg_alone
gb_dWu_alone gb_no_output gb_lddh gb_ldz gb_lddx gb_lddw gb_sdw_overlap gb_act m_null_H m_null_Wd
m_null_Y m_ldh m_ldy m_ldr mb_null_dY mb_null_H mb_null_Wd mb_no_output mb_lddy mb_ldh mb_lddh
mb_lddw mb_sdw_overlap qw_null_W qw_null_q qw_null_s qw_K0 qw_N0 qw_K_large qw_ldw qw_dt qx_null_X
qx_null_q qx_null_s qx_M0 qx_K0 qx_lds qx_lds_huge qx_ldx qx_dt f_null_X f_null_q f_null_s f_null_Y
f_M0 f_N0 f_K0 f_K_large f_lds f_ldx f_ldy f_dt""".split()
UNSUPPORTED = [f"{c}_{n}" for c in ("g", "gb", "m", "mb") for n in PLAN_UNSUPPORTED] + """
r_odd_x r_odd_x32 r_odd_ids r_odd_w r_odd_bias rb_odd_dx rb_odd_dx32 rb_odd_d p_odd_ids p_odd_order
p_odd_places p_odd_offsets p_ws_mis g_mis_X g_mis_H g_mis_G g_odd_w g_ldx_mis g_span gb_mis_dX gb_mis_dWg
gb_odd_dw m_mis_R m_mis_Y mb_mis_dH mb_mis_dWd qw_K24 qw_N60 qw_mis_W qw_mis_q qx_K24 qx_mis_X
qx_mis_q f_K24 f_N60 f_mis_X f_mis_q f_mis_b f_mis_Y f_ws_mis f_M_huge""".split()
WORKSPACE = """g_ws_small g_ws_null gb_ws_null gb_ws_small m_ws_null m_ws_small mb_ws_null
mb_ws_small p_ws_null p_ws_small f_ws_null f_ws_small""".split()


def test_refusals_before_any_hip_call():
    env = dict(os.environ, HIP_VISIBLE_DEVICES="-1", ROCR_VISIBLE_DEVICES="-1",
               CUDA_VISIBLE_DEVICES="-1")
    out = subprocess.run([sys.executable, "-c", CHILD, LIB], capture_output=True, text=True,
                         env=env, timeout=120)
    assert out.returncode == 0, out.stderr
    res, q = json.loads(out.stdout.strip().splitlines()[-1])
    want = {**{n: 1 for n in ARG}, **{n: 2 for n in UNSUPPORTED}, **{n: 4 for n in WORKSPACE}}
    assert {n: v for n, v in res.items() if want.get(n) != v} == {}
    assert set(res) == set(want)
    # a token's experts: partial sums of both products; X in the experts' order
    assert q["gated_few"] % (2 * 64 * 4) == 0
    assert (1 << 20) * 2048 * 2 <= q["gated_copy"] < (1 << 20) * 2048 * 2 + (1 << 20)
    # dG, dU, X and dX's rows in fp32; the rows of Y and of dY
    assert q["gated_back"] >= 600 * (2 * 128 * 2 + 64 * 2 + 64 * 4)
    assert q["matmul"] >= 6000 * 64 * 2 and q["matmul_back"] >= 600 * 64 * 2
    assert not any(q["bad"])
    # counts of 64 and of 256 chunks
    assert q["plan"] == [0, 64 * 257 * 4, 256 * 257 * 4, 0, 0, 0]
    assert q["fp8"][0] == 0 and q["fp8"][1] >= 300 * 4096 and not any(q["fp8"][2:])


def test_binding_refuses_before_the_library():
    import bit_quantized_matmul_col_amd as lm
    h, f = torch.zeros((4, 64), dtype=torch.float16), torch.zeros((4, 2))
    ids = torch.zeros((4, 2), dtype=torch.int32)
    W = torch.zeros((8, 64, 64), dtype=torch.float16)
    plan = lm.ExpertPlan(torch.zeros(9, dtype=torch.int32), torch.zeros(8, dtype=torch.int32), ids)
    q, s = torch.zeros((64, 64), dtype=torch.uint8), torch.zeros((1, 1), dtype=torch.uint8)
    for call in (lambda: lm.llmint8_route(h, 2), lambda: lm.llmint8_route_backward(f, h, ids),
                 lambda: lm.llmint8_expert_plan(ids, 8),
                 lambda: lm.llmint8_experts_gated(h, W, W, plan),
                 lambda: lm.llmint8_experts_matmul(h, W, plan),
                 lambda: lm.llmint8_experts_gated_backward(h, h, W, W, h, h, plan),
                 lambda: lm.llmint8_experts_matmul_backward(h, h, W, plan),
                 lambda: lm.llmint8_quantize_blockwise_fp8(h),
                 lambda: lm.llmint8_quantize_rowblock_fp8(h),
                 lambda: lm.llmint8_linear_blockwise_fp8(h, q, s)):
        with pytest.raises(ValueError, match="GPU"):
            call()
    with pytest.raises(TypeError):
        lm.llmint8_route(h.double(), 2)
    with pytest.raises(TypeError):
        lm.llmint8_route([1.0], 2)
    with pytest.raises(TypeError):
        lm.llmint8_expert_plan(ids.long(), 8)
    for call in (lm.llmint8_quantize_blockwise_fp8, lm.llmint8_quantize_rowblock_fp8):
        with pytest.raises(TypeError):
            call(h.float())


# ---- definitions ------------------------------------------------------------------------

def directional(f, at, grads, seed, h=1e-5, tol=1e-6):
    """The gradients against central differences along a random direction of each input."""
    g = torch.Generator().manual_seed(seed)
    for i, grad in enumerate(grads):
        V = torch.randn(at[i].shape, generator=g, dtype=torch.float64)
        up, down = list(at), list(at)
        up[i], down[i] = at[i] + h * V, at[i] - h * V
        d = float((f(*up) - f(*down)) / (2 * h))
        assert abs(d - float((grad * V).sum())) < tol * max(1.0, abs(d)), i


@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_definition_of_the_router_gradient_against_differences(scores, renorm):
    g = torch.Generator().manual_seed(1)
    x = torch.randn((5, 12), generator=g, dtype=torch.float64)
    ids = eo.choose(x, 4, scores)
    ids[2, 3] = -1
    D = torch.randn((5, 4), generator=g, dtype=torch.float64)
    dx, _ = eo.route_backward(D, x, ids, scores, renorm, 2.5)
    # (the bound's own arithmetic aside, mix works in 64 bits)
    directional(lambda x: (D * 2.5 * eo.mix(x, ids, scores, renorm)[0]).sum(), [x], [dx], 2)


def test_definition_of_the_choice():
    """Worked values: ties to the lower index, masked experts out, groups by their best two."""
    nan, inf = math.nan, math.inf
    x = torch.tensor([[1.0, 3, 3, 0], [-inf, nan, 2, -inf], [inf, 1, inf, 0], [-inf] * 4])
    assert eo.choose(x, 3).tolist() == [[1, 2, 0], [2, -1, -1], [0, 2, 1], [-1, -1, -1]]
    y = torch.tensor([[0.0, 4, 3, 3, 1, 1]])
    assert eo.choose(y, 2, groups=3, top_groups=1).tolist() == [[1, 0]]
    # softmax: the run of 3 and 3 holds more than that of 0 and 4 only by their sum, and does not
    assert eo.choose(y, 2, groups=3, top_groups=1, best=2).tolist() == [[1, 0]]
    assert eo.choose(y, 2, "sigmoid", groups=3, top_groups=1, best=2).tolist() == [[2, 3]]
    b = torch.tensor([0.0, 0, 0, 0, 9, 8])
    assert eo.choose(y, 3, "sigmoid", bias=b).tolist() == [[4, 5, 1]]
    w, _ = eo.mix(x, eo.choose(x, 3), "softmax", True)
    assert w[3].tolist() == [0, 0, 0] and w[1].tolist() == [1, 0, 0] and float(w[2, 2]) == 0
    assert torch.allclose(w[0], torch.softmax(torch.tensor([3.0, 3, 1], dtype=torch.float64), 0))


def test_definition_of_the_experts_gradients_against_differences():
    """The whole block: gated, second product, residual."""
    g = torch.Generator().manual_seed(3)
    r = lambda *s: torch.randn(s, generator=g, dtype=torch.float64)  # noqa: E731
    M, K, N, E, k = 6, 8, 16, 3, 2
    ids = torch.tensor([[0, 1], [2, 0], [-1, 1], [1, 2], [0, 2], [-1, -1]], dtype=torch.int32)
    p = eo.plan(ids, E)
    last = int(p[0][-1])
    X, Wg, Wu, Wd, w, D = r(M, K), r(E, K, N), r(E, K, N), r(E, N, K), r(M, k), r(M, K)
    f16 = torch.float16
    gated = lambda x, a, b, w: eo.gated(x, a, b, p, w, "gelu", f16)["H"][0]  # noqa: E731
    out = eo.gated(X, Wg, Wu, p, w, "gelu", f16)
    second = eo.matmul_backward(D, out["H"][0], Wd, p, f16)
    dH = second["dH"][0]
    back = eo.gated_backward(dH, X, Wg, Wu, out["G"][0], out["U"][0], p, w, "gelu", f16)
    assert not dH[last:].any()

    def loss(x, a, b, w, d):
        return (D * eo.matmul(gated(x, a, b, w), d, p, None, f16, False)[0]).sum()
    directional(loss, [X, Wg, Wu, w, Wd],
                [back["dX"][0], back["dWg"][0], back["dWu"][0], back["dw"][0], second["dWd"][0]], 4)
    assert not back["dX"][0][5].any() and not back["dw"][0][5].any()


def test_definition_of_the_block_codes():
    """Worked values: a block whose largest entry is 449 has the scale 2, one of 448 the scale 1."""
    x = torch.zeros((3, 256), dtype=torch.float64)
    x[0, :5] = torch.tensor([449.0, -2.0, 0.0, 34.0, 2.0 ** -9])  # 34 / 2 = 17: a tie of 16 and 18
    x[0, 128] = 448
    x[1, 3] = math.inf
    x[2, 0] = 2.0 ** -133
    q, byte = bo.rows(x)
    assert byte.tolist() == [[128, 127], [255, 0], [0, 0]]
    assert q[0, :5].tolist() == [0x76, 0xb8, 0, 0x58, 0]
    v = bo.values(q, bo.spread_rows(byte, 256))
    assert v[0, :5].tolist() == [448.0, -2.0, 0.0, 32.0, 0.0] and float(v[0, 128]) == 448
    assert v[1, :128].isnan().all() and not v[1, 128:].any()
    assert float(v[2, 0]) == 2.0 ** -133  # 2^-6 of the smallest scale
    t = bo.table("cpu")
    assert t[126] == 448 and t[1] == 2.0 ** -9 and t[8] == 2.0 ** -6 and t[127].isnan()
    # every value is its own code
    c = torch.arange(127)
    assert torch.equal(bo.encode(t[:127]), c) and torch.equal(bo.encode(-t[:127]), c + 128)
    w = torch.randn((200, 136), generator=torch.Generator().manual_seed(1), dtype=torch.float64)
    q, byte = bo.weights(w)
    v = bo.values(q, bo.spread_weights(byte, 136, 200))
    # a rounding of half a step, of 3 significant bits or of 2^-9 of the scale
    unit = torch.exp2((bo.spread_weights(byte, 136, 200) - 127).double())
    assert bool(((v - w.t()).abs() <= torch.maximum(w.t().abs() * 2.0 ** -4, unit * 2.0 ** -10)).all())


def test_oracle_sees_a_planted_mistake():
    """The bounds are tight enough to tell a wrong operator from a rounding: a dropped row, a
    weight of another choice, a block's scale off by one step."""
    g = torch.Generator().manual_seed(6)
    r = lambda *s: torch.randn(s, generator=g, dtype=torch.float64)  # noqa: E731
    M, K, N, E, k = 40, 64, 64, 4, 2
    ids = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(M)]).to(torch.int32)
    p = eo.plan(ids, E)
    X, Wg, Wu, w = r(M, K), 0.1 * r(E, K, N), 0.1 * r(E, K, N), torch.rand((M, k), generator=g)
    y, tol = eo.gated(X, Wg, Wu, p, w, "silu", torch.bfloat16)["H"]
    z, _ = eo.gated(X, Wg, Wu, p, w.flip(1), "silu", torch.bfloat16)["H"]
    assert float(((y - z).abs() > tol).double().mean()) > 0.8
    H, Wd = r(M * k, N), 0.1 * r(E, N, K)
    y, tol = eo.matmul(H, Wd, p, None, torch.bfloat16, True)
    H[3] = 0
    z, _ = eo.matmul(H, Wd, p, None, torch.bfloat16, True)
    token = int(p[1][3]) // k
    assert float(((y - z).abs() > tol)[token].double().mean()) > 0.8
    x, wt = r(8, 256).to(torch.bfloat16), 0.1 * r(256, 128)
    wq, sw = bo.weights(wt)
    y, tol = bo.linear(x, wq, sw, None, torch.bfloat16)
    sw[0, 1] += 1
    z, _ = bo.linear(x, wq, sw, None, torch.bfloat16)
    assert float(((y - z).abs() > tol).double().mean()) > 0.8
    assert set(fo.ACTS) >= {"silu", "gelu"}
