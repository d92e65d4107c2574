"""The 16-bit feed-forward operators on the GPU against their definitions in 64
bits (tests/ffn_oracle.py, which also derives the bounds): every operand order
and kernel variant, odd and ragged sizes, row strides with NaN between the rows,
canaries around the outputs, non-finite inputs, streams, repeatability and graph
replay."""
import sys

import pytest
import torch

import ffn_oracle as fo

pytestmark = pytest.mark.gpu

F16, BF16 = torch.float16, torch.bfloat16
PAD = 16  # columns between the end of a row and the next


@pytest.fixture(scope="module")
def lm():
    import bit_quantized_matmul_col_amd as lm
    lm.lib()
    return lm


def say(*a):
    print("case", *a, file=sys.stderr, flush=True)


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def rand(g, M, N, dtype, scale=1.0):
    return (torch.randn((M, N), generator=g, device="cuda") * scale).to(dtype)


def strided(t):
    """t with NaN in the gap between its rows."""
    M, N = t.shape
    big = torch.full((M, N + PAD), float("nan"), dtype=t.dtype, device=t.device)
    big[:, :N] = t
    return big[:, :N]


class Band:
    """An output [M, N] in the middle of a buffer whose other entries must not change."""

    def __init__(self, M, N, dtype, pad=PAD):
        self.big = torch.full((M + 16, N + pad), 77.0, dtype=dtype, device="cuda")
        self.t = self.big[8:8 + M, :N]

    def check(self):
        torch.cuda.synchronize()
        M, N = self.t.shape
        rest = self.big.clone()
        rest[8:8 + M, :N] = 77.0
        assert bool((rest == 77.0).all()), "wrote outside the output"


def near(got, want):
    y, tol = want
    d = (got.double() - y).abs()
    bad = ~(d <= tol)
    assert not bool(bad.any()), (
        f"{int(bad.sum())} of {bad.numel()} off; worst {float((d / tol)[bad].max()):.2f} times the "
        f"bound at {[int(i) for i in bad.nonzero()[0]]}")


# M, K, N: one row, odd rows, partial tiles and stages on every side; small-M, 128- and
# 256-row tiles; a long reduction over few tiles
SHAPES = [(1, 8, 8), (1, 1040, 520), (2, 4096, 1032), (7, 72, 24), (16, 256, 128), (17, 264, 136),
          (33, 1000, 72), (64, 2048, 264), (65, 64, 264), (129, 40, 1032), (300, 1040, 520),
          (300, 4104, 136), (1000, 96, 1096), (2049, 72, 4104),
          # few rows with 64- and 128-column blocks, whole and split; split 128- and
          # 256-tiles; 256-tiles with and without a tail of half tiles
          (5, 11008, 520), (3, 520, 28680), (1, 11008, 4096), (20, 4096, 11008), (40, 4104, 1032),
          (500, 2056, 1032), (1025, 8200, 2056), (2100, 2056, 4104), (1400, 4104, 4104),
          (2300, 1032, 8200),
          # few rows in groups of 16, 32 and 64 with blocks of 32, 64 and 128 columns, split
          # and whole
          (18, 4408, 5192), (70, 9304, 1880), (69, 264, 14080), (1, 4664, 4976), (465, 80, 520),
          (372, 10200, 168), (17, 7840, 2544), (42, 9496, 1640), (1, 10776, 1552),
          (55, 7264, 656), (167, 6880, 472), (310, 72, 776)]


@pytest.mark.parametrize("M,K,N", SHAPES)
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_matmul(lm, M, K, N, dtype):
    say("matmul", M, K, N, dtype)
    g = gen(M * 3 + K + N)
    X, W = rand(g, M, K, dtype), rand(g, K, N, dtype, 0.05)
    bias, R = rand(g, 1, N, dtype)[0], rand(g, M, N, dtype)
    name = fo.ACTS[(M + K + N) // 8 % 5]
    Y, Z = Band(M, N, dtype), Band(M, N, dtype)
    out = lm.llmint8_matmul(strided(X), strided(W), bias=bias, activation=name,
                            residual=strided(R), Y=Y.t, Z=Z.t)
    assert out is Y.t
    Y.check(), Z.check()
    want = fo.matmul(X.double(), W.double(), bias.double(), R.double(), name, dtype)
    near(Y.t, want[0])
    near(Z.t, want[1])
    # the plain product, contiguous, and twice the same
    a, b = lm.llmint8_matmul(X, W), lm.llmint8_matmul(X, W)
    assert torch.equal(a, b)
    near(a, fo.matmul(X.double(), W.double(), None, None, "none", dtype)[0])


def test_rows_more_than_2_gib_apart(lm):
    """Row strides of 2 MiB: byte offsets pass 31 and 32 bits, also those of the stages that
    the loop asks for past the end of the reduction."""
    pitch, n = 1 << 20, 72
    base = torch.empty((2200, pitch), dtype=BF16, device="cuda")
    g = gen(3)

    def wide(rows, column):
        v = base[:rows, column:column + n]
        v.copy_(rand(g, rows, n, BF16))
        return v

    for M, K in ((5, 2192), (400, 1104), (400, 2192)):
        say("wide strides, forward", M, K)
        X, W, Wu = rand(g, M, K, BF16, 0.05), wide(K, 0), wide(K, 512)
        near(lm.llmint8_matmul(X, W), fo.matmul(X.double(), W.double(), None, None, "none", BF16)[0])
        h, dh = fo.gated(X.double(), W.double(), Wu.double(), "silu", BF16)[0]
        near(lm.llmint8_gated(X, W, Wu), (h, dh))
    for M in (1103, 2200):
        say("wide strides, backward", M)
        dY, X, W = wide(M, 0), wide(M, 512), rand(g, n, n, BF16)
        dX, dW, _ = lm.llmint8_matmul_backward(dY, X, W)
        alone = lm.llmint8_matmul_backward(dY, X, W, need_dX=False)[1]
        wx = fo.product(dY.double(), W.double().t())
        ww = fo.product(X.double().t(), dY.double())
        near(dX, (wx[0], fo.stored(*wx, BF16)))
        near(dW, (ww[0], fo.stored(*ww, BF16)))
        near(alone, (ww[0], fo.stored(*ww, BF16)))


@pytest.mark.parametrize("name", fo.ACTS)
@pytest.mark.parametrize("M", [5, 200])
def test_matmul_activations(lm, name, M):
    say("matmul activation", name, M)
    g = gen(11)
    X, W = rand(g, M, 64, F16), rand(g, 64, 64, F16, 0.5)
    near(lm.llmint8_matmul(X, W, activation=name),
         fo.matmul(X.double(), W.double(), None, None, name, F16)[0])


@pytest.mark.parametrize("M,K,N", SHAPES)
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_gated(lm, M, K, N, dtype):
    say("gated", M, K, N, dtype)
    g = gen(M + K * 3 + N)
    X, Wg, Wu = rand(g, M, K, dtype), rand(g, K, N, dtype, 0.05), rand(g, K, N, dtype, 0.05)
    name = fo.ACTS[1 + (M + K + N) // 8 % 4]
    want, (G, dG), (U, dU) = fo.gated(X.double(), Wg.double(), Wu.double(), name, dtype)
    H = Band(M, N, dtype)
    h, g16, u16 = lm.llmint8_gated(strided(X), strided(Wg), strided(Wu), activation=name,
                                   save="full", H=H.t)
    H.check()
    near(h, want)
    near(g16, (G, fo.stored(G, dG, dtype)))
    near(u16, (U, fo.stored(U, dU, dtype)))
    assert torch.equal(lm.llmint8_gated(X, Wg, Wu, activation=name), h)
    h8, g8, u8 = lm.llmint8_gated(X, Wg, Wu, activation=name, save="8bit")
    assert torch.equal(h8, h)
    for c, v, dv in ((g8, G, dG), (u8, U, dU)):
        # half a step of the block's scale (a whole one at the clamp), besides the sum's error;
        # the scale itself may be the next one where the largest entry is near a power of two
        _, byte = fo.pack(v)
        assert int((c.scales.int() - byte.int()).abs().max()) <= 1
        step = fo.pow2(c.scales.long() - 127).repeat_interleave(32, dim=1)[:, :N]
        near(fo.unpack(c.codes, c.scales), (v, step + dv))
        assert int(c.codes.min()) >= -127


BACK = [(1, 8, 8), (1, 264, 72), (37, 72, 136), (64, 128, 128), (129, 264, 520), (300, 1040, 264),
        (1000, 40, 1096), (513, 2056, 72), (65, 2304, 3336), (4097, 264, 136),
        (1030, 4104, 4104), (2000, 2056, 11008), (520, 4096, 4096), (2304, 8200, 1032)]


@pytest.mark.parametrize("M,K,N", BACK)
@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("held", ["full", "8bit"])
def test_matmul_backward(lm, M, K, N, dtype, held):
    say("matmul backward", M, K, N, dtype, held)
    g = gen(M + K + 5 * N)
    X, W = rand(g, M, K, dtype), rand(g, K, N, dtype, 0.05)
    dY, Z = rand(g, M, N, dtype, 0.5), rand(g, M, N, dtype, 1.5)
    name = fo.ACTS[(M + K + N) // 8 % 5]
    x, xd = strided(X), X.double()
    if held == "8bit":
        x = lm.llmint8_checkpoint_pack(X)
        xd = fo.unpack(*fo.pack(X))
    dX, dW = Band(M, K, dtype), Band(K, N, dtype)
    _, _, db = lm.llmint8_matmul_backward(strided(dY), x, strided(W), Z=strided(Z),
                                          activation=name, need_dbias=True, dX=dX.t, dW=dW.t)
    dX.check(), dW.check()
    want = fo.matmul_backward(dY.double(), xd, W.double(), Z.double(), name, dtype)
    near(dX.t, want[0])
    near(dW.t, want[1])
    near(db, want[2])
    # the same call again gives the same bits
    again = lm.llmint8_matmul_backward(dY, x, W, Z=Z, activation=name, need_dbias=True)
    assert torch.equal(again[0], dX.t) and torch.equal(again[1], dW.t)
    assert torch.equal(again[2], db)
    # each output alone, with only what it needs (a product alone may be split otherwise)
    a = lm.llmint8_matmul_backward(dY, None, W, Z=Z, activation=name, need_dW=False)
    b = lm.llmint8_matmul_backward(dY, x, None, Z=Z, activation=name, need_dX=False)
    c = lm.llmint8_matmul_backward(dY, None, W, Z=Z, activation=name, need_dX=False,
                                   need_dW=False, need_dbias=True)
    near(a[0], want[0])
    near(b[1], want[1])
    assert torch.equal(c[2], db)


@pytest.mark.parametrize("M,K,N", BACK)
@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("held", ["full", "8bit"])
def test_gated_backward(lm, M, K, N, dtype, held):
    say("gated backward", M, K, N, dtype, held)
    g = gen(M + 7 * K + N)
    X = rand(g, M, K, dtype)
    Wg, Wu = rand(g, K, N, dtype, 0.05), rand(g, K, N, dtype, 0.05)
    dH, G, U = (rand(g, M, N, dtype, s) for s in (0.5, 1.5, 1.0))
    name = fo.ACTS[1 + (M + K + N) // 8 % 4]
    args = [strided(X), strided(G), strided(U)]
    vals = [X.double(), G.double(), U.double()]
    if held == "8bit":
        args = [lm.llmint8_checkpoint_pack(t) for t in (X, G, U)]
        vals = [fo.unpack(*fo.pack(t)) for t in (X, G, U)]
    dX, dWg, dWu = Band(M, K, dtype), Band(K, N, dtype), Band(K, N, dtype)
    lm.llmint8_gated_backward(strided(dH), args[0], strided(Wg), strided(Wu), args[1], args[2],
                              activation=name, dX=dX.t, dWg=dWg.t, dWu=dWu.t)
    for o in (dX, dWg, dWu):
        o.check()
    want = fo.gated_backward(dH.double(), vals[0], Wg.double(), Wu.double(), vals[1], vals[2],
                             name, dtype)
    for o, w in zip((dX, dWg, dWu), want):
        near(o.t, w)
    again = lm.llmint8_gated_backward(dH, args[0], Wg, Wu, args[1], args[2], activation=name)
    for o, t in zip((dX, dWg, dWu), again):
        assert torch.equal(o.t, t)
    a = lm.llmint8_gated_backward(dH, None, Wg, Wu, args[1], args[2], activation=name,
                                  need_dW=False)
    b = lm.llmint8_gated_backward(dH, args[0], Wg, Wu, args[1], args[2], activation=name,
                                  need_dX=False)
    assert a[1] is None and a[2] is None and b[0] is None
    near(a[0], want[0])
    near(b[1], want[1])
    near(b[2], want[2])


@pytest.mark.parametrize("M,K", [(1, 8), (3, 24), (5, 32), (37, 1000), (129, 4104), (2, 28672),
                                 (3000, 64)])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_checkpoint(lm, M, K, dtype):
    say("checkpoint", M, K, dtype)
    g = gen(M + K)
    X = rand(g, M, K, dtype)
    X[:, 0] *= 40
    X[0] *= 2.0 ** -20 if dtype == F16 else 2.0 ** -120  # subnormal values and scales
    X[-1, : K // 2] = 0
    c = lm.llmint8_checkpoint_pack(strided(X))
    codes, scales = fo.pack(X)
    assert torch.equal(c.codes, codes) and torch.equal(c.scales, scales)
    out = Band(M, K, dtype)
    back = lm.llmint8_checkpoint_unpack(c, dtype, X=out.t)
    out.check()
    v = fo.unpack(codes, scales)
    assert torch.equal(back.double(), v), "a checkpoint's values are exact in 16 bits"
    # at most half a step off, a whole one at the clamp
    step = fo.pow2(scales.long() - 127).repeat_interleave(32, dim=1)[:, :K]
    assert bool(((v - X.double()).abs() <= step).all())


def test_checkpoint_edges(lm):
    """Every scale, the clamp, ties, and blocks that are not finite."""
    say("checkpoint edges")
    # one block per power of two of bf16, its largest entry just below the next
    e = torch.arange(-133, 128, device="cuda")
    X = torch.zeros((e.numel(), 32), dtype=torch.float64, device="cuda")
    X[:, 3] = fo.pow2(e) * (2 - 2.0 ** -7)
    X[:, 4] = -X[:, 3]
    X[:, 5] = fo.pow2(e) * 2.5 / 64  # a tie
    X[:, 6] = fo.pow2(e)
    X = X.to(BF16)
    c = lm.llmint8_checkpoint_pack(X)
    codes, scales = fo.pack(X)
    assert torch.equal(c.codes, codes) and torch.equal(c.scales, scales)
    assert torch.equal(lm.llmint8_checkpoint_unpack(c, BF16).double(), fo.unpack(codes, scales))
    for bad in (float("inf"), float("-inf"), float("nan")):
        for dtype in (F16, BF16):
            X = torch.ones((3, 72), dtype=dtype, device="cuda")
            X[1, 40] = bad
            c = lm.llmint8_checkpoint_pack(X)
            assert int(c.scales[1, 1]) == 255 and not bool(c.codes[1, 32:64].any())
            back = lm.llmint8_checkpoint_unpack(c, dtype)
            want = torch.ones_like(X)
            want[1, 32:64] = float("nan")
            assert torch.equal(back.isnan(), want.isnan())
            assert torch.equal(back.nan_to_num(), want.nan_to_num())


@pytest.mark.parametrize("M,K,N", [(6, 72, 136), (130, 72, 136)])
def test_non_finite_rows_stay_alone(lm, M, K, N):
    """An infinity or NaN in one row of X leaves every other row's bits unchanged, also
    where the row is the neighbour of a partial stage; in dY likewise."""
    say("non-finite", M, K, N)
    g = gen(3)
    for dtype in (F16, BF16):
        X, W, W2 = (rand(g, M, K, dtype), rand(g, K, N, dtype, 0.1), rand(g, K, N, dtype, 0.1))
        rows = torch.arange(M, device="cuda")
        for bad in (float("inf"), float("nan")):
            Xb = X.clone()
            Xb[3] = bad
            keep = rows != 3
            assert torch.equal(lm.llmint8_matmul(Xb, W)[keep], lm.llmint8_matmul(X, W)[keep])
            assert not bool(torch.isfinite(lm.llmint8_matmul(Xb, W)[3]).any())
            a = lm.llmint8_gated(Xb, W, W2, save="8bit")
            b = lm.llmint8_gated(X, W, W2, save="8bit")
            assert torch.equal(a[0][keep], b[0][keep])
            for i in (1, 2):
                assert torch.equal(a[i].codes[keep], b[i].codes[keep])
                assert bool((a[i].scales[3] == 255).all())
            dY = rand(g, M, N, dtype)
            db = dY.clone()
            db[3] = bad
            a = lm.llmint8_matmul_backward(db, X, W)
            b = lm.llmint8_matmul_backward(dY, X, W)
            assert torch.equal(a[0][keep], b[0][keep])
            # a NaN column of dY reaches that column of dW alone
            db = dY.clone()
            db[:, 9] = bad
            a = lm.llmint8_matmul_backward(db, X, W, need_dX=False)
            cols = torch.arange(N, device="cuda") != 9
            assert torch.equal(a[1][:, cols], b[1][:, cols])


def test_activations_at_large_arguments(lm):
    """Saturated and infinite pre-activations: what the formulas give, and no NaN for any
    finite argument, forward and backward."""
    say("large arguments")
    z = torch.tensor([0.0, -0.0, 1e-7, -1e-7, 5.0, -5.0, 20.0, -20.0, 88.0, -88.0, 89.0, -89.0,
                      200.0, -200.0, 3e4, -3e4], dtype=BF16, device="cuda")
    M = z.numel()
    X = torch.zeros((M, 8), dtype=BF16, device="cuda")
    X[:, 0] = z
    W = torch.zeros((8, 8), dtype=BF16, device="cuda")
    W[0] = 1
    Z = z[:, None].expand(M, 8).contiguous()
    dY = torch.ones((M, 8), dtype=BF16, device="cuda")
    eye = torch.eye(8, dtype=BF16, device="cuda")
    for name in fo.ACTS:
        near(lm.llmint8_matmul(X, W, activation=name),
             fo.matmul(X.double(), W.double(), None, None, name, BF16)[0])
        dX, _, _ = lm.llmint8_matmul_backward(dY, None, eye, Z=Z, activation=name, need_dW=False)
        near(dX, fo.matmul_backward(dY.double(), X.double(), eye.double(), Z.double(), name,
                                    BF16)[0])
        h = lm.llmint8_gated(X, W, W, activation=name)
        near(h, fo.gated(X.double(), W.double(), W.double(), name, BF16)[0])


def test_other_stream(lm):
    """Calls follow torch's current stream, workspaces included."""
    say("other stream")
    g = gen(21)
    X, Wg, Wu = rand(g, 40, 2048, F16), rand(g, 2048, 264, F16, 0.05), rand(g, 2048, 264, F16, 0.05)
    dH = rand(g, 40, 264, F16)
    def run():
        h, G, U = lm.llmint8_gated(X, Wg, Wu, save="8bit")
        return [h, *lm.llmint8_gated_backward(dH, lm.llmint8_checkpoint_pack(X), Wg, Wu, G, U)]
    want = run()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = [run() for _ in range(3)]
    torch.cuda.synchronize()
    for r in got:
        for a, b in zip(r, want):
            assert torch.equal(a, b)


@pytest.mark.parametrize("M,K,N", [(1, 4096, 264), (40, 2048, 264), (300, 1040, 520)])
def test_graph_replay(lm, M, K, N):
    say("graph replay", M, K, N)
    g = gen(22)
    X, Wg, Wu = rand(g, M, K, BF16), rand(g, K, N, BF16, 0.05), rand(g, K, N, BF16, 0.05)
    Wd, dY, bias = rand(g, N, K, BF16, 0.05), rand(g, M, K, BF16), rand(g, 1, K, BF16)[0]
    def step():
        h, G, U = lm.llmint8_gated(X, Wg, Wu, save="8bit")
        y = lm.llmint8_matmul(h, Wd, bias=bias, residual=X)
        dH, dWd, db = lm.llmint8_matmul_backward(dY, h, Wd, need_dbias=True)
        c = lm.llmint8_checkpoint_pack(X)
        return [y, dWd, db, *lm.llmint8_gated_backward(dH, c, Wg, Wu, G, U)]
    want = [t.clone() for t in step()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for rep in range(4):
        for t in out:
            t.fill_(3.0)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, want):
            assert torch.equal(a, b), rep
        other = step()  # eager work between replays
        torch.cuda.synchronize()
        for a, b in zip(other, want):
            assert torch.equal(a, b), rep


@pytest.mark.parametrize("name", fo.ACTS[1:])
def test_gradients_against_differences(lm, name):
    """The kernels' gradients against central differences of the block's output in 64 bits
    along random directions of every input: for the loss <D, gated(X) Wd + residual>, the
    difference quotient at step h is off by at most the third derivative times h^2 / 6, and
    the gradients by the bounds of their roundings (relu is differenced away from its kink)."""
    say("differences", name)
    g = gen(41)
    M, K, N, dt = 24, 64, 96, F16
    X, Wg, Wu, D = (rand(g, M, K, dt), rand(g, K, N, dt, 0.2), rand(g, K, N, dt, 0.2),
                    rand(g, M, N, dt))
    if name == "relu":  # keep every pre-activation at least 0.02 from the kink
        G = X.double() @ Wg.double()
        D = torch.where(G.abs() < 0.02, torch.zeros_like(D), D)
    H, G, U = lm.llmint8_gated(X, Wg, Wu, activation=name, save="full")
    grads = lm.llmint8_gated_backward(D, X, Wg, Wu, G, U, activation=name)
    at = [X.double(), Wg.double(), Wu.double()]

    def loss(x, wg, wu):
        return (D.double() * fo.act(name, x @ wg) * (x @ wu)).sum()
    for i, grad in enumerate(grads):
        V = torch.randn(at[i].shape, generator=g, device="cuda", dtype=torch.float64)
        V /= V.norm()
        h = 1e-4
        up, down = [list(at), list(at)]
        up[i], down[i] = at[i] + h * V, at[i] - h * V
        want = float((loss(*up) - loss(*down)) / (2 * h))
        got = float((grad.double() * V).sum())
        # V has norm 1: independent relative errors of the gradient's entries (its own
        # rounding, G and U rounded to 16 bits, dG and dU rounded) stay below 8 u of its
        # norm, differences below 1e-6 of it
        assert abs(got - want) <= 8 * fo.U[dt] * float(grad.double().norm()) + 1e-6, (name, i)


def test_training_example():
    """The example runs the operators together. Against the same training in plain fp32: the
    weights start alike and see the same tokens, and the 8-bit checkpoints and 16-bit gradients
    move Adam's steps by a few hundredths at random, so the loss stays within 5 % of the first
    one throughout. The int8 layers agree with the trained block."""
    say("training example")
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "train_feed_forward.py")
    spec = importlib.util.spec_from_file_location("train_feed_forward", path)
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    steps, tokens, width, hidden, lr = 40, 256, 128, 352, 2e-3
    losses, W = ex.train(steps, tokens, width, hidden, lr=lr)
    g = torch.Generator(device="cuda").manual_seed(0)
    target, master = ex.setup(width, hidden, BF16, g)
    target = [w.float() for w in target]
    params = [w.requires_grad_() for w in master]
    opt = torch.optim.Adam(params, lr=lr, betas=(0.9, 0.99), eps=1e-8)
    block = lambda x, w: x + (torch.nn.functional.silu(x @ w[0]) * (x @ w[1])) @ w[2]
    for step in range(steps):
        X = torch.randn((tokens, width), generator=g, device="cuda").to(BF16).float()
        err = block(X, params) - block(X, target)
        loss = err.square().mean()
        now = float(loss.detach())
        assert abs(now - losses[step]) < 0.05 * losses[0], (step, now, losses[step])
        opt.zero_grad()
        (err.square().sum() / tokens).backward()
        opt.step()
    assert losses[-1] < losses[0]
    X = rand(gen(5), 3, 128, F16)
    half = [w.half() for w in W]
    y16, _ = ex.forward(X, half, keep=False)
    y8 = ex.serve_int8(X, half)
    # int8 codes of rows and columns: steps of 1/127 of the largest entry, rounded
    assert float((y8.float() - y16.float()).norm() / y16.float().norm()) < 0.05
