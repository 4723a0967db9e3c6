"""The gated feed-forward block, forward and backward, on the GPU against 64 bits.

The tensor cores multiply exactly and add in fp32, 16 products or more to an
instruction: a sum over K passes K / 16 additions in a chain (and the joins of a
split contraction), each within 2^-23 of the magnitudes summed so far -- the
bound used here allows for truncating adders.  Activations have slopes of at
most 1.13 and are evaluated within a few ulp of fp32 of 1 + |z|.
"""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import gated_plain as plain  # noqa: E402
import ops_plain  # noqa: E402
from ops_gpu import E, TINY, Out, U, assert_close, bits, f64, make, scratch, strided  # noqa: E402

pytestmark = pytest.mark.gpu
BF, F16, F32 = torch.bfloat16, torch.float16, torch.float32
Q8 = torch.float8_e4m3fn
HALF = [BF, F16]
ACTS = ["none", "relu", "gelu", "gelu_tanh", "silu"]


def code(arx, act):
    return getattr(arx, "ARX_ACT_" + act.upper())


def chain(k):
    return (k / 16 + 16) * 2 * E


def matmul(a, b):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda().matmul(torch.from_numpy(np.ascontiguousarray(b)).cuda()).cpu().numpy()


def eight(rows, cols, seed, scale, pad=0):
    """An e4m3 matrix on rows of 16 bytes (``pad`` more of them in each row), with values of all magnitudes."""
    pitch = (cols + 15) // 16 * 16 + 16 * pad
    buf = torch.zeros(rows, pitch, dtype=torch.uint8, device="cuda").view(Q8)
    buf[:, :cols] = (make((rows, cols), F32, seed) * scale).to(Q8)
    return buf[:, :cols]


def operands(M, N, K, dtype, pad=0, lead=0, seed=0):
    if dtype is Q8:
        return (eight(M, K, seed + 1, 30.0, pad), eight(N, K, seed + 2, 30.0, pad), eight(N, K, seed + 3, 30.0))
    s = max(K, 1) ** -0.5
    return (strided(make((M, K), dtype, seed + 1), pad, lead), strided(make((N, K), dtype, seed + 2, s), pad, lead),
            strided(make((N, K), dtype, seed + 3, s), pad, lead))


def check_forward(x, w, act, out, zg=None, zu=None, bias=(None, None), scales=None):
    """Outputs against 64 bits of the operands as numbers."""
    X, W = f64(x), [f64(t) for t in w]
    K = X.shape[1]
    z, ez = [], []
    for i in range(2):
        v, size = matmul(X, W[i].T), matmul(np.abs(X), np.abs(W[i]).T)
        e = chain(K) * size
        if scales is not None:
            s = scales[0][:, None] * scales[1 + i]
            v, e = v * s, (e + 3 * E * np.abs(v)) * s
        if bias[i] is not None:
            v = v + f64(bias[i])
            e = e + 2 * E * np.abs(v)
        z.append(v)
        ez.append(e)
    g, u = z
    if zg is not None:
        assert_close(zg, g, ez[0], "z_gate")
    if zu is not None:
        assert_close(zu, u, ez[1], "z_up")
    f = ops_plain.act(g, act)
    ef = 1.2 * ez[0] + (0 if act == "none" else 24 * E * (1 + np.abs(g)))
    assert_close(out, f * u, ef * (np.abs(u) + ez[1]) + np.abs(f) * ez[1] + 2 * E * np.abs(f * u), "out")


def forward(arx, M, N, K, dtype, act="silu", bias=True, z=True, wdtype=None, otype=None, pad=0, lead=0, opad=0, olead=0,
            scaled=True, **more):
    o = otype or (BF if dtype is Q8 else dtype)
    x, wg, wu = operands(M, N, K, dtype, pad, lead)
    b = [make((N,), wdtype or o, 4 + i) for i in range(2)] if bias else [None, None]
    out = Out((M, N), o, opad, olead)
    zs = [Out((M, N), o, opad, olead) for _ in range(2)] if z else [None, None]
    scales = None
    if dtype is Q8 and scaled:
        g = torch.Generator(device="cuda").manual_seed(9)
        # Sums of K products of numbers of about 30, brought to about 1.
        scales = [(0.5 + torch.rand(n, generator=g, device="cuda")) * s
                  for n, s in ((M, 1 / 30), (N, max(K, 1) ** -0.5 / 30), (N, max(K, 1) ** -0.5 / 30))]
        more |= dict(zip(("x_scale", "gate_scale", "up_scale"), scales))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    if z:
        more |= {"z_gate": zs[0].t, "z_up": zs[1].t}
    arx.arx_gated_linear(x, wg, wu, out.t, bias_gate=b[0], bias_up=b[1], act=code(arx, act), status=status, **more)
    torch.cuda.synchronize()
    assert int(status) == 0
    check_forward(x, (wg, wu), act, out, *zs, bias=b, scales=scales and [f64(s) for s in scales])


# One token to many, one feature to many, a contraction inside a stage, at its end and beyond:
# dot products, clusters of 1 to 8 blocks over 16 to 256 tokens, pairs on accumulators of 128
# and 256 columns and on two of them.
SHAPES = [(1, 1, 1), (1, 8, 8), (1, 128, 64), (2, 136, 72), (3, 8, 8), (16, 128, 128), (17, 129, 65), (33, 1000, 200),
          (64, 256, 512), (65, 264, 1032), (129, 127, 63), (200, 1536, 256), (257, 257, 257), (300, 64, 4096),
          (1, 4096, 4096), (2, 2048, 4096), (1000, 130, 96), (1280, 2560, 128), (1291, 2563, 130), (2000, 1000, 264),
          (500, 1023, 4096), (300, 4096, 4096), (1000, 4072, 2048), (1000, 4070, 2056)]


@pytest.mark.parametrize("dtype", [BF, F16, Q8], ids=str)
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_forward(arx, M, N, K, dtype):
    forward(arx, M, N, K, dtype)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M,N,K", [(1, 264, 128), (40, 200, 72), (1400, 2600, 64)])
def test_activations(arx, M, N, K, act):
    forward(arx, M, N, K, BF, act, wdtype=F32)
    forward(arx, M, N, K, F16, act, z=False)
    forward(arx, M, N, K, F16, act, bias=False)
    forward(arx, M, N, K, Q8, act, otype=F16, wdtype=F32)
    forward(arx, M, N, K, Q8, act, otype=BF, bias=False, z=False)


# Tiles of 80 to 128 features on one accumulator and on two, whole and cut, with a last run of
# 16 columns; the last round of tiles in halves.
@pytest.mark.parametrize("M,N,K", [(3000, 776, 2048), (3000, 775, 2050), (1500, 792, 1024), (1500, 1920, 4096),
                                   (1500, 1925, 4096), (3000, 1184, 4096), (3000, 1186, 4096), (3000, 1344, 4096),
                                   (3000, 1181, 520), (3000, 800, 264), (4864, 1024, 2048)])
@pytest.mark.parametrize("dtype", [BF, Q8], ids=str)
def test_large_forms(arx, M, N, K, dtype):
    forward(arx, M, N, K * (2 if dtype is Q8 else 1), dtype, "gelu", z=False, bias=False)
    forward(arx, M, N, K * (2 if dtype is Q8 else 1), dtype, opad=1 if K == 264 else 0)


@pytest.mark.parametrize("N", [5072, 5074])
def test_a_last_round_of_tiles_in_halves(arx, N):
    # Six rounds of whole tiles and 24 tiles more; compared on the GPU, row block by row block.
    M, K = 6144, 8192
    x, wg, wu = operands(M, N, K, BF)
    out = Out((M, N), BF)
    arx.arx_gated_linear(x, wg, wu, out.t)
    out.check_guards()
    for r in range(0, M, 1024):
        X, W = x[r:r + 1024].double(), [t.double().t() for t in (wg, wu)]
        (g, u), (eg, eu) = [X @ w for w in W], [chain(K) * (X.abs() @ w.abs()) for w in W]
        f = g * torch.sigmoid(g)
        want, err = f * u, (1.2 * eg + 24 * E * (1 + g.abs())) * (u.abs() + eu) + f.abs() * eu
        off = (out.t[r:r + 1024].double() - want).abs() - err - U[BF] * want.abs() * (1 + 2 * U[BF]) - 2 * E * want.abs()
        assert bool((off <= TINY[BF]).all())


@pytest.mark.parametrize("M,N,K", [(2, 72, 136), (5, 72, 136), (1300, 2600, 80)])
@pytest.mark.parametrize("pad,lead,opad,olead", [(8, 8, 8, 8), (0, 1, 0, 0), (3, 0, 0, 0), (8, 0, 3, 1), (1, 3, 0, 4)])
def test_strides_and_alignment(arx, M, N, K, pad, lead, opad, olead):
    forward(arx, M, N, K, BF, "gelu", pad=pad, lead=lead, opad=opad, olead=olead)


@pytest.mark.parametrize("M,N,K", [(1, 72, 136), (2, 200, 160), (5, 72, 136), (1300, 2600, 80)])
@pytest.mark.parametrize("pad,opad,olead", [(1, 8, 8), (0, 3, 1), (2, 0, 4)])
def test_strides_of_eight_bits(arx, M, N, K, pad, opad, olead):
    forward(arx, M, N, K, Q8, pad=pad, opad=opad, olead=olead)


@pytest.mark.parametrize("given", [(1, 0, 0), (0, 1, 0), (0, 1, 1), (1, 0, 1), (1, 1, 0), (0, 0, 0)])
@pytest.mark.parametrize("M", [1, 40])
def test_some_scales(arx, M, given):
    # The operands' values brought near 1 by the scales that are there.
    N, K = 96, 160
    x, wg, wu = (eight(r, K, s, 1.0) for r, s in ((M, 1), (N, 2), (N, 3)))
    names, sizes = ("x_scale", "gate_scale", "up_scale"), (M, N, N)
    kw = {n: torch.rand(k, device="cuda") + 0.1 for n, k, on in zip(names, sizes, given) if on}
    out = Out((M, N), BF)
    arx.arx_gated_linear(x, wg, wu, out.t, **kw)
    check_forward(x, (wg, wu), "silu", out, scales=[f64(kw[n]) if n in kw else np.ones(k) for n, k in zip(names, sizes)])


@pytest.mark.parametrize("dtype", [BF, Q8], ids=str)
@pytest.mark.parametrize("M,N", [(1, 72), (7, 40), (1300, 2600)])
def test_no_contraction(arx, M, N, dtype):
    # Sums of nothing: out is that of the biases.
    forward(arx, M, N, 0, dtype, scaled=False)


@pytest.mark.parametrize("M", [1, 20, 1500])
def test_parts_of_one_buffer(arx, M):
    # Both weights in one matrix, one after the other or row by row in turn; both outputs too.
    N, K = 264, 136
    x, both = make((M, K), BF, 1), make((2 * N, K), BF, 2, K ** -0.5)
    for wg, wu in ((both[:N], both[N:]), (both[::2], both[1::2])):
        buf = torch.full((M, 3 * N), 97.0, dtype=BF, device="cuda")
        arx.arx_gated_linear(x, wg, wu, buf[:, N:2 * N], z_gate=buf[:, :N], z_up=buf[:, 2 * N:])
        check_forward(x, (wg, wu), "silu", buf[:, N:2 * N], buf[:, :N], buf[:, 2 * N:])
    # One weight for both projections.
    out = torch.empty(M, N, dtype=BF, device="cuda")
    arx.arx_gated_linear(x, both[:N], both[:N], out, act=arx.ARX_ACT_NONE)
    check_forward(x, (both[:N], both[:N]), "none", out)


def test_a_single_projection_is_kept(arx):
    M, N, K = 70, 200, 72
    x, wg, wu = operands(M, N, K, BF)
    for names in (("z_gate",), ("z_up",)):
        z, out = Out((M, N), BF), Out((M, N), BF)
        arx.arx_gated_linear(x, wg, wu, out.t, **{n: z.t for n in names})
        check_forward(x, (wg, wu), "silu", out, *([z, None] if names[0] == "z_gate" else [None, z]))


@pytest.mark.parametrize("M,N,K", [(1, 64, 128), (20, 64, 128), (1500, 2600, 128)])
@pytest.mark.parametrize("dtype", [BF, Q8], ids=str)
def test_infinities_and_nan(arx, M, N, K, dtype):
    x, wg, wu = operands(M, N, K, dtype)
    x, wg = x.clone(), wg.clone()
    special = torch.tensor([float("nan"), 1.0], device="cuda").to(dtype)
    x[M - 1, 3] = special[0]
    wg[5, 7] = special[0]
    out = torch.empty(M, N, dtype=BF, device="cuda")
    kw = {} if dtype is BF else {"x_scale": torch.full((M,), 1e-2, device="cuda")}
    arx.arx_gated_linear(x, wg, wu, out, **kw)
    nan = torch.isnan(out)
    assert bool(nan[M - 1].all()) and bool(nan[:, 5].all())
    nan[M - 1], nan[:, 5] = False, False
    assert not bool(nan.any())
    if dtype is BF:  # act(-inf) is 0, and its product with a finite u too
        x2, w2 = torch.ones(M, K, dtype=BF, device="cuda"), torch.zeros(N, K, dtype=BF, device="cuda")
        b = torch.full((N,), float("-inf"), device="cuda")
        b[1] = float("inf")
        arx.arx_gated_linear(x2, w2, w2 + 1, out, bias_gate=b.to(BF))
        assert bool((out[:, 0] == 0).all()) and bool((out[:, 1] == float("inf")).all())


def backward(arx, M, N, K, dtype, act="silu", bias=True, wdtype=None, pad=0, lead=0, opad=0, olead=0, what="xgu"):
    x, wg, wu = operands(M, N, K, dtype, pad, lead)
    d, g, u = (strided(make((M, N), dtype, 10 + i), pad, lead) for i in range(3))
    dx = Out((M, K), dtype, opad, olead) if "x" in what else None
    dw = [Out((N, K), dtype, opad, olead) if c in what else None for c in "gu"]
    db = [Out((N,), wdtype or dtype) if bias else None for _ in range(2)]
    t = lambda o: None if o is None else o.t  # noqa: E731
    ws, status = scratch(arx.arx_gated_linear_bwd_workspace_bytes(M, N)), torch.zeros(1, dtype=torch.int32, device="cuda")
    arx.arx_gated_linear_bwd(d, x, wg, wu, g, u, dx=t(dx), dw_gate=t(dw[0]), dw_up=t(dw[1]), dbias_gate=t(db[0]),
                             dbias_up=t(db[1]), act=code(arx, act), workspace=ws, status=status)
    torch.cuda.synchronize()
    assert int(status) == 0
    D, G, V, X, W = f64(d), f64(g), f64(u), f64(x), [f64(wg), f64(wu)]
    dz = [D * V * ops_plain.act_grad(G, act), D * ops_plain.act(G, act)]
    # dg and du: the activation's error, two products, and (as operands) a rounding.
    ez = [np.abs(D * V) * (0 if act == "none" else 32 * E * (1 + np.abs(G))) + 3 * E * np.abs(dz[0]),
          np.abs(D) * (0 if act == "none" else 24 * E * (1 + np.abs(G))) + 3 * E * np.abs(dz[1])]
    er = [e + U[dtype] * (np.abs(z) + e) + TINY[dtype] for e, z in zip(ez, dz)]
    size = [np.abs(z) + e for z, e in zip(dz, er)]
    if dx is not None:
        err = sum(matmul(er[i] + chain(2 * N) * size[i], np.abs(W[i])) for i in range(2))
        assert_close(dx, matmul(dz[0], W[0]) + matmul(dz[1], W[1]), err, "dx")
    for i in range(2):
        if dw[i] is not None:
            assert_close(dw[i], matmul(dz[i].T, X), matmul((er[i] + chain(M) * size[i]).T, np.abs(X)), f"dw {i}")
        if db[i] is not None:
            assert_close(db[i], dz[i].sum(0), ez[i].sum(0) + (M + 70) * E * np.abs(dz[i]).sum(0), f"dbias {i}")


@pytest.mark.parametrize("dtype", HALF, ids=str)
@pytest.mark.parametrize("M,N,K", [(1, 1, 1), (1, 8, 8), (2, 136, 72), (5, 64, 128), (17, 129, 65), (33, 1000, 200),
                                   (64, 256, 512), (129, 127, 63), (257, 257, 257), (1000, 130, 96), (259, 2050, 1030),
                                   (1280, 2560, 128), (1291, 2563, 130), (2000, 1000, 264), (700, 64, 2000)])
def test_backward(arx, M, N, K, dtype):
    backward(arx, M, N, K, dtype)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M,N,K", [(3, 264, 128), (40, 200, 72), (1400, 520, 264)])
def test_backward_activations(arx, M, N, K, act):
    backward(arx, M, N, K, BF, act, wdtype=F32)
    backward(arx, M, N, K, F16, act, bias=False)


@pytest.mark.parametrize("M,N,K", [(1000, 2048, 4096), (2050, 1000, 4100), (512, 4096, 2048)])
def test_backward_large_forms(arx, M, N, K):
    backward(arx, M, N, K, BF)


@pytest.mark.parametrize("what", ["", "x", "g", "u", "gu", "xg", "xu"])
def test_backward_parts(arx, what):
    backward(arx, 70, 200, 136, BF, what=what)
    backward(arx, 70, 203, 131, F16, what=what, bias=what == "")


@pytest.mark.parametrize("M,N,K", [(5, 72, 136), (300, 1000, 520)])
@pytest.mark.parametrize("pad,lead,opad,olead", [(8, 8, 8, 8), (0, 1, 0, 0), (3, 0, 0, 0), (8, 0, 3, 1), (1, 3, 0, 4)])
def test_backward_strides(arx, M, N, K, pad, lead, opad, olead):
    backward(arx, M, N, K, BF, "gelu", pad=pad, lead=lead, opad=opad, olead=olead)


def test_backward_against_differences(arx):
    # The gradient of sum(out dout) by central differences of the forward formula in 64 bits at the
    # 16-bit operands: the gradients carry dz's rounding and their own, each 2^-11 of the magnitudes.
    M, N, K, h = 6, 40, 24, 1e-5
    x, wg, wu = operands(M, N, K, F16)
    d, out, zg, zu = make((M, N), F16, 9), *(torch.empty(M, N, dtype=F16, device="cuda") for _ in range(3))
    arx.arx_gated_linear(x, wg, wu, out, z_gate=zg, z_up=zu)
    dx, dg, du = torch.empty_like(x), torch.empty_like(wg), torch.empty_like(wu)
    ws = scratch(arx.arx_gated_linear_bwd_workspace_bytes(M, N))
    arx.arx_gated_linear_bwd(d, x, wg, wu, zg, zu, dx=dx, dw_gate=dg, dw_up=du, workspace=ws)
    at, D = [f64(x), f64(wg), f64(wu)], f64(d)
    loss = lambda a: (plain.gated(*a, "silu")[0] * D).sum()  # noqa: E731
    for i, grad in enumerate((dx, dg, du)):
        grad = f64(grad)
        # z is rounded to 16 bits too: of values of about 1 with slopes of about 1, over the contraction.
        size = np.sqrt((grad * grad).mean())
        for r, c in ((0, 0), (3, 17), (5, 23)):
            a, b = [t.copy() for t in at], [t.copy() for t in at]
            a[i][r, c] += h
            b[i][r, c] -= h
            assert abs((loss(a) - loss(b)) / (2 * h) - grad[r, c]) < 2.0 ** -7 * max(size, abs(grad[r, c]))


@pytest.mark.parametrize("M,N,K", [(0, 24, 16), (5, 0, 16), (5, 24, 0)])
def test_empty(arx, M, N, K):
    x, wg, wu = operands(M, N, K, BF)
    out = torch.full((M, N), 3.0, dtype=BF, device="cuda")
    arx.arx_gated_linear(x, wg, wu, out)
    assert not bool(out.any())
    d = torch.ones(M, N, dtype=BF, device="cuda")
    dx, dg, du = (torch.full_like(t, 3.0) for t in (x, wg, wu))
    db = [torch.full((N,), 3.0, device="cuda") for _ in range(2)]
    ws = scratch(arx.arx_gated_linear_bwd_workspace_bytes(M, N))
    arx.arx_gated_linear_bwd(d, x, wg, wu, d, d, dx=dx, dw_gate=dg, dw_up=du, dbias_gate=db[0], dbias_up=db[1], workspace=ws)
    assert not bool(dx.any()) and not bool(dg.any()) and not bool(du.any())
    if M == 0:
        assert not bool(db[0].any()) and not bool(db[1].any())


@pytest.mark.parametrize("M,N,K", [(1, 2048, 1024), (24, 1000, 520), (1291, 2563, 130), (1000, 1024, 2048)])
def test_same_bits_on_side_streams_and_in_graphs(arx, M, N, K):
    x, wg, wu = operands(M, N, K, BF)
    d = make((M, N), BF, 8)

    def buffers():
        n = lambda r, c: torch.empty(r, c, dtype=BF, device="cuda")  # noqa: E731
        return {"out": n(M, N), "zg": n(M, N), "zu": n(M, N), "dx": n(M, K), "dg": n(N, K), "du": n(N, K),
                "db": torch.empty(N, device="cuda"), "ws": scratch(arx.arx_gated_linear_bwd_workspace_bytes(M, N))}

    def step(b):
        arx.arx_gated_linear(x, wg, wu, b["out"], z_gate=b["zg"], z_up=b["zu"])
        arx.arx_gated_linear_bwd(d, x, wg, wu, b["zg"], b["zu"], dx=b["dx"], dw_gate=b["dg"], dw_up=b["du"],
                                 dbias_up=b["db"], workspace=b["ws"])

    want, other, captured = buffers(), buffers(), buffers()
    step(want)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        for _ in range(3):
            step(other)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(captured)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    for k in want:
        if k != "ws":
            assert torch.equal(bits(want[k]), bits(other[k])) and torch.equal(bits(want[k]), bits(captured[k])), k


def test_a_plan_with_copies_of_its_own(arx):
    # Operands off 16 bytes: the plan's copies are its own, a captured call's the graph's.
    M, N, K = 130, 1001, 2051
    x, wg, wu = operands(M, N, K, BF)
    outs = [torch.empty(M, N, dtype=BF, device="cuda") for _ in range(2)]
    assert arx.arx_gated_linear_copies_bytes(x, wg, wu) == (M + 2 * N) * 2056 * 2
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    plans = [arx.arx_gated_linear_plan(x, wg, wu, o, stream=side) for o in outs]
    plans[0]()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        plans[1]()
    del plans
    torch.cuda.synchronize()
    x.mul_(2.0)
    graph.replay()
    torch.cuda.synchronize()
    check_forward(x, (wg, wu), "silu", outs[1])
    assert not torch.equal(outs[0], outs[1])


def test_offsets_beyond_32_bits(arx):
    # Rows 2^31 elements apart: the third starts beyond 2^32 elements.
    N, K, ld = 40, 72, 1 << 31
    buf = torch.empty(2 * ld + 96 + N, dtype=BF, device="cuda")
    x = torch.as_strided(buf, (3, K), (ld, 1))
    x.copy_(make((3, K), BF, 1))
    _, wg, wu = operands(3, N, K, BF)
    out = Out((3, N), BF)
    arx.arx_gated_linear(x, wg, wu, out.t)
    check_forward(x, (wg, wu), "silu", out)
    far = torch.as_strided(buf, (3, N), (ld, 1), 96)
    arx.arx_gated_linear(x, wg, wu, far)
    assert torch.equal(far, out.t)


# ---- waits that run out -------------------------------------------------------------------

FORMS = {"split": (64, 64, 1 << 23, BF), "split_wide": (1300, 2048, 1 << 19, BF), "pairs": (2000, 1000, 1 << 19, BF),
         "two_accumulators": (4096, 4096, 1 << 18, BF), "split_eight": (64, 64, 1 << 24, Q8),
         "pairs_eight": (4096, 4096, 1 << 19, Q8)}


@pytest.mark.parametrize("form", FORMS)
def test_a_wait_that_runs_out_ends_with_a_status(arx, form):
    M, N, K, t = FORMS[form]
    x, wg, wu = (torch.ones(r, K, device="cuda", dtype=BF).to(t) for r in (M, N, N))
    scale = {} if t is BF else {"x_scale": torch.full((M,), 1.0 / K, device="cuda")}
    value = float(K) ** 2 if t is BF else 1.0
    out, zg, zu = (torch.full((M, N), 3.0, dtype=BF, device="cuda") for _ in range(3))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    arx.arx_gated_linear(x, wg, wu, out, z_gate=zg, z_up=zu, act=arx.ARX_ACT_RELU, status=status, wait_us=1000, **scale)
    torch.cuda.synchronize()
    assert int(status) & 0xFF == arx.ARX_ETIMEOUT
    for o, v in ((out, value), (zg, value ** 0.5), (zu, value ** 0.5)):
        nan = torch.isnan(o)
        assert bool(nan.any()) and bool((o[~nan] == v).all())
    # The context and the SMs' memory are in order: the same call with the default limit is right.
    for _ in range(2):
        status.zero_()
        out.zero_()
        arx.arx_gated_linear(x, wg, wu, out, act=arx.ARX_ACT_RELU, status=status, **scale)
        torch.cuda.synchronize()
        assert int(status) == 0 and bool((out == value).all())


# M, N, K and the gradients asked for: dx as one sum over both projections, and both weights'
# gradients in one launch, in the split form and over pairs.
BACKWARD_FORMS = {"dx_split": (64, 1 << 20, 128, "x"), "dx_pairs": (2000, 1 << 17, 2000, "x"),
                  "dw_split": (1 << 20, 64, 64, "gu"), "dw_pairs": (1 << 18, 1500, 2000, "gu")}


@pytest.mark.parametrize("form", BACKWARD_FORMS)
def test_a_gradients_wait_that_runs_out(arx, form):
    M, N, K, what = BACKWARD_FORMS[form]
    ones = lambda r, c: torch.ones(r, c, dtype=BF, device="cuda")  # noqa: E731
    d, x, w = ones(M, N), ones(M, K), ones(N, K)
    outs = {"dx": torch.full((M, K), 3.0, dtype=BF, device="cuda")} if what == "x" else \
        {n: torch.full((N, K), 3.0, dtype=BF, device="cuda") for n in ("dw_gate", "dw_up")}
    value = 2.0 * N if what == "x" else float(M)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = torch.empty(arx.arx_gated_linear_bwd_workspace_bytes(M, N), dtype=torch.uint8, device="cuda")
    call = lambda **kw: arx.arx_gated_linear_bwd(d, x, w, w, d, d, act=arx.ARX_ACT_NONE, workspace=ws, status=status,  # noqa: E731
                                                 **outs, **kw)
    call(wait_us=100)
    torch.cuda.synchronize()
    assert int(status) & 0xFF == arx.ARX_ETIMEOUT
    some = False
    for o in outs.values():
        nan = torch.isnan(o)
        some |= bool(nan.any())
        assert bool((o[~nan] == value).all())
    assert some
    for _ in range(2):
        status.zero_()
        for o in outs.values():
            o.zero_()
        call()
        torch.cuda.synchronize()
        assert int(status) == 0 and all(bool((o == value).all()) for o in outs.values())
