"""The matrix product with its epilogue, forward and backward, on the GPU against 64 bits.

The tensor cores multiply exactly and add in fp32, 16 products to an
instruction: a result passes K / 16 additions in a chain (and the joins of a
split contraction), each within 2^-23 of the magnitudes summed so far -- the
bound used here allows for truncating adders.
"""

import numpy as np
import pytest
import torch

import ops_plain as plain
from ops_gpu import E, Out, U, assert_close, bits, f64, make, scratch, strided

pytestmark = pytest.mark.gpu
HALF = [torch.bfloat16, torch.float16]
ACTS = ["none", "relu", "gelu", "gelu_tanh", "silu"]


def _code(arx, act):
    return getattr(arx, "ARX_ACT_" + act.upper())


def _chain(k):
    return (k / 16 + 16) * 2 * E


def _matmul(a, b):
    return torch.from_numpy(a).cuda().matmul(torch.from_numpy(b).cuda()).cpu().numpy()


def _forward(arx, M, N, K, dtype, act="none", bias=True, residual=True, z=True, wdtype=None, pad=0, lead=0, opad=0,
             olead=0, copies=None):
    x = strided(make((M, K), dtype, 1), pad, lead)
    w = strided(make((N, K), dtype, 2, max(K, 1) ** -0.5), pad, lead)
    b = make((N,), wdtype or dtype, 3) if bias else None
    r = strided(make((M, N), dtype, 4), opad, olead) if residual else None
    out = Out((M, N), dtype, opad, olead)
    zo = Out((M, N), dtype, opad, olead) if z else None
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    arx.arx_linear(x, w, out.t, bias=b, residual=r, z=zo.t if z else None, act=_code(arx, act), status=status,
                   copies=copies)
    torch.cuda.synchronize()
    assert int(status) == 0
    xd, wd = f64(x), f64(w)
    wz = _matmul(xd, wd.T.copy())
    ez = _chain(K) * _matmul(np.abs(xd), np.abs(wd).T.copy())
    if bias:
        wz = wz + f64(b)
        ez = ez + 2 * E * np.abs(wz)
    if z:
        assert_close(zo, wz, ez, "z")
    want = plain.act(wz, act)
    # Slopes are at most 1.13; the functions are evaluated within a few ulp of fp32 of 1 + |z|.
    lim = 1.2 * ez + (0 if act == "none" else 24 * E * (1 + np.abs(wz)))
    if residual:
        want = want + f64(r)
    assert_close(out, want, lim + 2 * E * np.abs(want), "out")


# One token to many, one feature to many, a contraction inside a stage, at its end and beyond.
SHAPES = [(1, 1, 1), (1, 8, 8), (1, 128, 64), (2, 136, 72), (16, 128, 128), (17, 129, 65), (33, 1000, 200),
          (64, 256, 512), (65, 264, 1032), (129, 127, 63), (200, 1536, 256), (257, 257, 257), (300, 64, 4096),
          (1, 4096, 4096), (1000, 130, 96), (1280, 2560, 128), (1291, 2563, 130), (2000, 2000, 264)]


@pytest.mark.parametrize("dtype", HALF)
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_forward(arx, M, N, K, dtype):
    _forward(arx, M, N, K, dtype)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M,N,K", [(1, 264, 128), (40, 200, 72), (1400, 2600, 64)])
def test_activations(arx, M, N, K, act):
    _forward(arx, M, N, K, torch.bfloat16, act, wdtype=torch.float32)
    _forward(arx, M, N, K, torch.float16, act, residual=False, z=False)
    _forward(arx, M, N, K, torch.float16, act, bias=False)


@pytest.mark.parametrize("M,N,K", [(5, 72, 136), (1300, 2600, 80)])
@pytest.mark.parametrize("pad,lead,opad,olead", [(8, 8, 8, 8), (0, 1, 0, 0), (3, 0, 0, 0), (8, 0, 3, 1), (1, 3, 0, 4)])
def test_strides_and_alignment(arx, M, N, K, pad, lead, opad, olead):
    _forward(arx, M, N, K, torch.bfloat16, "gelu", pad=pad, lead=lead, opad=opad, olead=olead)


# Sizes that take the forms the shapes above do not: tiles on two accumulators
# (long contractions, whole and cut tiles), a cluster over 256 rows.
@pytest.mark.parametrize("M,N,K", [(1000, 8136, 2048), (1000, 8130, 2056), (512, 2048, 4096), (500, 2045, 4096)])
def test_large_forms(arx, M, N, K):
    _forward(arx, M, N, K, torch.bfloat16, "gelu")
    _forward(arx, M, N, K, torch.float16, residual=False, bias=False, z=False)


@pytest.mark.parametrize("M,N,K", [(1000, 2048, 8192), (2050, 1000, 8192), (2050, 1000, 8200)])
def test_backward_large_forms(arx, M, N, K):
    _backward(arx, M, N, K, torch.bfloat16)


# One operand by the copy engine, the other by threads.
@pytest.mark.parametrize("M,N,K", [(5, 72, 136), (300, 2047, 520), (1400, 2600, 264), (3, 200, 1000)])
@pytest.mark.parametrize("xpad,wpad", [(3, 0), (0, 3), (4, 0), (0, 4), (8, 1)])
def test_operands_of_different_alignment(arx, M, N, K, xpad, wpad):
    x, w = make((M, K), torch.bfloat16, 1), make((N, K), torch.bfloat16, 2, K ** -0.5)
    d = make((M, N), torch.bfloat16, 3)
    out, want = Out((M, N), torch.bfloat16), torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    xs, ws = strided(x, xpad), strided(w, wpad)
    arx.arx_linear(xs, ws, out.t)
    wd = _matmul(f64(x), f64(w).T.copy())
    assert_close(out, wd, _chain(K) * _matmul(np.abs(f64(x)), np.abs(f64(w)).T.copy()), "out")
    dx, dw = Out((M, K), torch.bfloat16), Out((N, K), torch.bfloat16)
    arx.arx_linear_bwd(d, xs, ws, dx=dx.t, dw=dw.t)
    torch.cuda.synchronize()
    dd, ad = f64(d), np.abs(f64(d))
    assert_close(dx, _matmul(dd, f64(w)), _chain(N) * _matmul(ad, np.abs(f64(w))), "dx")
    assert_close(dw, _matmul(dd.T.copy(), f64(x)), _chain(M) * _matmul(ad.T.copy(), np.abs(f64(x))), "dw")


@pytest.mark.parametrize("M,N", [(3, 40), (1300, 2600)])
def test_empty_contraction(arx, M, N):
    _forward(arx, M, N, 0, torch.bfloat16, "silu")


@pytest.mark.parametrize("M,N,K", [(6, 200, 256), (1300, 2600, 64)])
def test_in_place_over_the_residual(arx, M, N, K):
    x, w, r = make((M, K), torch.bfloat16, 1), make((N, K), torch.bfloat16, 2), make((M, N), torch.bfloat16, 3)
    want = torch.empty_like(r)
    arx.arx_linear(x, w, want, residual=r)
    arx.arx_linear(x, w, r, residual=r)
    assert torch.equal(bits(r), bits(want))


@pytest.mark.parametrize("M,N,K", [(3, 200, 256), (1300, 2600, 128)])
def test_infinities_and_nan_stay_in_their_rows(arx, M, N, K):
    # Padding multiplies nothing: an infinite or NaN input reaches its own row (or feature) only.
    x, w = make((M, K), torch.bfloat16, 1), make((N, K), torch.bfloat16, 2)
    clean = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    arx.arx_linear(x, w, clean)
    x[1, 5] = float("nan")
    w[7, 2] = float("inf")
    out = torch.empty_like(clean)
    arx.arx_linear(x, w, out)
    assert torch.isnan(out[1]).all() and not torch.isfinite(out[:, 7]).any()
    rows = torch.ones(M, dtype=torch.bool)
    rows[1] = False
    cols = torch.ones(N, dtype=torch.bool)
    cols[7] = False
    assert torch.equal(bits(out[rows][:, cols]), bits(clean[rows][:, cols]))


@pytest.mark.parametrize("act", ACTS)
def test_activation_limits(arx, act):
    # z = the weight itself (x = 1): infinities, the largest values, zeros.
    v = torch.tensor([0.0, -0.0, 1.0, -1.0, 88.0, -88.0, 120.0, -120.0, 6e4, -6e4, float("inf"), -float("inf"),
                      float("nan"), 3e-5, -3e-5, 10.0], dtype=torch.float16, device="cuda")
    x = torch.zeros(1, 8, dtype=torch.float16, device="cuda")
    x[0, 0] = 1
    w = torch.zeros(16, 8, dtype=torch.float16, device="cuda")
    w[:, 0] = v
    out = torch.empty(1, 16, dtype=torch.float16, device="cuda")
    arx.arx_linear(x, w, out, act=_code(arx, act))
    z = f64(v)
    with np.errstate(all="ignore"):
        want = plain.act(z, act)
    if act != "none":
        want[11] = 0.0                              # the limit at -infinity
    want[12] = np.nan
    # inf * 0 of the padding columns of w's own rows is not formed: w's other columns are 0, x's are 0.
    assert_close(out[0], want, 24 * E * (1 + np.abs(np.where(np.isfinite(z), z, 0))), act)


def _backward(arx, M, N, K, dtype, act="none", wdtype=None, pad=0, lead=0, which="xwb", copies=None):
    x = strided(make((M, K), dtype, 1), pad, lead)
    w = strided(make((N, K), dtype, 2), pad, lead)
    d = strided(make((M, N), dtype, 3), pad, lead)
    z = strided(make((M, N), dtype, 4, 1.5), pad, lead) if act != "none" else None
    dx = Out((M, K), dtype, pad, lead) if "x" in which else None
    dw = Out((N, K), dtype, pad, lead) if "w" in which else None
    db = Out((N,), wdtype or dtype) if "b" in which else None
    ws = scratch(arx.arx_linear_bwd_workspace_bytes(M, N))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    arx.arx_linear_bwd(d, x, w, dx=dx.t if dx else None, dw=dw.t if dw else None, dbias=db.t if db else None, z=z,
                       act=_code(arx, act), workspace=ws, status=status, copies=copies)
    torch.cuda.synchronize()
    assert int(status) == 0
    dz, edz = f64(d), np.zeros((M, N))
    if act != "none":
        g = plain.act_grad(f64(z), act)
        edz = np.abs(dz) * 24 * E * (1 + np.abs(g))
        dz = dz * g
    if db:
        assert_close(db, dz.sum(0), (M + 2) * E * np.abs(dz).sum(0) + edz.sum(0), "dbias")
    if act != "none":
        edz = edz + U[dtype] * np.abs(dz) + 2.0 ** -25   # dz is rounded to be an operand
    a, xa, wa = np.abs(dz), f64(x), f64(w)
    if dx:
        assert_close(dx, _matmul(dz, wa), _chain(N) * _matmul(a, np.abs(wa)) + _matmul(edz, np.abs(wa)), "dx")
    if dw:
        t = a.T.copy()
        assert_close(dw, _matmul(dz.T.copy(), xa), _chain(M) * _matmul(t, np.abs(xa)) + _matmul(edz.T.copy(), np.abs(xa)),
                     "dw")


@pytest.mark.parametrize("dtype", HALF)
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_backward(arx, M, N, K, dtype):
    _backward(arx, M, N, K, dtype)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M,N,K", [(1, 264, 128), (75, 200, 72), (1400, 1300, 1320)])
def test_backward_activations(arx, M, N, K, act):
    _backward(arx, M, N, K, torch.bfloat16, act, wdtype=torch.float32)
    _backward(arx, M, N, K, torch.float16, act)


@pytest.mark.parametrize("pad,lead", [(8, 8), (3, 0), (0, 1)])
@pytest.mark.parametrize("M,N,K", [(20, 72, 136), (1300, 1290, 1290)])
def test_backward_strides_and_alignment(arx, M, N, K, pad, lead):
    _backward(arx, M, N, K, torch.bfloat16, "gelu", pad=pad, lead=lead)


@pytest.mark.parametrize("which", ["x", "w", "b", "xb", "wb", "xw"])
def test_backward_parts(arx, which):
    _backward(arx, 70, 136, 200, torch.bfloat16, "silu", which=which)
    _backward(arx, 70, 136, 200, torch.bfloat16, "none", which=which)


def test_backward_of_no_tokens(arx):
    x, d = (torch.empty(0, n, dtype=torch.bfloat16, device="cuda") for n in (40, 24))
    w = make((24, 40), torch.bfloat16, 1)
    dw, db = Out((24, 40), torch.bfloat16), Out((24,), torch.bfloat16)
    arx.arx_linear_bwd(d, x, w, dx=torch.empty_like(x), dw=dw.t, dbias=db.t, workspace=scratch(64))
    assert_close(dw, np.zeros((24, 40)))
    assert_close(db, np.zeros(24))


def test_backward_without_an_activation_needs_no_workspace(arx):
    x, w, d = make((30, 64), torch.bfloat16, 1), make((80, 64), torch.bfloat16, 2), make((30, 80), torch.bfloat16, 3)
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    arx.arx_linear_bwd(d, x, w, dx=dx, dw=dw)
    assert_close(dx, f64(d) @ f64(w), _chain(80) * (np.abs(f64(d)) @ np.abs(f64(w))))


@pytest.mark.parametrize("act", ["gelu", "gelu_tanh", "silu"])
def test_gradients_against_differences(arx, act):
    # Directional differences of the 64-bit forward; the kernel's fp16 results
    # (u = 2^-11 each, independent over the elements) project to within u times
    # the norms, five times over.
    M, N, K, h = 24, 40, 56, 1e-4
    x, w, b = (make(s, torch.float16, i, sc) for s, i, sc in (((M, K), 1, 1.0), ((N, K), 2, K ** -0.5), ((N,), 3, 1.0)))
    g = make((M, N), torch.float16, 4)
    z, out = torch.empty(M, N, dtype=torch.float16, device="cuda"), torch.empty(M, N, dtype=torch.float16, device="cuda")
    arx.arx_linear(x, w, out, bias=b, z=z, act=_code(arx, act))
    dx, dw, db = torch.empty_like(x), torch.empty_like(w), torch.empty(N, device="cuda")
    arx.arx_linear_bwd(g, x, w, dx=dx, dw=dw, dbias=db, z=z, act=_code(arx, act),
                       workspace=scratch(arx.arx_linear_bwd_workspace_bytes(M, N)))
    X, W, B, G = f64(x), f64(w), f64(b), f64(g)
    loss = lambda X, W, B: (plain.act(X @ W.T + B, act) * G).sum()  # noqa: E731
    r = np.random.default_rng(1)
    for got, at in ((f64(dx), 0), (f64(dw), 1), (f64(db), 2)):
        for _ in range(4):
            v = r.normal(size=got.shape)
            up = [X, W, B]
            dn = [X, W, B]
            up[at], dn[at] = up[at] + h * v, dn[at] - h * v
            diff = (loss(*up) - loss(*dn)) / (2 * h)
            lim = 5 * 2 * U[torch.float16] * np.sqrt((v * v).sum()) * np.sqrt((got * got).sum())
            assert abs(diff - (got * v).sum()) < lim


@pytest.mark.parametrize("M,N,K", [(1, 2048, 4096), (100, 300, 2000), (1500, 2600, 512)])
def test_same_bits_on_every_run_and_plan(arx, M, N, K):
    x, w = make((M, K), torch.bfloat16, 1), make((N, K), torch.bfloat16, 2)
    outs = []
    for i in range(4):
        o = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
        if i < 3:
            arx.arx_linear(x, w, o, act=arx.ARX_ACT_GELU)
        else:
            arx.arx_linear_plan(x, w, o, act=arx.ARX_ACT_GELU)()
        outs.append(bits(o))
    assert all(torch.equal(o, outs[0]) for o in outs[1:])


def test_back_to_back_products_read_their_predecessors_output(arx):
    # Each call's input is the call before's output, without a synchronisation.
    n, layers = 512, 12
    ws = [make((n, n), torch.bfloat16, 50 + i, n ** -0.5) for i in range(layers)]
    for M in (1, 64, 4000):
        a = make((M, n), torch.bfloat16, 1)
        chained, waited = a, a
        for w in ws:
            o = torch.empty_like(a)
            arx.arx_linear(chained, w, o)
            chained = o
        torch.cuda.synchronize()
        for w in ws:
            o = torch.empty_like(a)
            arx.arx_linear(waited, w, o)
            torch.cuda.synchronize()
            waited = o
        assert torch.equal(bits(chained), bits(waited))


def test_two_streams_at_once(arx):
    x, w = make((64, 1024), torch.bfloat16, 1), make((2048, 1024), torch.bfloat16, 2)
    big = make((3000, 1024), torch.bfloat16, 3)
    want, wbig = torch.empty(64, 2048, dtype=torch.bfloat16, device="cuda"), torch.empty(3000, 2048, dtype=torch.bfloat16,
                                                                                      device="cuda")
    arx.arx_linear(x, w, want)
    arx.arx_linear(big, w, wbig)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    a, b = torch.empty_like(want), torch.empty_like(wbig)
    for _ in range(50):
        arx.arx_linear(x, w, a, stream=s1)
        arx.arx_linear(big, w, b, stream=s2)
    torch.cuda.synchronize()
    assert torch.equal(bits(a), bits(want)) and torch.equal(bits(b), bits(wbig))


def test_graph(arx):
    x, w = make((8, 512), torch.bfloat16, 1), make((640, 512), torch.bfloat16, 2)
    o, want = (torch.empty(8, 640, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    arx.arx_linear(x, w, o)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        arx.arx_linear(x, w, o)
    x.mul_(2)
    g.replay()
    arx.arx_linear(x, w, want)
    torch.cuda.synchronize()
    assert torch.equal(bits(o), bits(want))


def test_offsets_past_32_bits(arx):
    ld, K, N = (1 << 30) + 8, 256, 96
    buf = torch.empty(4 * ld + K, dtype=torch.bfloat16, device="cuda")
    x = buf.as_strided((5, K), (ld, 1))
    src, w = make((5, K), torch.bfloat16, 4), make((N, K), torch.bfloat16, 5)
    x.copy_(src)
    got, want = (torch.empty(5, N, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    arx.arx_linear(x, w, got)
    arx.arx_linear(src, w, want)
    assert torch.equal(bits(got), bits(want))
    far = buf.as_strided((5, N), (ld, 1))
    arx.arx_linear(src, w, far)
    assert torch.equal(bits(far), bits(want))


# Sizes at which operands off 16 bytes are copied to aligned rows, if there is a buffer.
COPIED = [(300, 2047, 4099), (1003, 2044, 4100), (1300, 2600, 1026)]


@pytest.mark.parametrize("copies", [None, False])
@pytest.mark.parametrize("M,N,K", COPIED)
@pytest.mark.parametrize("pad,lead", [(0, 0), (0, 1), (3, 2), (5, 7)])
def test_operands_copied_to_aligned_rows_or_loaded_by_threads(arx, M, N, K, pad, lead, copies):
    _forward(arx, M, N, K, torch.float16, "silu", pad=pad, lead=lead, copies=copies)
    _backward(arx, M, N, K, torch.bfloat16, "gelu", pad=pad, lead=lead, copies=copies)


@pytest.mark.parametrize("K", [1024, 1025, 1030, 1031, 1535, 1537])
@pytest.mark.parametrize("xlead,wlead", [(1, 1), (0, 3), (2, 5), (7, 4)])
def test_copied_operands_give_the_bits_of_aligned_ones(arx, K, xlead, wlead):
    M, N = 1300, 2600
    x, w = make((M, K), torch.bfloat16, 1), make((N, K), torch.bfloat16, 2)
    up = -K % 8
    got, want = Out((M, N), torch.bfloat16), Out((M, N), torch.bfloat16)
    xo, wo = strided(x, up, xlead), strided(w, up, wlead)
    plan = arx.arx_linear_plan(xo, wo, got.t)
    assert plan._args.copies_bytes == arx.arx_linear_copies_bytes(xo, wo) > 0
    plan()
    arx.arx_linear(strided(x, up), strided(w, up), want.t)
    assert torch.equal(bits(got.t), bits(want.t))
    got.check_guards()


def test_a_row_past_its_end_is_not_read(arx):
    # NaN around and between the rows of both operands.
    M, N, K, ld = 1300, 2600, 1027, 1031
    buf = [torch.full((n * ld + 9,), float("nan"), dtype=torch.bfloat16, device="cuda") for n in (M, N)]
    x, w = (b[5:5 + n * ld].view(n, ld)[:, :K] for b, n in zip(buf, (M, N)))
    x.copy_(make((M, K), torch.bfloat16, 1))
    w.copy_(make((N, K), torch.bfloat16, 2))
    for copies in (None, False):
        o = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
        dx, dw = torch.empty(M, K, dtype=torch.bfloat16, device="cuda"), torch.empty(N, K, dtype=torch.bfloat16, device="cuda")
        arx.arx_linear(x, w, o, copies=copies)
        arx.arx_linear_bwd(o, x, w, dx=dx, dw=dw, copies=copies)
        assert bool(torch.isfinite(o).all()) and bool(torch.isfinite(dx).all()) and bool(torch.isfinite(dw).all())


def test_copies_on_a_side_stream_and_in_a_graph(arx):
    M, N, K = COPIED[0]
    x, w = make((M, K), torch.bfloat16, 1), make((N, K), torch.bfloat16, 2)
    want, a, b, c = (torch.empty(M, N, dtype=torch.bfloat16, device="cuda") for _ in range(4))
    arx.arx_linear(x, w, want)
    buf = torch.empty(arx.arx_linear_copies_bytes(x, w), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(20):
        arx.arx_linear(x, w, a, stream=side)
        arx.arx_linear(x, w, b, copies=buf)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        arx.arx_linear(x, w, c)
    g.replay()
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(bits(t), bits(want)) for t in (a, b, c))


def test_large_copies(arx):
    # Rows of x past an offset of 2^32 elements, one element off alignment.
    M, N, K, ld = 300, 2047, 4099, 1 << 24
    buf = torch.zeros(M * ld + 1, dtype=torch.bfloat16, device="cuda")
    x = buf[1:].as_strided((M, K), (ld, 1), 1)
    src, w = make((M, K), torch.bfloat16, 4), make((N, K), torch.bfloat16, 5)
    x.copy_(src)
    got, want = (torch.empty(M, N, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    assert arx.arx_linear_copies_bytes(x, w) > 0
    arx.arx_linear(x, w, got)
    arx.arx_linear(src, w, want)
    assert torch.equal(bits(got), bits(want))
