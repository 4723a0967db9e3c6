"""Root-mean-square norm on the GPU: forward with the residual's addition and the 8-bit
output, its end of the rank-order reduce, and the backward pass, against the 64-bit
formulas.

Tolerances: a sum of squares is a chain of at most ``chain(cols)`` additions, so rstd is
within half of that many units (and four for the mean, the root and the quotient); h's own
additions enter y and rstd as they are; every product adds a unit.  q is within half a step
of e4m3: 2^-4 of a normal number, 2^-10 of a subnormal one.
"""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import gated_plain as plain  # noqa: E402
from ops_gpu import E, TYPES, Out, assert_close, bits, f64, make, scratch, strided  # noqa: E402

pytestmark = pytest.mark.gpu
BF, HALF, F32 = TYPES
Q8 = torch.float8_e4m3fn
WIDTHS = [1, 7, 8, 200, 256, 257, 264, 1000, 1024, 1032, 2048, 2050, 2056, 4096, 4099, 4104, 5003, 5128, 8192, 8193, 8200,
          12288, 16384, 16385, 16392, 20001]


def chain(cols):
    return 80 + cols // 512  # a thread's own terms, its warp's and the warps'


class OutQ:
    """An 8-bit output between guard bytes."""

    def __init__(self, rows, cols, pad=0, lead=0):
        self.buf = torch.full((64 + lead + rows * (cols + pad) + 64,), 0x55, dtype=torch.uint8, device="cuda")
        body = self.buf[64 + lead:64 + lead + rows * (cols + pad)].view(rows, cols + pad)
        self.t = body[:, :cols].view(Q8) if pad else body.view(Q8)
        self.rest = torch.ones_like(self.buf, dtype=torch.bool)
        self.rest[64 + lead:64 + lead + rows * (cols + pad)].view(rows, cols + pad)[:, :cols] = False

    def check_guards(self):
        assert bool((self.buf[self.rest] == 0x55).all()), "wrote outside q"


def check(parts, weight, eps, h=None, y=None, q=None, scale=None, rstd=None):
    """Outputs against the sum of ``parts`` (64-bit arrays, in order of addition) and its norm."""
    total, size = sum(parts), sum(np.abs(p) for p in parts)
    cols = total.shape[1]
    dh = (len(parts) - 1) * E * size
    want, want_s, want_r = plain.rms_norm(total, weight, eps)
    w = 1.0 if weight is None else np.abs(weight)
    ss = (total * total).sum(1) + eps * cols
    rel = (chain(cols) / 2 + 4) * E + np.sqrt((dh * dh).sum(1) / ss)  # of rstd
    err = np.abs(want) * (rel[:, None] + 3 * E) + dh * want_r[:, None] * w
    if h is not None:
        assert_close(h, total, dh, "h")
    if y is not None:
        assert_close(y, want, err, "y")
    if rstd is not None:
        assert_close(rstd, want_r, want_r * rel, "rstd")
    if q is not None:
        q.check_guards()
        err_s = err.max(1) / plain.TOP + 4 * E * want_s
        assert_close(scale, want_s, err_s, "scale")
        s = f64(scale.t if isinstance(scale, Out) else scale)[:, None]
        v = want / s
        got = f64(q.t.float())
        lim = 2.0 ** -4 * np.abs(v) + 2.0 ** -10 + (err / s + 2 * E * np.abs(v)) * (1 + 2.0 ** -4)
        assert (np.abs(got - v) <= lim).all(), f"q: off by {np.max(np.abs(got - v) / lim)} of the limit"
        assert (np.abs(got) <= plain.TOP).all()


def forward(arx, rows, cols, dtype, wdtype=None, res=True, form="both", stats=True, pads=(0, 0, 0, 0, 0), lead=0, seed=0,
            eps=1e-6, scale=1.0):
    """x, residual, h, y, q padded by ``pads``."""
    x = strided(make((rows, cols), dtype, seed, scale, 0.1 * scale), pads[0], lead)
    r = strided(make((rows, cols), dtype, seed + 1, scale), pads[1], lead) if res else None
    w = make((cols,), wdtype, seed + 2, 0.2, 1.0) if wdtype else None
    h = Out((rows, cols), dtype, pads[2], lead) if res else None
    y = Out((rows, cols), dtype, pads[3], lead) if form != "q" else None
    q = OutQ(rows, cols, pads[4], lead) if form != "y" else None
    s = Out((rows,), F32) if form != "y" else None
    rstd = Out((rows,), F32) if stats else None
    t = lambda o: None if o is None else o.t  # noqa: E731
    arx.arx_rms_norm(x, t(y), residual=r, h=t(h), weight=w, q=t(q), scale=t(s), rstd=t(rstd), eps=eps)
    torch.cuda.synchronize()
    check([f64(x)] + ([f64(r)] if res else []), f64(w), eps, h, y, q, s, rstd)


@pytest.mark.parametrize("cols", WIDTHS)
@pytest.mark.parametrize("dtype", TYPES, ids=str)
def test_forward_widths(arx, dtype, cols):
    for rows, form in ((1, "both"), (5, "q"), (6, "y")):
        forward(arx, rows, cols, dtype, wdtype=dtype if rows == 1 else F32, res=rows != 6, form=form, seed=cols)


@pytest.mark.parametrize("pads", [(8, 0, 8, 0, 8), (3, 0, 0, 0, 0), (0, 5, 0, 0, 0), (0, 0, 1, 0, 0), (0, 0, 0, 7, 0),
                                  (0, 0, 0, 0, 3), (0, 0, 0, 0, 16)])
@pytest.mark.parametrize("cols", [264, 1000, 4104])
def test_forward_strides(arx, cols, pads):
    forward(arx, 5, cols, BF, wdtype=BF, pads=pads)
    forward(arx, 4, cols, F32, wdtype=F32, pads=pads, lead=1)


@pytest.mark.parametrize("cols", [6001, 12001])
def test_16_bit_rows_that_leave_the_range(arx, cols):
    # As above, in bf16 and by units that lie alike: zeros, tiny numbers, NaN, and an infinity.
    x, w = make((5, cols), BF, 1), make((cols,), BF, 2, 0.2, 1.0)
    x[0], x[1] = 0.0, x[1] * 2.0 ** -100
    y, q, s = Out(x.shape, BF), OutQ(*x.shape), Out((5,), F32)
    arx.arx_rms_norm(x, y.t, weight=w, q=q.t, scale=s.t)
    check([f64(x)], f64(w), 1e-6, None, y, q, s)
    assert float(s.t[0]) == 1.0 and not bool(q.t[0].float().any())
    x[2, cols - 1], x[3, 0] = float("nan"), float("inf")
    arx.arx_rms_norm(x, y.t, weight=w, q=q.t, scale=s.t)
    for row in (2, 3):
        assert bool(torch.isnan(s.t[row])) and bool(torch.isnan(q.t[row].float()).all())
    assert bool(torch.isnan(y.t[2]).all()) and bool(torch.isnan(y.t[3, 0])) and not bool(y.t[3, 1:].any())
    assert bool(torch.isfinite(y.t[4]).all()) and bool(torch.isfinite(s.t[4]))


@pytest.mark.parametrize("rows,cols", [(609, 4096), (2433, 1024), (5000, 264), (1300, 8192), (1000, 4099), (700, 5000),
                                       (3000, 2048), (9000, 256), (700, 16384), (2500, 4096), (2440, 5000), (2440, 8192),
                                       (700, 8191), (100, 12001), (400, 12288), (2000, 500)])
@pytest.mark.parametrize("dtype", TYPES, ids=str)
def test_forward_many_rows(arx, dtype, rows, cols):
    forward(arx, rows, cols, dtype, wdtype=F32, seed=rows)
    forward(arx, rows, cols, dtype, wdtype=dtype, res=False, form="y", stats=False, seed=rows)
    forward(arx, rows, cols, dtype, wdtype=dtype, form="q", stats=False, seed=rows)


@pytest.mark.parametrize("cols", [256, 1000, 4096, 4099, 20001])
def test_rows_that_leave_the_range(arx, cols):
    """Rows of zeros, of one value, tiny and large ones, and with infinities and NaN."""
    rows = []
    r = np.random.default_rng(1)
    rows.append(np.zeros(cols))
    rows.append(np.eye(1, cols, cols // 2)[0] * 3.0)
    rows.append(r.normal(size=cols) * 1e-24)        # squares are 0 in 32 bits; eps alone counts
    rows.append(r.normal(size=cols) * 1e-42)        # subnormal numbers
    rows.append(r.normal(size=cols) * 1e16)
    rows.append(np.full(cols, -2.5))
    x = torch.tensor(np.array(rows), dtype=torch.float32, device="cuda")
    y, q, s, rstd = Out(x.shape, F32), OutQ(*x.shape), Out((len(rows),), F32), Out((len(rows),), F32)
    arx.arx_rms_norm(x, y.t, q=q.t, scale=s.t, rstd=rstd.t, eps=1e-6)
    # (Squares below the range count as 0: at most 2^-149 each, against eps.)
    check([f64(x)], None, 1e-6, None, y, q, s, rstd)
    assert float(s.t[0]) == 1.0 and not bool(q.t[0].float().any())
    x[0, cols // 3] = float("nan")
    x[1, 0] = float("inf")
    arx.arx_rms_norm(x, y.t, q=q.t, scale=s.t, rstd=rstd.t, eps=1e-6)
    for row in (0, 1):
        assert bool(torch.isnan(s.t[row])) and bool(torch.isnan(q.t[row].float()).all())
    assert bool(torch.isnan(y.t[0]).all()) and bool(torch.isnan(y.t[1, 0])) and not bool(y.t[1, 1:].any())
    assert bool(torch.isfinite(y.t[2:]).all()) and bool(torch.isfinite(s.t[2:]).all())


@pytest.mark.parametrize("cols", [1000, 4096, 4099, 20001])
def test_a_row_beyond_32_bit_squares(arx, cols):
    # The sum of squares is infinite and rstd 0: y is 0, and q's scale that of a row of zeros.
    x = torch.full((2, cols), 1e25, device="cuda")
    w = torch.full((cols,), 1e15, device="cuda")  # x * w is beyond the range too
    y, q, s = torch.empty_like(x), torch.empty(2, cols, dtype=Q8, device="cuda"), torch.empty(2, device="cuda")
    arx.arx_rms_norm(x, y, weight=w, q=q, scale=s)
    assert not bool(y.any()) and not bool(q.float().any()) and bool((s == 1).all())


@pytest.mark.parametrize("cols", [4096, 8192, 5000])
def test_in_place_through_the_ring(arx, cols):
    x, r, w = make((2500, cols), BF, 1), make((2500, cols), BF, 2), make((cols,), BF, 3, 0.2, 1)
    want_h, want_y = torch.empty_like(x), torch.empty_like(x)
    arx.arx_rms_norm(x, want_y, residual=r, h=want_h, weight=w)
    arx.arx_rms_norm(x, r, residual=r, h=x, weight=w)
    assert torch.equal(r, want_y) and torch.equal(x, want_h)


def test_h_without_a_residual_is_x(arx):
    x = make((5, 1000), BF, 1)
    h, y, want = (torch.empty_like(x) for _ in range(3))
    arx.arx_rms_norm(x, y, h=h)
    arx.arx_rms_norm(x, want)
    assert torch.equal(h, x) and torch.equal(y, want)


@pytest.mark.parametrize("lead", range(8))
@pytest.mark.parametrize("cols", [6000, 8177, 8185, 9001])
def test_units_that_lie_alike(arx, cols, lead):
    # Contiguous matrices that begin `lead` elements after 16 bytes, with weights on 16 bytes, whole
    # units or not; and one that begins elsewhere.
    forward(arx, 3, cols, BF, wdtype=BF, lead=lead)
    forward(arx, 4, cols, torch.float16, wdtype=torch.float16, lead=lead, res=False, form="y")
    forward(arx, 2, cols, BF, wdtype=BF, lead=lead, pads=(0, 1, 0, 0, 0))


@pytest.mark.parametrize("cols", [1000, 4096, 4099, 6001, 12001, 20001])
def test_in_place(arx, cols):
    x, r, w = make((7, cols), BF, 1), make((7, cols), BF, 2), make((cols,), BF, 3, 0.2, 1)
    want_h, want_y = torch.empty_like(x), torch.empty_like(x)
    arx.arx_rms_norm(x, want_y, residual=r, h=want_h, weight=w)
    for hy in ((0, 1), (1, 0), (0, None), (1, None), (None, 0), (None, 1)):
        x2, r2, new = x.clone(), r.clone(), torch.empty_like(x)
        h, y = ((x2, r2)[k] if k is not None else None for k in hy)
        y = new if y is None else y
        arx.arx_rms_norm(x2, y, residual=r2, h=h, weight=w)
        assert torch.equal(y, want_y) and (h is None or torch.equal(h, want_h))


@pytest.mark.parametrize("cols", [200, 1000, 2048, 4096, 4099, 8192, 16384, 20001])
@pytest.mark.parametrize("W", [1, 2, 3, 4, 5, 6, 7, 8])
def test_reduce_forward(arx, W, cols):
    for rows, form, res in ((3, "both", True), (9, "q", True), (2, "y", False)):
        slots = [make((rows, cols), BF, 10 + k) for k in range(W)]
        r = make((rows, cols), BF, 1) if res else None
        w = make((cols,), BF, 2, 0.2, 1.0)
        h = Out((rows, cols), BF)
        y = Out((rows, cols), BF) if form != "q" else None
        q, s = (OutQ(rows, cols, pad=0 if rows == 3 else 8), Out((rows,), F32)) if form != "y" else (None, None)
        rstd = Out((rows,), F32)
        arx.arx_reduce_rms_norm(slots, h.t, y and y.t, residual=r, weight=w, q=q and q.t, scale=s and s.t, rstd=rstd.t)
        check([f64(t) for t in slots] + ([f64(r)] if res else []), f64(w), 1e-6, h, y, q, s, rstd)


@pytest.mark.parametrize("rows,cols", [(700, 4096), (1300, 1024), (3000, 264), (400, 8192), (500, 4100), (2500, 4096),
                                       (2440, 5120), (800, 8192), (400, 12288), (700, 6001)])
@pytest.mark.parametrize("W", [2, 4, 5, 8])
def test_reduce_many_rows(arx, W, rows, cols):
    slots = [make((rows, cols), BF, 10 + k) for k in range(W)]
    r, w = make((rows, cols), BF, 1), make((cols,), BF, 2, 0.2, 1.0)
    h, y, q, s, rstd = Out((rows, cols), BF), Out((rows, cols), BF), OutQ(rows, cols), Out((rows,), F32), Out((rows,), F32)
    arx.arx_reduce_rms_norm(slots, h.t, y.t, residual=r, weight=w, q=q.t, scale=s.t, rstd=rstd.t)
    check([f64(t) for t in slots] + [f64(r)], f64(w), 1e-6, h, y, q, s, rstd)
    h2, y2 = Out((rows, cols), BF), Out((rows, cols), BF)  # without q, which other kernels may take
    arx.arx_reduce_rms_norm(slots, h2.t, y2.t, residual=r, weight=w)
    check([f64(t) for t in slots] + [f64(r)], f64(w), 1e-6, h2, y2)


def test_reduce_is_the_reduce_and_then_the_norm(arx):
    # Slots whose sum is exact in bf16: the fused form and its parts give the same bits.
    rows, cols, W = 6, 4096, 4
    g = torch.Generator(device="cuda").manual_seed(5)
    slots = [torch.randint(-8, 9, (rows, cols), generator=g, device="cuda").to(BF) for _ in range(W)]
    r, w = torch.randint(-8, 9, (rows, cols), generator=g, device="cuda").to(BF), make((cols,), BF, 2, 0.2, 1.0)
    total = torch.empty_like(r)
    arx.arx_reduce(slots, total)
    a = [torch.empty_like(r) for _ in range(4)]
    s = [torch.empty(rows, device="cuda") for _ in range(2)]
    q = [torch.empty(rows, cols, dtype=Q8, device="cuda") for _ in range(2)]
    arx.arx_rms_norm(total, a[0], residual=r, h=a[1], weight=w, q=q[0], scale=s[0])
    arx.arx_reduce_rms_norm(slots, a[3], a[2], residual=r, weight=w, q=q[1], scale=s[1])
    assert torch.equal(a[0], a[2]) and torch.equal(a[1], a[3]) and torch.equal(s[0], s[1])
    assert torch.equal(bits(q[0]), bits(q[1]))


@pytest.mark.parametrize("cols", [1000, 4096, 4099, 6001, 12001, 20001])
def test_reduce_in_place(arx, cols):
    slots, r, w = [make((5, cols), BF, k) for k in range(3)], make((5, cols), BF, 9), make((cols,), BF, 8, 0.2, 1)
    want = torch.empty_like(r), torch.empty_like(r)
    arx.arx_reduce_rms_norm(slots, *want, residual=r, weight=w)
    for hy in ((0, 2), (1, 3), (3, 0)):
        at = [t.clone() for t in slots] + [r.clone()]
        arx.arx_reduce_rms_norm(at[:3], at[hy[0]], at[hy[1]], residual=at[3], weight=w)
        assert torch.equal(at[hy[0]], want[0]) and torch.equal(at[hy[1]], want[1])
    same = slots[0]  # one buffer for every rank
    arx.arx_reduce_rms_norm([same, same], want[0], want[1])
    check([f64(same)] * 2, None, 1e-6, want[0], want[1])


def backward(arx, rows, cols, dtype, wdtype=None, dres=True, pads=(0, 0, 0, 0), lead=0, seed=0, dx=True, dw=True):
    """dy, h, dresidual and dx padded by ``pads``."""
    h = strided(make((rows, cols), dtype, seed, 1.0, 0.1), pads[1], lead)
    dy = strided(make((rows, cols), dtype, seed + 1), pads[0], lead)
    dr = strided(make((rows, cols), dtype, seed + 2), pads[2], lead) if dres else None
    w = make((cols,), wdtype, seed + 3, 0.2, 1.0) if wdtype else None
    rstd = torch.rsqrt(h.float().square().mean(1) + 1e-6)
    dxo = Out((rows, cols), dtype, pads[3], lead) if dx else None
    dwo = Out((cols,), wdtype or dtype) if dw else None
    ws = scratch(arx.arx_rms_norm_bwd_workspace_bytes(rows, cols))
    arx.arx_rms_norm_bwd(dy, h, rstd, dxo and dxo.t, weight=w, dresidual=dr, dweight=dwo and dwo.t, workspace=ws)
    D, H, R, W = f64(dy), f64(h), f64(rstd), f64(w)
    want, want_w = plain.rms_norm_bwd(D, H, R, W, f64(dr))
    v, n = D * (1.0 if W is None else W), H * R[:, None]
    if dx:
        mean = (v * n).mean(1, keepdims=True)
        dm = ((chain(cols) + 4) * E * np.abs(v * n).mean(1, keepdims=True))
        err = R[:, None] * (4 * E * np.abs(v) + np.abs(n) * (dm + 6 * E * np.abs(mean))) + 2 * E * np.abs(want)
        assert_close(dxo, want, err, "dx")
    if dw:
        assert_close(dwo, want_w, (rows + 70) * E * np.abs(D * n).sum(0), "dweight")


@pytest.mark.parametrize("cols", WIDTHS)
@pytest.mark.parametrize("dtype", TYPES, ids=str)
def test_backward_widths(arx, dtype, cols):
    for rows in (1, 5):
        backward(arx, rows, cols, dtype, wdtype=dtype if rows == 1 else F32, dres=rows == 5, seed=cols)


@pytest.mark.parametrize("pads", [(8, 0, 8, 0), (3, 0, 0, 0), (0, 5, 0, 0), (0, 0, 1, 0), (0, 0, 0, 7)])
@pytest.mark.parametrize("cols", [264, 1000, 4104])
def test_backward_strides(arx, cols, pads):
    backward(arx, 5, cols, BF, wdtype=BF, pads=pads)
    backward(arx, 4, cols, F32, wdtype=F32, pads=pads, lead=1)


@pytest.mark.parametrize("rows,cols", [(1300, 4096), (2600, 1024), (9000, 264), (700, 8192), (1000, 4099), (700, 5003),
                                       (3000, 2048), (700, 16384), (200, 20001), (400, 12288), (400, 12001), (700, 8191)])
@pytest.mark.parametrize("dtype", TYPES, ids=str)
def test_backward_many_rows(arx, dtype, rows, cols):
    backward(arx, rows, cols, dtype, wdtype=F32, seed=rows)
    backward(arx, rows, cols, dtype, dres=False, dw=False, seed=rows)
    backward(arx, rows, cols, dtype, wdtype=dtype, dx=False, seed=rows)


def test_backward_against_differences(arx):
    # The gradient of sum(y dy) by central differences of the 32-bit forward: the step's square
    # times a third derivative of about 1, and the forward's rounding (64 terms of about 1) over the step.
    rows, cols, step = 3, 64, 1e-2
    x, w, dy = make((rows, cols), F32, 1), make((cols,), F32, 2, 0.2, 1.0), make((rows, cols), F32, 3)
    y, rstd, dx, dw = torch.empty_like(x), torch.empty(rows, device="cuda"), torch.empty_like(x), torch.empty_like(w)
    loss = lambda a, b: (arx.arx_rms_norm(a, y, weight=b), float((y.double() * dy.double()).sum()))[1]  # noqa: E731
    arx.arx_rms_norm(x, y, weight=w, rstd=rstd)
    ws = scratch(arx.arx_rms_norm_bwd_workspace_bytes(rows, cols))
    arx.arx_rms_norm_bwd(dy, x, rstd, dx, weight=w, dweight=dw, workspace=ws)
    for i, j in ((0, 0), (1, 17), (2, 63)):
        e = torch.zeros_like(x)
        e[i, j] = step
        assert abs((loss(x + e, w) - loss(x - e, w)) / (2 * step) - float(dx[i, j])) < 2e-3
    for j in (0, 40):
        e = torch.zeros_like(w)
        e[j] = step
        assert abs((loss(x, w + e) - loss(x, w - e)) / (2 * step) - float(dw[j])) < 2e-3


@pytest.mark.parametrize("cols", [264, 4096, 4099, 20001])
def test_backward_in_place(arx, cols):
    dy, h, dr = (make((40, cols), BF, k) for k in range(3))
    rstd = torch.rsqrt(h.float().square().mean(1))
    want, want_w = torch.empty_like(dy), torch.empty(cols, dtype=BF, device="cuda")
    ws = scratch(arx.arx_rms_norm_bwd_workspace_bytes(40, cols))
    arx.arx_rms_norm_bwd(dy, h, rstd, want, dresidual=dr, dweight=want_w, workspace=ws)
    for k in range(3):
        t, dw = [dy.clone(), h.clone(), dr.clone()], torch.empty_like(want_w)
        arx.arx_rms_norm_bwd(t[0], t[1], rstd, t[k], dresidual=t[2], dweight=dw, workspace=ws)
        assert torch.equal(t[k], want) and torch.equal(dw, want_w)


def test_empty(arx):
    none, w = torch.empty(0, 64, dtype=BF, device="cuda"), torch.full((64,), 3.0, device="cuda")
    arx.arx_rms_norm(none, none.clone())
    arx.arx_rms_norm_bwd(none, none.clone(), torch.empty(0, device="cuda"), dweight=w, workspace=scratch(16))
    assert not bool(w.any())


def test_same_bits_on_side_streams_and_in_graphs(arx):
    rows, cols = 700, 4096
    slots, r = [make((rows, cols), BF, k) for k in range(3)], make((rows, cols), BF, 9)
    w, dy = make((cols,), F32, 5, 0.2, 1.0), make((rows, cols), BF, 6)

    def buffers():
        n = lambda d=BF: torch.empty(rows, cols, dtype=d, device="cuda")  # noqa: E731
        return {"h": n(), "y": n(), "q": n(Q8), "s": torch.empty(rows, device="cuda"), "rstd": torch.empty(rows, device="cuda"),
                "y2": n(), "h2": n(), "dx": n(), "dw": torch.empty(cols, device="cuda"),
                "ws": scratch(arx.arx_rms_norm_bwd_workspace_bytes(rows, cols))}

    def step(b):
        arx.arx_reduce_rms_norm(slots, b["h"], b["y"], residual=r, q=b["q"], scale=b["s"], rstd=b["rstd"])
        arx.arx_rms_norm(b["y"], b["y2"], residual=b["h"], h=b["h2"], weight=w, rstd=b["rstd"])
        arx.arx_rms_norm_bwd(dy, b["h2"], b["rstd"], b["dx"], weight=w, dresidual=dy, dweight=b["dw"], workspace=b["ws"])

    want, other, captured = buffers(), buffers(), buffers()
    step(want)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
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


def test_offsets_beyond_32_bits(arx):
    # Rows 2^31 elements apart: the third starts beyond 2^32 elements.
    cols, ld = 1000, 1 << 31
    buf = torch.empty(2 * ld + cols, dtype=BF, device="cuda")
    x = torch.as_strided(buf, (3, cols), (ld, 1))
    x.copy_(make((3, cols), BF, 1))
    y = Out((3, cols), BF)
    arx.arx_rms_norm(x, y.t)
    check([f64(x)], None, 1e-6, None, y)
    rstd = torch.rsqrt(x.float().square().mean(1))
    dy, dx = make((3, cols), BF, 2), Out((3, cols), BF)
    arx.arx_rms_norm_bwd(dy, x, rstd, dx.t)
    want, _ = plain.rms_norm_bwd(f64(dy), f64(x), f64(rstd))
    assert_close(dx, want, 100 * E * (np.abs(want) + np.abs(f64(x)) * np.abs(f64(dy)).mean()), "dx")


@pytest.mark.parametrize("rows,cols", [(3, 200), (700, 1000), (40, 4096), (5, 4099), (40, 8192), (3, 12288), (3, 20001)])
def test_scale_and_q_are_the_definition_s_to_within_four_roundings(arx, rows, cols):
    # Of v = x rstd weight in 64 bits, from the rstd that was returned: the scale is within 4 2^-24 of
    # max |v| / 448, and q lies between the roundings of v / scale to either side (one 2^-24 more: the
    # way to 8 bits leads through 32).
    x, w = make((rows, cols), F32, rows), make((cols,), F32, 2, 0.2, 1.0)
    q, s, rstd = torch.empty(rows, cols, dtype=Q8, device="cuda"), *(torch.empty(rows, device="cuda") for _ in range(2))
    arx.arx_rms_norm(x, None, weight=w, q=q, scale=s, rstd=rstd)
    v = x.double() * rstd.double()[:, None] * w.double()
    most = v.abs().amax(1) / 448
    assert bool(((s.double() - most).abs() <= 4 * E * most).all())
    lo, hi = ((v / s.double()[:, None] * (1 + k * E)).clamp(-448, 448).float().to(Q8).float() for k in (-5, 5))
    got = q.float()
    assert bool((got >= torch.minimum(lo, hi)).all()) and bool((got <= torch.maximum(lo, hi)).all())
