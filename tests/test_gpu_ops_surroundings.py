"""What lies around and between rows does not reach the results, and matrices may begin anywhere.

The norm's and the gated block's inputs stand in buffers that are NaN everywhere else --
before the first row, between rows, behind the last -- and workspaces and copies are NaN
before the call: a read past a row's end, or of a workspace's padding, would turn a result
into NaN.  The reduce's slots, residual and outputs begin off 16 bytes, alike or not.
Results and tolerances are those of the operators' own tests.
"""

import pytest

torch = pytest.importorskip("torch")

import test_gpu_ops_gated as gated  # noqa: E402
import test_gpu_ops_rms as rms  # noqa: E402
from ops_gpu import Out, f64, make  # noqa: E402

pytestmark = pytest.mark.gpu
BF, F16, F32 = torch.bfloat16, torch.float16, torch.float32
Q8 = torch.float8_e4m3fn
AROUND = 64  # elements before and behind


def in_nan(t, pad, lead=0):
    """The matrix in rows ``pad`` elements longer, ``lead`` elements past 16 bytes, NaN around it."""
    r, c = t.shape
    buf = torch.full((AROUND + lead + r * (c + pad) + AROUND,), float("nan"), dtype=t.dtype, device=t.device)
    v = buf[AROUND + lead:AROUND + lead + r * (c + pad)].view(r, c + pad)[:, :c]
    v.copy_(t)
    return v


def eight_in_nan(rows, cols, seed, scale, pad=0):
    pitch = (cols + 15) // 16 * 16 + 16 * pad
    buf = torch.full((2 * AROUND + rows * pitch,), 0x7F, dtype=torch.uint8, device="cuda").view(Q8)  # NaN
    v = buf[AROUND:AROUND + rows * pitch].view(rows, pitch)[:, :cols]
    v.copy_((make((rows, cols), F32, seed) * scale).to(Q8))
    return v


def nan_bytes(n):
    return torch.full((max(n, 16),), 0xFF, dtype=torch.uint8, device="cuda")


@pytest.fixture
def surrounded(arx, monkeypatch):
    """The operators' own tests, with their inputs, workspaces and copies in NaN."""
    from deterministic_shot_all_gb300 import _ops
    for module in (gated, rms):
        monkeypatch.setattr(module, "strided", in_nan)
        monkeypatch.setattr(module, "scratch", nan_bytes)
    monkeypatch.setattr(gated, "eight", eight_in_nan)
    monkeypatch.setattr(_ops, "_buffer", lambda n, device, stream: nan_bytes(n))
    assert bool(torch.isnan(in_nan(make((2, 3), BF, 0), 1)._base).any())
    return arx


# Dot products in units and one by one, the split form, pairs; contractions that end inside
# 16 bytes, inside a stage and at its end.
@pytest.mark.parametrize("dtype", [BF, F16, Q8], ids=str)
@pytest.mark.parametrize("M,N,K", [(1, 72, 13), (1, 264, 128), (2, 136, 72), (2, 2048, 4100), (3, 8, 1), (5, 72, 129),
                                   (17, 129, 65), (65, 264, 1037), (300, 130, 200), (1300, 2600, 83), (3000, 1181, 523)])
def test_gated_forward(surrounded, M, N, K, dtype):
    gated.forward(surrounded, M, N, K, dtype)
    gated.forward(surrounded, M, N, K, dtype, pad=1, z=False)
    if dtype is not Q8:
        gated.forward(surrounded, M, N, K, dtype, pad=8, lead=8, bias=False)
        gated.forward(surrounded, M, N, K, dtype, pad=3, lead=5, opad=3, olead=1)


@pytest.mark.parametrize("dtype", [BF, F16], ids=str)
@pytest.mark.parametrize("M,N,K", [(1, 8, 8), (1, 13, 7), (5, 72, 136), (17, 129, 65), (259, 1026, 515), (1291, 2563, 130)])
def test_gated_backward(surrounded, M, N, K, dtype):
    gated.backward(surrounded, M, N, K, dtype)
    gated.backward(surrounded, M, N, K, dtype, pad=8, lead=8, bias=False)
    gated.backward(surrounded, M, N, K, dtype, pad=3, lead=5, opad=3, olead=1)


@pytest.mark.parametrize("dtype", [BF, F16, F32], ids=str)
@pytest.mark.parametrize("cols", [1, 7, 264, 1003, 2056, 4099, 5003, 6001, 8193, 12001, 16392, 20001])
def test_norm(surrounded, cols, dtype):
    for rows, pad, lead in ((1, 0, 1), (5, 8, 8), (4, 3, 5), (6, 0, 3)):
        rms.forward(surrounded, rows, cols, dtype, wdtype=dtype, pads=(pad, pad, 0, pad, pad), lead=lead)
        rms.backward(surrounded, rows, cols, dtype, wdtype=F32, pads=(pad, pad, pad, 0), lead=lead)


@pytest.mark.parametrize("rows,cols", [(2433, 264), (700, 1003), (2433, 4096), (1300, 4099), (700, 6001), (700, 8192), (400, 12001)])
def test_norm_of_many_rows(surrounded, rows, cols):
    for pad, lead in ((0, 0), (8, 8), (3, 5)):
        rms.forward(surrounded, rows, cols, BF, wdtype=BF, pads=(pad, pad, 0, 0, 0), lead=lead, form="y")
        rms.backward(surrounded, rows, cols, BF, wdtype=F32, pads=(pad, pad, pad, 0), lead=lead)


def reduce(arx, W, rows, cols, leads, form):
    """``leads``: elements past 16 bytes of the slots (in turn), the residual, h and y."""
    slots = [in_nan(make((rows, cols), BF, 10 + k), 0, leads[0][k % len(leads[0])]) for k in range(W)]
    r, w = in_nan(make((rows, cols), BF, 1), 0, leads[1]), make((cols,), BF, 2, 0.2, 1.0)
    h, rstd = Out((rows, cols), BF, 0, leads[2]), Out((rows,), F32)
    y = Out((rows, cols), BF, 0, leads[3]) if form != "q" else None
    q, s = (rms.OutQ(rows, cols), Out((rows,), F32)) if form != "y" else (None, None)
    # (A matrix seen through its buffer's middle is contiguous.)
    arx.arx_reduce_rms_norm(slots, h.t, y and y.t, residual=r, weight=w, q=q and q.t, scale=s and s.t, rstd=rstd.t)
    rms.check([f64(t) for t in slots] + [f64(r)], f64(w), 1e-6, h, y, q, s, rstd)


@pytest.mark.parametrize("leads", [((1,), 1, 1, 1), ((4,), 4, 4, 4), ((7,), 7, 7, 7), ((0, 3), 0, 0, 0), ((0,), 5, 0, 0),
                                   ((0,), 0, 1, 6), ((2, 5, 7), 1, 3, 4)], ids=str)
@pytest.mark.parametrize("cols", [200, 1000, 2050, 4099, 5003, 6001, 8177, 8192, 12001, 16384])
@pytest.mark.parametrize("W", [2, 3, 8])
def test_reduce_begins_anywhere(arx, W, cols, leads):
    reduce(arx, W, 3, cols, leads, "both")
    reduce(arx, W, 5, cols, leads, "y")


# To either side of 304 rows, where the threads to a row change.
@pytest.mark.parametrize("leads", [((3,), 3, 3, 3), ((2, 5, 7), 1, 3, 4)], ids=str)
@pytest.mark.parametrize("rows,cols", [(304, 6001), (305, 6001), (305, 8192), (305, 12001), (1217, 500), (1217, 512), (700, 1000)])
@pytest.mark.parametrize("W", [2, 3, 8])
def test_reduce_of_many_rows_begins_anywhere(arx, W, rows, cols, leads):
    for form in ("y", "q"):
        reduce(arx, W, rows, cols, leads, form)


@pytest.mark.parametrize("dtype", [BF, F32], ids=str)
@pytest.mark.parametrize("cols", [8, 200, 1000, 1024, 4096, 4099, 6001, 8192, 8200, 12001, 20001])
def test_a_row_whose_squares_vanish_without_eps(arx, cols, dtype):
    # Squares below 2^-149 add nothing: rstd is infinite, and so are y and the scale of a row
    # without zeros (columns that no element stands for, past the row's end, do not count).
    x = torch.full((3, cols), 1e-30, device="cuda").to(dtype)
    x[1] *= -1
    for form in ("both", "q"):
        y, q, s, rstd = torch.empty_like(x), rms.OutQ(3, cols), Out((3,), F32), Out((3,), F32)
        arx.arx_rms_norm(x, y if form == "both" else None, q=q.t, scale=s.t, rstd=rstd.t, eps=0.0)
        assert bool((rstd.t == float("inf")).all()) and bool((s.t == float("inf")).all())
        assert bool(torch.isnan(q.t.float()).all())
        if form == "both":
            assert bool((y[::2] == float("inf")).all()) and bool((y[1] == float("-inf")).all())
    x[2, cols // 2] = 0.0  # 0 times infinity
    q, s = rms.OutQ(3, cols), Out((3,), F32)
    arx.arx_rms_norm(x, None, q=q.t, scale=s.t, eps=0.0)
    assert bool(torch.isnan(s.t[2])) and bool((s.t[:2] == float("inf")).all())
