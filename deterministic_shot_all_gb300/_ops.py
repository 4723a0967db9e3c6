"""Binding of the operators around the reduce (``include/arx.h``, "The operators
around a sublayer's all-reduce"): matrix product with its epilogue, dropout
with bias and residual, layer norm, and the fused end of a sublayer.

Every operator has two forms: a function that checks its tensors and makes one
C call, and a plan (``arx_layer_norm_plan`` and so on) that checks them once
and makes the same C call each time it is called, for eager callers that
repeat it.  A plan keeps its tensors alive; their contents may change between
calls, their storage must not.

Matrices are tensors of two or more dimensions whose last one is contiguous
and whose leading ones collapse into one row stride; vectors are contiguous.
"""

from __future__ import annotations

import ctypes

ARX_BF16, ARX_F16, ARX_F32 = range(3)
ARX_ACT_NONE, ARX_ACT_RELU, ARX_ACT_GELU, ARX_ACT_GELU_TANH, ARX_ACT_SILU = range(5)

_vp, _u64, _i32, _f32, _f64 = ctypes.c_void_p, ctypes.c_uint64, ctypes.c_int32, ctypes.c_float, ctypes.c_double


def _struct(name, *fields):
    """Mirror of a struct of include/arx.h: (type, names) pairs in order."""
    flat = [(n, t) for t, names in fields for n in names.split()]
    return type(name, (ctypes.Structure,), {"_fields_": flat, "__doc__": f"Mirror of ``struct {name}`` in include/arx.h."})


arx_layer_norm_args = _struct(
    "arx_layer_norm_args", (_vp, "x weight bias y mean rstd"), (_u64, "rows cols ldx ldy"), (_f32, "eps"),
    (_i32, "dtype wdtype reserved"))
arx_layer_norm_bwd_args = _struct(
    "arx_layer_norm_bwd_args", (_vp, "dy x mean rstd weight dresidual dx dweight dbias workspace"),
    (_u64, "workspace_bytes rows cols lddy ldx lddresidual lddx"), (_i32, "dtype wdtype"))
arx_dropout_add_args = _struct(
    "arx_dropout_add_args", (_vp, "x bias residual out rng"), (_u64, "rows cols ldx ldresidual ldout"), (_f64, "p"),
    (_i32, "dtype wdtype"))
arx_dropout_add_bwd_args = _struct(
    "arx_dropout_add_bwd_args", (_vp, "dout dx dbias rng workspace"), (_u64, "workspace_bytes rows cols lddout lddx"),
    (_f64, "p"), (_i32, "dtype wdtype"))
arx_reduce_layer_norm_args = _struct(
    "arx_reduce_layer_norm_args", (_vp, "slots bias residual weight norm_bias h y mean rstd rng"), (_u64, "rows cols"),
    (_f64, "p"), (_f32, "eps"), (_i32, "W"))
arx_linear_args = _struct(
    "arx_linear_args", (_vp, "x w bias residual out z status copies"), (_u64, "copies_bytes M N K ldx ldw ldresidual ldout ldz"),
    (_i32, "act dtype wdtype wait_us"))
arx_linear_bwd_args = _struct(
    "arx_linear_bwd_args", (_vp, "dout z x w dx dw dbias workspace"), (_u64, "workspace_bytes"), (_vp, "status copies"),
    (_u64, "copies_bytes M N K lddout ldz ldx ldw lddx lddw"), (_i32, "act dtype wdtype wait_us"))

SIGNATURES = {
    **{f"arx_{op}": ([ctypes.POINTER(t), _vp], ctypes.c_int) for op, t in (
        ("layer_norm", arx_layer_norm_args), ("layer_norm_bwd", arx_layer_norm_bwd_args),
        ("dropout_add", arx_dropout_add_args), ("dropout_add_bwd", arx_dropout_add_bwd_args),
        ("reduce_layer_norm", arx_reduce_layer_norm_args), ("linear", arx_linear_args),
        ("linear_bwd", arx_linear_bwd_args))},
    **{f"arx_{op}_workspace_bytes": ([_u64, _u64], ctypes.c_size_t)
       for op in ("layer_norm_bwd", "dropout_add_bwd", "linear_bwd")},
    "arx_stream_capturing": ([_vp], ctypes.c_int),
    **{f"arx_{op}_copies_bytes": ([ctypes.POINTER(t)], ctypes.c_size_t) for op, t in (
        ("linear", arx_linear_args), ("linear_bwd", arx_linear_bwd_args))},
}


def _core():
    import deterministic_shot_all_gb300 as core
    return core


_DTYPES: dict = {}


def _dtype(t, name, allowed):
    if not _DTYPES:
        import torch
        _DTYPES.update({torch.bfloat16: ARX_BF16, torch.float16: ARX_F16, torch.float32: ARX_F32})
    code = _DTYPES.get(t.dtype)
    if code not in allowed:
        raise TypeError(f"{name}: {t.dtype} not supported")
    return code


def _buffer(n, device, stream):
    """n bytes of the stream's own memory (what was freed on it is not in use by another), or
    of the graph's while torch captures the stream: they live as long as the graph."""
    import torch
    if stream is None:
        return torch.empty(n, dtype=torch.uint8, device=f"cuda:{device}")
    with torch.cuda.stream(torch.cuda.ExternalStream(_core()._stream(stream))):
        return torch.empty(n, dtype=torch.uint8, device=f"cuda:{device}")


class _Marshal:
    """Fills an argument struct from tensors, checking each against the others."""

    def __init__(self, args, first, name, types):
        self.a = args
        self.refs = []
        self.dtype = first.dtype
        self.device = None  # the current device, looked up once a tensor is on a GPU
        self.own_copies = 0  # bytes of a copies buffer that the caller does not hold
        if types is not None:
            args.dtype = _dtype(first, name, types)
        self.wdtype = None

    def _on_device(self, t, name):
        if not t.is_cuda:
            raise ValueError(f"{name}: expected a CUDA tensor, got one on {t.device}")
        if self.device is None:
            import torch
            self.device = torch.cuda.current_device()
        if t.device.index != self.device:
            raise ValueError(f"{name}: on {t.device}, but the current device is cuda:{self.device}")

    def matrix(self, t, name, rows=None, cols=None, ld=None):
        """Sets field ``name`` (and ``ld<name>``) to the matrix and returns (rows, cols)."""
        if t is None:
            return None
        if t.dtype is not self.dtype:
            raise TypeError(f"{name}: expected {self.dtype}, got {t.dtype}")
        if t.dim() < 2:
            raise ValueError(f"{name}: expected a matrix, got {t.dim()} dimension(s)")
        n = t.shape[-1]
        r = 1
        for s in t.shape[:-1]:
            r *= s
        if (rows is not None and r != rows) or (cols is not None and n != cols):
            raise ValueError(f"{name}: shape {tuple(t.shape)}, the call needs [{rows}, {cols}]")
        stride = t.stride(-2) if t.shape[-2] > 1 else n
        if r * n > 0:
            if n > 1 and t.stride(-1) != 1:
                raise ValueError(f"{name}: the last dimension must be contiguous")
            # The leading dimensions have to be one run of equally spaced rows.
            step, last = None, None
            for s, d in zip(reversed(t.shape[:-1]), reversed(t.stride()[:-1])):
                if s == 1:
                    continue
                if step is None:
                    step = d
                elif d != last:
                    raise ValueError(f"{name}: rows are not equally spaced (shape {tuple(t.shape)}, "
                                     f"strides {tuple(t.stride())})")
                last = d * s
            stride = n if step is None else step
            if step is not None and step < n:
                raise ValueError(f"{name}: rows overlap (stride {step} below {n} columns)")
        self._on_device(t, name)
        setattr(self.a, name, t.data_ptr())
        setattr(self.a, ld or "ld" + name, stride)
        self.refs.append(t)
        return r, n

    def contiguous(self, t, name, rows, cols):
        """A matrix without a leading dimension in the struct; returns its address."""
        if t is None:
            return None
        if t.dtype is not self.dtype:
            raise TypeError(f"{name}: expected {self.dtype}, got {t.dtype}")
        if t.dim() < 2 or t.shape[-1] != cols or t.numel() != rows * cols:
            raise ValueError(f"{name}: shape {tuple(t.shape)}, the call needs [{rows}, {cols}]")
        if not t.is_contiguous():
            raise ValueError(f"{name}: must be contiguous")
        self._on_device(t, name)
        self.refs.append(t)
        return t.data_ptr()

    def vector(self, t, name, n, dtype=None):
        """``dtype`` None: a parameter, of the matrices' type or 32 bits, all of a call alike."""
        if t is None:
            return
        import torch
        if dtype is None:
            if t.dtype is not self.dtype and t.dtype is not torch.float32:
                raise TypeError(f"{name}: expected {self.dtype} or torch.float32, got {t.dtype}")
            if self.wdtype is not None and t.dtype is not self.wdtype:
                raise TypeError(f"{name}: {t.dtype}, but another parameter is {self.wdtype}")
            self.wdtype = t.dtype
        elif t.dtype is not dtype:
            raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
        if t.dim() != 1 or t.shape[0] != n:
            raise ValueError(f"{name}: shape {tuple(t.shape)}, the call needs [{n}]")
        if n > 1 and t.stride(0) != 1:
            raise ValueError(f"{name}: must be contiguous")
        self._on_device(t, name)
        setattr(self.a, name, t.data_ptr())
        self.refs.append(t)

    def rng(self, p, rng):
        import torch
        self.a.p = p
        if rng is None:
            return
        if rng.dtype not in (torch.int64, getattr(torch, "uint64", torch.int64)) or rng.numel() != 2:
            raise TypeError("rng: expected two 64-bit integers (seed, offset)")
        if not rng.is_contiguous():
            raise ValueError("rng: must be contiguous")
        self._on_device(rng, "rng")
        self.a.rng = rng.data_ptr()
        self.refs.append(rng)

    def status(self, t):
        if t is None:
            return
        import torch
        if t.dtype not in (torch.int32, getattr(torch, "uint32", torch.int32)) or t.numel() < 1:
            raise TypeError("status: expected one 32-bit integer")
        self._on_device(t, "status")
        self.a.status = t.data_ptr()
        self.refs.append(t)

    def workspace(self, t):
        if t is None:
            return
        if not t.is_contiguous():
            raise ValueError("workspace: must be contiguous")
        self._on_device(t, "workspace")
        self.a.workspace = t.data_ptr() or None
        self.a.workspace_bytes = t.numel() * t.element_size()
        self.refs.append(t)

    def copies(self, t, query, operands, stream):
        """``t``: a buffer, None (allocated where the call is faster with one) or False (none)."""
        if t is False:
            return
        if t is None:
            # Rows on 16 bytes need none; a leading dimension counts from the second row on.
            off = 0
            for m, name in operands:
                if m is not None:
                    off |= m.data_ptr() | (getattr(self.a, "ld" + name) * 2 if m.numel() > m.shape[-1] else 0)
            n = query(ctypes.byref(self.a)) if off & 15 else 0
            if n == 0:
                return
            self.own_copies = n
            t = _buffer(n, self.device, stream)
        elif not t.is_contiguous():
            raise ValueError("copies: must be contiguous")
        self._on_device(t, "copies")
        self.a.copies = t.data_ptr() or None
        self.a.copies_bytes = t.numel() * t.element_size()
        self.refs.append(t)

    def done(self):
        if hasattr(self.a, "wdtype"):
            self.a.wdtype = self.a.dtype if self.wdtype in (None, self.dtype) else ARX_F32
        return self


_ROW_TYPES = (ARX_BF16, ARX_F16, ARX_F32)
_PRODUCT_TYPES = (ARX_BF16, ARX_F16)


def _layer_norm(x, y, weight=None, bias=None, mean=None, rstd=None, eps=1e-5, stream=None):
    import torch
    m = _Marshal(arx_layer_norm_args(eps=eps), x, "x", _ROW_TYPES)
    rows, cols = m.matrix(x, "x")
    m.matrix(y, "y", rows, cols)
    m.vector(weight, "weight", cols)
    m.vector(bias, "bias", cols)
    m.vector(mean, "mean", rows, torch.float32)
    m.vector(rstd, "rstd", rows, torch.float32)
    m.a.rows, m.a.cols = rows, cols
    return m.done()


def _layer_norm_bwd(dy, x, mean, rstd, dx=None, weight=None, dresidual=None, dweight=None, dbias=None,
                    workspace=None, stream=None):
    import torch
    m = _Marshal(arx_layer_norm_bwd_args(), x, "x", _ROW_TYPES)
    rows, cols = m.matrix(x, "x")
    m.matrix(dy, "dy", rows, cols)
    m.matrix(dresidual, "dresidual", rows, cols)
    m.matrix(dx, "dx", rows, cols)
    m.vector(mean, "mean", rows, torch.float32)
    m.vector(rstd, "rstd", rows, torch.float32)
    for t, name in ((weight, "weight"), (dweight, "dweight"), (dbias, "dbias")):
        m.vector(t, name, cols)
    m.workspace(workspace)
    m.a.rows, m.a.cols = rows, cols
    return m.done()


def _dropout_add(x, out, p, rng=None, bias=None, residual=None, stream=None):
    m = _Marshal(arx_dropout_add_args(), x, "x", _ROW_TYPES)
    rows, cols = m.matrix(x, "x")
    m.matrix(residual, "residual", rows, cols)
    m.matrix(out, "out", rows, cols)
    m.vector(bias, "bias", cols)
    m.rng(p, rng)
    m.a.rows, m.a.cols = rows, cols
    return m.done()


def _dropout_add_bwd(dout, dx, p, rng=None, dbias=None, workspace=None, stream=None):
    m = _Marshal(arx_dropout_add_bwd_args(), dout, "dout", _ROW_TYPES)
    rows, cols = m.matrix(dout, "dout")
    m.matrix(dx, "dx", rows, cols)
    m.vector(dbias, "dbias", cols)
    m.rng(p, rng)
    m.workspace(workspace)
    m.a.rows, m.a.cols = rows, cols
    return m.done()


def _reduce_layer_norm(slots, h, y, bias=None, residual=None, weight=None, norm_bias=None, mean=None, rstd=None,
                       eps=1e-5, p=0.0, rng=None, stream=None):
    import torch
    a = arx_reduce_layer_norm_args(eps=eps)
    if y.dtype is not torch.bfloat16:
        raise TypeError(f"y: expected torch.bfloat16, got {y.dtype}")
    if y.dim() < 2:
        raise ValueError(f"y: expected a matrix, got {y.dim()} dimension(s)")
    a.cols = cols = y.shape[-1]
    a.rows = rows = y.numel() // cols if cols else 0
    m = _Marshal(a, y, "y", None)
    a.W = len(slots)
    arr = (ctypes.c_void_p * max(1, len(slots)))(*[m.contiguous(s, f"slots[{i}]", rows, cols)
                                                   for i, s in enumerate(slots)])
    a.slots = ctypes.cast(arr, _vp)
    m.refs.append(arr)
    a.residual = m.contiguous(residual, "residual", rows, cols)
    a.h = m.contiguous(h, "h", rows, cols)
    a.y = m.contiguous(y, "y", rows, cols)
    for t, name in ((bias, "bias"), (weight, "weight"), (norm_bias, "norm_bias")):
        m.vector(t, name, cols, torch.bfloat16)
    m.vector(mean, "mean", rows, torch.float32)
    m.vector(rstd, "rstd", rows, torch.float32)
    m.rng(p, rng)
    return m.done()


def _linear(x, w, out, bias=None, residual=None, z=None, act=ARX_ACT_NONE, status=None, copies=None, wait_us=0,
            stream=None):
    m = _Marshal(arx_linear_args(act=act, wait_us=wait_us), x, "x", _PRODUCT_TYPES)
    M, K = m.matrix(x, "x")
    N, _ = m.matrix(w, "w", None, K)
    m.matrix(residual, "residual", M, N)
    m.matrix(out, "out", M, N)
    m.matrix(z, "z", M, N)
    m.vector(bias, "bias", N)
    m.status(status)
    m.a.M, m.a.N, m.a.K = M, N, K
    m.copies(copies, _core().lib.arx_linear_copies_bytes, ((x, "x"), (w, "w")), stream)
    return m.done()


def _linear_bwd(dout, x, w, dx=None, dw=None, dbias=None, z=None, act=ARX_ACT_NONE, workspace=None, status=None,
                copies=None, wait_us=0, stream=None):
    m = _Marshal(arx_linear_bwd_args(act=act, wait_us=wait_us), dout, "dout", _PRODUCT_TYPES)
    M, N = m.matrix(dout, "dout")
    K = next((t.shape[-1] for t in (x, w) if t is not None), 0)
    m.matrix(z, "z", M, N)
    m.matrix(x, "x", M, K)
    m.matrix(w, "w", N, K)
    m.matrix(dx, "dx", M, K)
    m.matrix(dw, "dw", N, K)
    m.vector(dbias, "dbias", N)
    m.workspace(workspace)
    m.status(status)
    m.a.M, m.a.N, m.a.K = M, N, K
    m.copies(copies, _core().lib.arx_linear_bwd_copies_bytes, ((dout, "dout"), (x, "x"), (w, "w")), stream)
    return m.done()


class _Plan:
    """A checked call: one C call with the stored arguments each time it is called."""

    _marshal = _name = None

    def __init__(self, *args, stream=None, **kwargs):
        core = _core()
        m = type(self)._marshal(*args, stream=stream, **kwargs)
        self._args, self._refs = m.a, m.refs
        self._ref = ctypes.byref(self._args)
        self._stream = core._stream(stream)
        self._fn = getattr(core.lib, self._name)
        self._own_copies, self._device = m.own_copies, m.device

    def __call__(self) -> None:
        ref = self._ref
        # The plan's own copies end with the plan, a graph's nodes with the graph: a captured
        # call gets copies of the graph's.
        if self._own_copies and _core().lib.arx_stream_capturing(self._stream):
            t = _buffer(self._own_copies, self._device, self._stream)
            a = type(self._args).from_buffer_copy(self._args)
            a.copies = t.data_ptr()
            ref = ctypes.byref(a)
        st = self._fn(ref, self._stream)
        if st:
            _core()._check(st)


def _function(name, marshal, doc):
    """The call and its plan; ``marshal`` also gets the stream, for buffers that it allocates."""
    def call(*args, stream=None, check=True, **kwargs):
        core = _core()
        m = marshal(*args, stream=stream, **kwargs)  # holds the tensors until the call is enqueued
        st = getattr(core.lib, name)(ctypes.byref(m.a), core._stream(stream))
        del m
        if check:
            core._check(st)
        return st
    call.__name__ = call.__qualname__ = name
    call.__doc__ = doc
    plan = type(name + "_plan", (_Plan,), {"_marshal": staticmethod(marshal), "_name": name,
                                           "__doc__": f"A prepared ``{name}``: the same arguments, checked once."})
    plan.__module__ = call.__module__ = "deterministic_shot_all_gb300"
    return call, plan


arx_layer_norm, arx_layer_norm_plan = _function("arx_layer_norm", _layer_norm, """\
Enqueue y = (x - mean) * rstd * weight + bias over the rows of ``x``.

    ``arx_layer_norm(x, y, weight=None, bias=None, mean=None, rstd=None, eps=1e-5, stream=None, check=True)``

    bf16, fp16 or fp32; weight and bias of the same type or fp32.  ``y`` may be ``x``.
    ``mean`` and ``rstd``: fp32 [rows] outputs for the backward pass.
    """)
arx_layer_norm_bwd, arx_layer_norm_bwd_plan = _function("arx_layer_norm_bwd", _layer_norm_bwd, """\
Enqueue the gradients of ``arx_layer_norm``.

    ``arx_layer_norm_bwd(dy, x, mean, rstd, dx=None, weight=None, dresidual=None, dweight=None, dbias=None,
    workspace=None, stream=None, check=True)``

    ``dresidual`` is added to dx; dx may be dy, x or dresidual.  ``workspace``: a device
    tensor of ``arx_layer_norm_bwd_workspace_bytes(rows, cols)`` bytes when dweight or
    dbias is asked for.
    """)
arx_dropout_add, arx_dropout_add_plan = _function("arx_dropout_add", _dropout_add, """\
Enqueue out = residual + keep(x + bias) / (1 - p), the mask from a counter-based generator.

    ``arx_dropout_add(x, out, p, rng=None, bias=None, residual=None, stream=None, check=True)``

    ``rng``: a device tensor of two int64, seed and offset, read when the kernel runs.
    ``out`` may be ``x`` or ``residual``.
    """)
arx_dropout_add_bwd, arx_dropout_add_bwd_plan = _function("arx_dropout_add_bwd", _dropout_add_bwd, """\
Enqueue dx = keep(dout) / (1 - p) with the forward's mask, and dbias, its sum over rows.

    ``arx_dropout_add_bwd(dout, dx, p, rng=None, dbias=None, workspace=None, stream=None, check=True)``

    dx may be dout or None; ``workspace`` of ``arx_dropout_add_bwd_workspace_bytes(rows,
    cols)`` bytes when dbias is asked for.
    """)
arx_reduce_layer_norm, arx_reduce_layer_norm_plan = _function("arx_reduce_layer_norm", _reduce_layer_norm, """\
Enqueue h = residual + keep(rank-order sum of slots + bias) / (1 - p), y = layer norm of h.

    ``arx_reduce_layer_norm(slots, h, y, bias=None, residual=None, weight=None, norm_bias=None, mean=None,
    rstd=None, eps=1e-5, p=0.0, rng=None, stream=None, check=True)``

    bf16, contiguous; ``h`` (may be None) and ``y`` may each be a slot or the residual.
    """)
arx_linear, arx_linear_plan = _function("arx_linear", _linear, """\
Enqueue out = act(x w^T + bias) + residual on the tensor cores.

    ``arx_linear(x, w, out, bias=None, residual=None, z=None, act=ARX_ACT_NONE, status=None, copies=None,
    wait_us=0, stream=None, check=True)``

    bf16 or fp16; x [M, K], w [N, K]; bias of the same type or fp32.  ``z`` receives
    x w^T + bias for the backward pass.  ``out`` may be ``residual``.  ``copies``: a buffer of
    ``arx_linear_copies_bytes`` bytes for operands whose rows are off 16 bytes, which calls
    that run in turn may share; None: one is allocated on the stream where the call is faster
    with it; False: none.  With None a plan keeps a buffer of its own for eager calls, of the
    operands' size (25 MB for [1003, 4100] x [2044, 4100] of 16 bits), and a call that torch
    captures into a graph takes one of the graph's memory, so that neither has to outlive the
    other.  Whoever captures by other means gives ``copies`` and keeps it as long as the graph.
    """)
arx_linear_bwd, arx_linear_bwd_plan = _function("arx_linear_bwd", _linear_bwd, """\
Enqueue dz = dout * act'(z), dx = dz w, dw = dz^T x, dbias = sum over rows of dz.

    ``arx_linear_bwd(dout, x, w, dx=None, dw=None, dbias=None, z=None, act=ARX_ACT_NONE, workspace=None,
    status=None, copies=None, wait_us=0, stream=None, check=True)``

    ``workspace`` of ``arx_linear_bwd_workspace_bytes(M, N)`` bytes, unless there is no
    activation and no dbias.  ``copies``, ``status`` and ``wait_us`` as in ``arx_linear``.
    """)


def arx_layer_norm_bwd_workspace_bytes(rows: int, cols: int) -> int:
    return int(_core().lib.arx_layer_norm_bwd_workspace_bytes(rows, cols))


def arx_dropout_add_bwd_workspace_bytes(rows: int, cols: int) -> int:
    return int(_core().lib.arx_dropout_add_bwd_workspace_bytes(rows, cols))


def arx_linear_bwd_workspace_bytes(M: int, N: int) -> int:
    return int(_core().lib.arx_linear_bwd_workspace_bytes(M, N))


def arx_stream_capturing(stream=None) -> bool:
    """Is the stream being captured into a graph?"""
    core = _core()
    return bool(core.lib.arx_stream_capturing(core._stream(stream)))


def arx_linear_copies_bytes(x, w) -> int:
    """Bytes of ``copies`` for ``arx_linear`` of these operands; 0: it is faster without."""
    a = _linear(x, w, None, copies=False).a
    return int(_core().lib.arx_linear_copies_bytes(ctypes.byref(a)))


def arx_linear_bwd_copies_bytes(dout, x=None, w=None, dx=None, dw=None, act=ARX_ACT_NONE, workspace=None) -> int:
    """Bytes of ``copies`` for ``arx_linear_bwd`` with these arguments."""
    a = _linear_bwd(dout, x, w, dx=dx, dw=dw, act=act, workspace=workspace, copies=False).a
    return int(_core().lib.arx_linear_bwd_copies_bytes(ctypes.byref(a)))


__all__ = [
    "ARX_BF16", "ARX_F16", "ARX_F32", "ARX_ACT_NONE", "ARX_ACT_RELU", "ARX_ACT_GELU", "ARX_ACT_GELU_TANH",
    "ARX_ACT_SILU",
    *(f"arx_{op}{suffix}" for op in ("layer_norm", "layer_norm_bwd", "dropout_add", "dropout_add_bwd",
                                     "reduce_layer_norm", "linear", "linear_bwd")
      for suffix in ("", "_plan", "_args")),
    "arx_layer_norm_bwd_workspace_bytes", "arx_dropout_add_bwd_workspace_bytes", "arx_linear_bwd_workspace_bytes",
    "arx_linear_copies_bytes", "arx_linear_bwd_copies_bytes", "arx_stream_capturing",
]
