"""The operators around a tensor-parallel sublayer's all-reduce, as measured cases.

A rank of a tensor-parallel transformer block computes a matrix product with a
fused epilogue (``linear``), the ranks' partials are summed in rank order, and
the sum goes through bias, dropout and the residual add into a layer norm
(``reduce_norm``; ``dropout_add`` and ``layer_norm`` are its parts with their
backward passes).  ``run`` computes each in plain torch operations, or, where
``own`` is true, through the package's entry points.

With x [rows, cols], widened to 32 bits:

* ``linear``       z = x w^T + b, out = act(z) + residual
* ``linear_bwd``   dz = dout act'(z), dx = dz w, dw = dz^T x, db = sum_rows dz
* ``layer_norm``   y = (x - mean) rstd g + b, with mean, rstd of each row
* ``layer_norm_bwd``  q = dy g, xh = (x - mean) rstd,
                   dx = rstd (q - mean(q) - xh mean(q xh)) + dres,
                   dg = sum_rows dy xh, db = sum_rows dy
* ``dropout_add``  out = residual + keep(x + b) / (1 - p)
* ``dropout_add_bwd``  dx = keep(dout) / (1 - p), db = sum_rows dx
* ``reduce_norm``  s = p_0 + p_1 + ... (rank order), h = residual + keep(s + b) / (1 - p),
                   y = layer_norm(h)

``keep`` is Philox4x32-10 (Salmon et al., "Parallel random numbers: as easy as
1, 2, 3", 2011): counter (col // 8, row, offset low, offset high), key the
seed's two halves; its four words are eight 16-bit values for columns
8g ... 8g + 7, low halves first, and an element is kept where its value is at
least T = round(65536 p); the scale is 65536 / (65536 - T).
"""

import math

import numpy as np
import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZE = {"bf16": 2, "f16": 2, "f32": 4}
ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")
EPS = 1e-5


# ---- cases --------------------------------------------------------------------------

def _linear(op, M, N, K, dtype, act="none", bias=False, residual=False, save_z=False, pad=0):
    """x [M, K], w [N, K]; ``pad`` elements more than a row between x's rows."""
    return {"op": op, "M": M, "N": N, "K": K, "dtype": dtype, "act": act, "bias": bias,
            "residual": residual, "save_z": save_z, "pad": pad}


def _rows(op, rows, cols, dtype, **more):
    return {"op": op, "rows": rows, "cols": cols, "dtype": dtype, **more}


def listed():
    return [
        # One token through a column-parallel projection: a rank's 2048 of 16384 features.
        {"name": "linear_token", **_linear("linear", 1, 2048, 4096, "bf16", "gelu_tanh", bias=True)},
        # A prompt chunk of 1024 tokens, hidden 8192, W = 4: a rank's 8192 features; z kept for a later backward pass.
        {"name": "linear_prefill", **_linear("linear", 1024, 8192, 8192, "bf16", "gelu", bias=True, save_z=True)},
        # Ragged: rows that end off 16 bytes, tiles cut on every side, the residual in the epilogue.
        {"name": "linear_ragged", **_linear("linear", 1003, 2044, 4100, "f16", "silu", bias=True, residual=True)},
        # A training step's backward product with the activation's gradient and every output; the largest case.
        {"name": "linear_bwd_train", **_linear("linear_bwd", 8185, 8192, 4096, "bf16", "gelu", bias=True)},
        # The norm of a decode step's [32, 4096] hidden state.
        {"name": "norm_decode", **_rows("layer_norm", 32, 4096, "bf16", wdtype="bf16", stats=False, pad=0)},
        # A training step's norm backward: 8192 tokens, 32-bit master weights, the residual stream's gradient joined.
        {"name": "norm_bwd_train", **_rows("layer_norm_bwd", 8192, 4096, "bf16", wdtype="f32", dres=True, pad=0)},
        # Odd rows and columns in 32 bits.
        {"name": "norm_bwd_odd", **_rows("layer_norm_bwd", 3001, 5003, "f32", wdtype="f32", dres=False, pad=0)},
        # A training step's bias, dropout and residual add, and its backward pass with the bias's gradient.
        {"name": "dropout_train", **_rows("dropout_add", 8192, 4096, "bf16", p=0.1, bias=True, residual=True)},
        {"name": "dropout_bwd_train", **_rows("dropout_add_bwd", 8192, 4096, "bf16", p=0.1, bias=True)},
        # The end of a sublayer at decode ([32, 4096], 8 ranks), on a prompt chunk ([1024, 8192], 4 ranks) and in training.
        {"name": "reduce_norm_decode", **_rows("reduce_norm", 32, 4096, "bf16", W=8, p=0.0, bias=False, stats=False)},
        {"name": "reduce_norm_prefill", **_rows("reduce_norm", 1024, 8192, "bf16", W=4, p=0.0, bias=True, stats=False)},
        {"name": "reduce_norm_train", **_rows("reduce_norm", 8192, 4096, "bf16", W=8, p=0.1, bias=True, stats=True)},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    """A feature count: mostly a multiple of 8 as models have them, one in four any number."""
    n = _log(rng, lo, hi)
    return n if rng.random() < 0.25 else max(8, n // 8 * 8)


def draw(rng):
    op = rng.choice(("linear", "linear", "linear_bwd", "layer_norm", "layer_norm_bwd", "dropout_add",
                     "dropout_add_bwd", "reduce_norm"))
    flip = lambda: rng.random() < 0.5  # noqa: E731
    if op.startswith("linear"):
        M, N, K = _log(rng, 1, 8192), _width(rng, 64, 8192), _width(rng, 64, 8192)
        most = 8185 * 8192 * 4096 * (2 if op == "linear" else 1)
        while M * N * K > most:
            M = (M + 1) // 2
        return _linear(op, M, N, K, rng.choice(("bf16", "f16")), rng.choice(ACTS), bias=flip(),
                       residual=op == "linear" and flip(), save_z=op == "linear" and flip(),
                       pad=rng.choice((0, 0, 0, 8, 3)))
    rows, cols = _log(rng, 1, 16384), _width(rng, 64, 16384)
    while rows * cols > 8192 * 4096:
        rows = (rows + 1) // 2
    if op == "reduce_norm":
        return _rows(op, rows, cols, "bf16", W=rng.randint(1, 8), p=rng.choice((0.0, 0.0, 0.1, 0.25)),
                     bias=flip(), stats=flip())
    dtype = rng.choice(("bf16", "bf16", "f16", "f32"))
    if op.startswith("dropout"):
        c = _rows(op, rows, cols, dtype, p=rng.choice((0.05, 0.1, 0.5)), bias=flip())
        return {**c, "residual": flip()} if op == "dropout_add" else c
    c = _rows(op, rows, cols, dtype, wdtype=rng.choice((dtype, "f32")), pad=rng.choice((0, 0, 8, 3)))
    return {**c, "stats": flip()} if op == "layer_norm" else {**c, "dres": flip()}


# ---- inputs -------------------------------------------------------------------------

def _inputs(c, seed):
    """What the pass reads, from the seed alone."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    t = TYPES[c["dtype"]]

    def normal(*shape, scale=1.0, dtype=t):
        return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)

    def padded(rows, cols, pad, make):
        """A view of ``cols`` columns of a buffer with ``pad`` more in each row."""
        buf = torch.zeros(rows, cols + pad, dtype=t, device="cuda")
        buf[:, :cols] = make
        return buf[:, :cols]

    def activations(rows, cols, scale=1.0):
        """Hidden states: a few channels far larger than the rest, a mean off zero."""
        s = torch.ones(cols, device="cuda")
        s[torch.randperm(cols, generator=g, device="cuda")[: max(1, cols // 256)]] = 12.0
        return (torch.randn(rows, cols, generator=g, device="cuda") * s + 0.1) * scale

    v = {}
    if c["op"].startswith("linear"):
        M, N, K = c["M"], c["N"], c["K"]
        v["x"] = padded(M, K, c["pad"], normal(M, K))
        v["w"] = normal(N, K, scale=K ** -0.5)
        if c["op"] == "linear":
            v["bias"] = normal(N, scale=0.5) if c["bias"] else None
            v["residual"] = normal(M, N) if c["residual"] else None
        else:
            v["z"] = normal(M, N, scale=1.5) if c["act"] != "none" else None
            v["dout"] = normal(M, N, scale=0.01)
        return v
    rows, cols = c["rows"], c["cols"]
    if c["op"].startswith("layer_norm"):
        w = TYPES[c["wdtype"]]
        v["x"] = padded(rows, cols, c["pad"], activations(rows, cols).to(t))
        v["weight"] = (1 + 0.2 * torch.randn(cols, generator=g, device="cuda")).to(w)
        if c["op"] == "layer_norm":
            v["bias"] = normal(cols, scale=0.2, dtype=w)
        else:
            x = v["x"].double()
            m = x.mean(1)
            v["mean"] = m.float()
            v["rstd"] = (((x - m[:, None]) ** 2).mean(1) + EPS).rsqrt().float()
            v["dy"] = normal(rows, cols, scale=0.01)
            v["dres"] = normal(rows, cols, scale=0.01) if c["dres"] else None
        return v
    v["rng"] = torch.tensor([seed * 0x9E3779B1 + 12345, seed * 7 + (5 << 33)], dtype=torch.int64, device="cuda")
    if c["op"] == "reduce_norm":
        v["slots"] = [activations(rows, cols, c["W"] ** -0.5).to(t) for _ in range(c["W"])]
        v["residual"] = activations(rows, cols).to(t)
        v["weight"] = (1 + 0.2 * torch.randn(cols, generator=g, device="cuda")).to(t)
        v["norm_bias"] = normal(cols, scale=0.2)
    elif c["op"] == "dropout_add":
        v["x"] = normal(rows, cols)
        v["residual"] = normal(rows, cols) if c["residual"] else None
    else:
        v["dout"] = normal(rows, cols, scale=0.01)
    if c["op"] != "dropout_add_bwd":
        v["bias"] = normal(cols, scale=0.5) if c["bias"] else None
    return v


def prepare(case, seed):
    c, v = case, _inputs(case, seed)
    if not own:
        return {"case": c, **v}
    # What a program that repeats the call keeps: its output buffers, the workspace and the checked call.
    import deterministic_shot_all_gb300 as arx
    op, t = c["op"], TYPES[c["dtype"]]
    new = lambda *shape, dtype=t: torch.empty(*shape, dtype=dtype, device="cuda")  # noqa: E731
    scratch = lambda n: torch.empty(max(n, 1), dtype=torch.uint8, device="cuda")  # noqa: E731
    if op.startswith("linear"):
        M, N, K = c["M"], c["N"], c["K"]
        act = getattr(arx, "ARX_ACT_" + c["act"].upper())
        if op == "linear":
            out = {"out": new(M, N)}
            if c["save_z"]:
                out["z"] = new(M, N)
            plan = arx.arx_linear_plan(v["x"], v["w"], out["out"], bias=v["bias"], residual=v["residual"],
                                       z=out.get("z"), act=act)
        else:
            out = {"dx": new(M, K), "dw": new(N, K)}
            if c["bias"]:
                out["dbias"] = new(N)
            ws = scratch(arx.arx_linear_bwd_workspace_bytes(M, N))
            plan = arx.arx_linear_bwd_plan(v["dout"], v["x"], v["w"], dx=out["dx"], dw=out["dw"],
                                           dbias=out.get("dbias"), z=v["z"], act=act, workspace=ws)
        return {"case": c, "plan": plan, "out": out}
    rows, cols = c["rows"], c["cols"]
    if op == "layer_norm":
        out = {"y": new(rows, cols)}
        if c["stats"]:
            out |= {"mean": new(rows, dtype=torch.float32), "rstd": new(rows, dtype=torch.float32)}
        plan = arx.arx_layer_norm_plan(v["x"], out["y"], weight=v["weight"], bias=v["bias"], mean=out.get("mean"),
                                       rstd=out.get("rstd"), eps=EPS)
    elif op == "layer_norm_bwd":
        w = TYPES[c["wdtype"]]
        out = {"dx": new(rows, cols), "dweight": new(cols, dtype=w), "dbias": new(cols, dtype=w)}
        ws = scratch(arx.arx_layer_norm_bwd_workspace_bytes(rows, cols))
        plan = arx.arx_layer_norm_bwd_plan(v["dy"], v["x"], v["mean"], v["rstd"], out["dx"], weight=v["weight"],
                                           dresidual=v["dres"], dweight=out["dweight"], dbias=out["dbias"],
                                           workspace=ws)
    elif op == "dropout_add":
        out = {"out": new(rows, cols)}
        plan = arx.arx_dropout_add_plan(v["x"], out["out"], c["p"], v["rng"], bias=v["bias"], residual=v["residual"])
    elif op == "dropout_add_bwd":
        out = {"dx": new(rows, cols)}
        ws = None
        if c["bias"]:
            out["dbias"] = new(cols)
            ws = scratch(arx.arx_dropout_add_bwd_workspace_bytes(rows, cols))
        plan = arx.arx_dropout_add_bwd_plan(v["dout"], out["dx"], c["p"], v["rng"], dbias=out.get("dbias"),
                                            workspace=ws)
    else:
        out = {"h": new(rows, cols), "y": new(rows, cols)}
        if c["stats"]:
            out |= {"mean": new(rows, dtype=torch.float32), "rstd": new(rows, dtype=torch.float32)}
        plan = arx.arx_reduce_layer_norm_plan(v["slots"], out["h"], out["y"], bias=v["bias"], residual=v["residual"],
                                              weight=v["weight"], norm_bias=v["norm_bias"], mean=out.get("mean"),
                                              rstd=out.get("rstd"), eps=EPS, p=c["p"], rng=v["rng"])
    return {"case": c, "plan": plan, "out": out}


# ---- the plain form -----------------------------------------------------------------

def _act(z, act):
    if act == "relu":
        return z.clamp(min=0)
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    if act == "silu":
        return z / (1 + torch.exp(-z))
    return z


def _act_grad(z, act):
    if act == "relu":
        return (z > 0).float()
    if act == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    if act == "gelu_tanh":
        t = torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * z * z)
    s = 1 / (1 + torch.exp(-z))
    return s * (1 + z * (1 - s))


def _philox_round(c0, c1, c2, c3, k0, k1):
    m = 0xFFFFFFFF
    p0, p1 = c0 * 0xD2511F53, c2 * 0xCD9E8D57
    return ((p1 >> 32) & m) ^ c1 ^ k0, p1 & m, ((p0 >> 32) & m) ^ c3 ^ k1, p0 & m


def _keep(rows, cols, p, rng):
    """(mask [rows, cols], scale); the words are kept in 64-bit integers."""
    m = 0xFFFFFFFF
    groups = (cols + 7) // 8
    c0 = torch.arange(groups, device="cuda").expand(rows, groups)
    c1 = torch.arange(rows, device="cuda")[:, None].expand(rows, groups)
    k0, k1 = rng[0] & m, (rng[0] >> 32) & m
    w = (c0, c1, rng[1] & m, (rng[1] >> 32) & m)
    for i in range(10):
        w = _philox_round(*w, (k0 + i * 0x9E3779B9) & m, (k1 + i * 0xBB67AE85) & m)
    u = torch.stack([h for x in w for h in (x & 0xFFFF, x >> 16)], dim=-1).reshape(rows, groups * 8)[:, :cols]
    T = round(p * 65536)
    return u >= T, 65536 / (65536 - T)


def _norm(x, weight, bias):
    mean = x.mean(1, keepdim=True)
    d = x - mean
    rstd = 1 / torch.sqrt((d * d).mean(1, keepdim=True) + EPS)
    return d * rstd * weight.float() + bias.float(), mean[:, 0], rstd[:, 0]


def _drop_add(s, bias, residual, p, rng):
    if bias is not None:
        s = s + bias.float()
    if p > 0:
        keep, scale = _keep(*s.shape, p, rng)
        s = torch.where(keep, s * scale, 0.0)
    return s if residual is None else residual.float() + s


def run(state):
    if "plan" in state:
        state["plan"]()
        return state["out"]
    c, v = state["case"], state
    op, t = c["op"], TYPES[c["dtype"]]
    if op == "linear":
        z = v["x"].float() @ v["w"].float().t()
        if v["bias"] is not None:
            z = z + v["bias"].float()
        y = _act(z, c["act"])
        if v["residual"] is not None:
            y = y + v["residual"].float()
        return {"out": y.to(t), "z": z.to(t)} if c["save_z"] else {"out": y.to(t)}
    if op == "linear_bwd":
        dz = v["dout"].float()
        if v["z"] is not None:
            dz = dz * _act_grad(v["z"].float(), c["act"])
        out = {"dx": (dz @ v["w"].float()).to(t), "dw": (dz.t() @ v["x"].float()).to(t)}
        if c["bias"]:
            out["dbias"] = dz.sum(0).to(t)
        return out
    if op == "layer_norm":
        y, mean, rstd = _norm(v["x"].float(), v["weight"], v["bias"])
        return {"y": y.to(t), "mean": mean, "rstd": rstd} if c["stats"] else {"y": y.to(t)}
    if op == "layer_norm_bwd":
        dy, rstd = v["dy"].float(), v["rstd"][:, None]
        xh = (v["x"].float() - v["mean"][:, None]) * rstd
        q = dy * v["weight"].float()
        dx = rstd * (q - q.mean(1, keepdim=True) - xh * (q * xh).mean(1, keepdim=True))
        if v["dres"] is not None:
            dx = dx + v["dres"].float()
        w = TYPES[c["wdtype"]]
        return {"dx": dx.to(t), "dweight": (dy * xh).sum(0).to(w), "dbias": dy.sum(0).to(w)}
    if op == "dropout_add":
        return {"out": _drop_add(v["x"].float(), v["bias"], v["residual"], c["p"], v["rng"]).to(t)}
    if op == "dropout_add_bwd":
        dx = _drop_add(v["dout"].float(), None, None, c["p"], v["rng"])
        return {"dx": dx.to(t), "dbias": dx.sum(0).to(t)} if c["bias"] else {"dx": dx.to(t)}
    s = v["slots"][0].float()
    for p in v["slots"][1:]:
        s = s + p.float()
    h = _drop_add(s, v["bias"], v["residual"], c["p"], v["rng"])
    y, mean, rstd = _norm(h, v["weight"], v["norm_bias"])
    out = {"h": h.to(t), "y": y.to(t)}
    return {**out, "mean": mean, "rstd": rstd} if c["stats"] else out


# ---- the definition in 64 bits ------------------------------------------------------

def _exact_kept(rows, cols, p, rng):
    """Scale factors [rows, cols], 0 where dropped (unsigned 64-bit words, on the host)."""
    u64 = np.uint64
    seed, offset = (int(x) & (2 ** 64 - 1) for x in rng.tolist())
    groups = -(-cols // 8)
    x = [np.tile(np.arange(groups, dtype=u64), rows), np.repeat(np.arange(rows, dtype=u64), groups),
         u64(offset & 0xFFFFFFFF), u64(offset >> 32)]
    key = [seed & 0xFFFFFFFF, seed >> 32]
    low, half = u64(0xFFFFFFFF), u64(32)
    for _ in range(10):
        a, b = x[0] * u64(0xD2511F53), x[2] * u64(0xCD9E8D57)
        x = [(b >> half) ^ x[1] ^ u64(key[0]), b & low, (a >> half) ^ x[3] ^ u64(key[1]), a & low]
        key = [(key[0] + 0x9E3779B9) % 2 ** 32, (key[1] + 0xBB67AE85) % 2 ** 32]
    bits = np.stack([w.astype(np.uint32) for w in x], axis=1).reshape(rows, groups * 4)
    u = bits.astype("<u4").view("<u2")[:, :cols]
    T = round(p * 65536)
    return torch.from_numpy(np.where(u >= T, 65536 / (65536 - T), 0.0)).cuda()


def exact(case, seed):
    c, v = case, _inputs(case, seed)
    d = lambda x: None if x is None else x.double()  # noqa: E731
    op = c["op"]
    if op == "linear":
        z = torch.matmul(d(v["x"]), d(v["w"]).T)
        if c["bias"]:
            z += d(v["bias"])
        phi = lambda a: torch.special.ndtr(a)  # noqa: E731
        y = {"none": lambda: z, "relu": lambda: torch.maximum(z, torch.zeros_like(z)), "gelu": lambda: z * phi(z),
             "gelu_tanh": lambda: z * torch.sigmoid(math.sqrt(8 / math.pi) * (z + 0.044715 * z ** 3)),
             "silu": lambda: z * torch.sigmoid(z)}[c["act"]]()
        y = y + d(v["residual"]) if c["residual"] else y
        return {"out": y, "z": z} if c["save_z"] else {"out": y}
    if op == "linear_bwd":
        dz = d(v["dout"])
        if c["act"] != "none":
            z = d(v["z"])
            if c["act"] == "relu":
                dz = torch.where(z > 0, dz, torch.zeros_like(dz))
            elif c["act"] == "gelu":
                dz = dz * (torch.special.ndtr(z) + z * torch.exp(-z * z / 2) / (2 * math.pi) ** 0.5)
            elif c["act"] == "gelu_tanh":
                k = math.sqrt(8 / math.pi)
                s = torch.sigmoid(k * (z + 0.044715 * z ** 3))
                dz = dz * (s + z * s * (1 - s) * k * (1 + 0.134145 * z ** 2))
            else:
                s = torch.sigmoid(z)
                dz = dz * (s + z * s * (1 - s))
        out = {"dx": torch.matmul(dz, d(v["w"])), "dw": torch.matmul(dz.T, d(v["x"]))}
        return {**out, "dbias": dz.sum(0)} if c["bias"] else out
    if op == "layer_norm_bwd":
        x, dy, r = d(v["x"]), d(v["dy"]), d(v["rstd"])
        xh = (x - d(v["mean"])[:, None]) * r[:, None]
        q = dy * d(v["weight"])
        n = x.shape[1]
        dx = q - (q.sum(1) / n)[:, None] - xh * (torch.einsum("ij,ij->i", q, xh) / n)[:, None]
        dx = dx * r[:, None]
        if c["dres"]:
            dx += d(v["dres"])
        return {"dx": dx, "dweight": torch.einsum("ij,ij->j", dy, xh), "dbias": dy.sum(0)}
    if op in ("dropout_add", "dropout_add_bwd"):
        k = _exact_kept(c["rows"], c["cols"], c["p"], v["rng"])
        if op == "dropout_add_bwd":
            dx = d(v["dout"]) * k
            return {"dx": dx, "dbias": dx.sum(0)} if c["bias"] else {"dx": dx}
        x = d(v["x"])
        x = (x + d(v["bias"]) if c["bias"] else x) * k
        return {"out": x + d(v["residual"]) if c["residual"] else x}
    if op == "reduce_norm":
        h = torch.zeros_like(v["slots"][0], dtype=torch.float64)
        for s in v["slots"]:
            h += s
        if c["bias"]:
            h += v["bias"]
        if c["p"] > 0:
            h *= _exact_kept(c["rows"], c["cols"], c["p"], v["rng"])
        h += v["residual"]
        g, b = v["weight"], v["norm_bias"]
    else:
        h, g, b = d(v["x"]), v["weight"], v["bias"]
    var, mean = torch.var_mean(h, dim=1, correction=0)
    rstd = (var + EPS) ** -0.5
    out = {"y": (h - mean[:, None]) * rstd[:, None] * d(g) + d(b)}
    if op == "reduce_norm":
        out["h"] = h
    return {**out, "mean": mean, "rstd": rstd} if c["stats"] else out


# ---- what a pass cannot do without --------------------------------------------------

def work(case):
    c, e = case, SIZE[case["dtype"]]
    op = c["op"]
    if op.startswith("linear"):
        M, N, K = c["M"], c["N"], c["K"]
        if op == "linear":
            n = M * K + N * K + M * N * (1 + c["residual"] + c["save_z"]) + N * c["bias"]
            return {"bytes": e * n, "flops": 2 * M * N * K + 8 * M * N}
        n = M * N * (1 + (c["act"] != "none")) + 2 * M * K + 2 * N * K + N * c["bias"]
        return {"bytes": e * n, "flops": 4 * M * N * K + 16 * M * N}
    rows, cols = c["rows"], c["cols"]
    n = rows * cols
    if op == "layer_norm":
        return {"bytes": 2 * e * n + 2 * cols * SIZE[c["wdtype"]] + 8 * rows * c["stats"], "flops": 8 * n}
    if op == "layer_norm_bwd":
        return {"bytes": (3 + c["dres"]) * e * n + 3 * cols * SIZE[c["wdtype"]] + 8 * rows, "flops": 16 * n}
    if op == "dropout_add":
        return {"bytes": e * (n * (2 + c["residual"]) + cols * c["bias"]) + 16, "flops": 3 * n}
    if op == "dropout_add_bwd":
        return {"bytes": e * (2 * n + cols * c["bias"]) + 16, "flops": 2 * n}
    return {"bytes": e * (n * (c["W"] + 3) + cols * (2 + c["bias"])) + 8 * rows * c["stats"],
            "flops": (c["W"] + 11) * n}
