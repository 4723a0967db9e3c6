"""The operators of a gated, root-mean-square-normalised tensor-parallel sublayer, as measured cases.

The ranks' partials are summed in rank order onto the residual stream and
normalised (``reduce_rms_norm``; ``rms_norm`` is its form for one stream), in 16
or 32 bits or as 8-bit floating point with a scale for each row, and the gated
feed-forward block multiplies the result by two weight matrices and the
projections with each other (``gated_linear``).  ``run`` computes each in plain
torch operations, or, where ``own`` is true, through the package's entry points.

With every input widened to 32 bits:

* ``rms_norm``      h = x + residual, rstd = 1 / sqrt(sum(h^2) / cols + eps), y = h rstd g;
                    s = max |y| / 448 of each row (1 where that is below 2^-126), q = e4m3(y / s)
* ``rms_norm_bwd``  v = dy g, n = h rstd, dx = rstd (v - n mean(v n)) + dres, dg = sum_rows dy n
* ``reduce_rms_norm``  h = residual + (p_0 + p_1 + ...) (rank order), then as ``rms_norm``
* ``gated_linear``  a = x Wg^T + bg, b = x Wu^T + bu, out = act(a) b; 8-bit operands: the products
                    times the scales of x's row and of the weight's row, then the bias
* ``gated_linear_bwd``  da = dout b act'(a), db = dout act(a), dx = da Wg + db Wu,
                    dWg = da^T x, dWu = db^T x, dbg = sum_rows da, dbu = sum_rows db
"""

import math

import torch

own = False

E4M3 = torch.float8_e4m3fn
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32, "e4m3": E4M3}
SIZE = {"bf16": 2, "f16": 2, "f32": 4, "e4m3": 1}
ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")
EPS = 1e-6
TOP = 448.0            # largest e4m3 number
LEAST = 2.0 ** -126


# ---- cases --------------------------------------------------------------------------

def _rows(op, rows, cols, dtype, **more):
    return {"op": op, "rows": rows, "cols": cols, "dtype": dtype, **more}


def _gated(op, M, N, K, dtype, act="silu", bias=False, save_z=False, pad=0, out="bf16"):
    """x [M, K], both weights [N, K]; ``pad`` elements more than a row between x's rows."""
    return {"op": op, "M": M, "N": N, "K": K, "dtype": dtype, "out": out if dtype == "e4m3" else dtype, "act": act,
            "bias": bias, "save_z": save_z, "pad": pad}


def listed():
    return [
        # A decode step's hidden state on its way into an 8-bit block.
        {"name": "rms_decode", **_rows("rms_norm", 32, 4096, "bf16", wdtype="bf16", res=True, form="q", stats=False, pad=0)},
        # A training step's residual add and norm: 8192 tokens, 32-bit master weights, rstd kept.
        {"name": "rms_train", **_rows("rms_norm", 8192, 4096, "bf16", wdtype="f32", res=True, form="y", stats=True, pad=0)},
        # Its backward pass, joined by the residual stream's gradient.
        {"name": "rms_bwd_train", **_rows("rms_norm_bwd", 8192, 4096, "bf16", wdtype="f32", dres=True, pad=0)},
        # Odd rows and columns in 32 bits.
        {"name": "rms_bwd_odd", **_rows("rms_norm_bwd", 3001, 5003, "f32", wdtype="f32", dres=False, pad=0)},
        # The end of a sublayer at decode, 8 ranks, handing 8 bits to the next block.
        {"name": "reduce_rms_decode", **_rows("reduce_rms_norm", 32, 4096, "bf16", W=8, form="q", stats=False)},
        # The same on a prompt chunk, 4 ranks, in 16 bits.
        {"name": "reduce_rms_prefill", **_rows("reduce_rms_norm", 1024, 8192, "bf16", W=4, form="y", stats=False)},
        # One token through a rank's share of the gated projections.
        {"name": "gated_token", **_gated("gated_linear", 1, 2048, 4096, "bf16")},
        # A training step's forward pass on a packed batch, both projections kept for the backward pass.
        {"name": "gated_train", **_gated("gated_linear", 8185, 4096, 4096, "bf16", save_z=True)},
        # A decode batch with 8-bit operands: bound by reading the weights.
        {"name": "gated_e4m3_decode", **_gated("gated_linear", 32, 4096, 8192, "e4m3")},
        # A prompt chunk with 8-bit operands, hidden 8192.
        {"name": "gated_e4m3_prefill", **_gated("gated_linear", 1024, 8192, 8192, "e4m3")},
        # Ragged gradients: rows that end off 16 bytes, tiles cut on every side, bias gradients.
        {"name": "gated_bwd_ragged", **_gated("gated_linear_bwd", 259, 2050, 1030, "f16", "gelu", bias=True)},
        # A training step's backward pass; the largest case.
        {"name": "gated_bwd_train", **_gated("gated_linear_bwd", 8185, 4096, 4096, "bf16")},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    """A feature count: mostly a multiple of 8 as models have them, one in four any number."""
    n = _log(rng, lo, hi)
    return n if rng.random() < 0.25 else max(8, n // 8 * 8)


def draw(rng):
    op = rng.choice(("rms_norm", "rms_norm_bwd", "reduce_rms_norm", "gated_linear", "gated_linear", "gated_linear_bwd"))
    flip = lambda: rng.random() < 0.5  # noqa: E731
    if op.startswith("gated"):
        M, N, K = _log(rng, 1, 8192), _width(rng, 64, 8192), _width(rng, 64, 8192)
        while M * N * K > 8185 * 4096 * 4096:
            M = (M + 1) // 2
        dtype = rng.choice(("bf16", "f16", "e4m3") if op == "gated_linear" else ("bf16", "f16"))
        pad = 0 if dtype == "e4m3" else rng.choice((0, 0, 0, 8, 3))
        return _gated(op, M, N, K, dtype, rng.choice(ACTS), bias=flip(), save_z=op == "gated_linear" and flip(), pad=pad,
                      out=rng.choice(("bf16", "f16")))
    rows, cols = _log(rng, 1, 16384), _width(rng, 64, 16384)
    while rows * cols > 8192 * 4096:
        rows = (rows + 1) // 2
    if op == "reduce_rms_norm":
        return _rows(op, rows, cols, "bf16", W=rng.randint(1, 8), form=rng.choice(("y", "q", "both")), stats=flip())
    dtype = rng.choice(("bf16", "bf16", "f16", "f32"))
    c = _rows(op, rows, cols, dtype, wdtype=rng.choice((dtype, "f32")), pad=rng.choice((0, 0, 8, 3)))
    if op == "rms_norm_bwd":
        return {**c, "dres": flip()}
    return {**c, "res": flip(), "form": rng.choice(("y", "q", "both")), "stats": flip()}


# ---- inputs -------------------------------------------------------------------------

def _pitch(n):
    """Elements from row to row of an 8-bit matrix: rows on 16 bytes."""
    return (n + 15) // 16 * 16


def _inputs(c, seed):
    """What the pass reads, from the seed alone."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    t = TYPES[c["dtype"]]

    def normal(*shape, scale=1.0, dtype=t):
        return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)

    def padded(pad, make):
        """A view of the matrix in a buffer with ``pad`` more in each row."""
        buf = torch.zeros(make.shape[0], make.shape[1] + pad, dtype=make.dtype, device="cuda")
        buf[:, :make.shape[1]] = make
        return buf[:, :make.shape[1]]

    def activations(rows, cols, scale=1.0):
        """Hidden states: a few channels far larger than the rest, a mean off zero."""
        s = torch.ones(cols, device="cuda")
        s[torch.randperm(cols, generator=g, device="cuda")[: max(1, cols // 256)]] = 12.0
        return (torch.randn(rows, cols, generator=g, device="cuda") * s + 0.1) * scale

    def eight_bits(x):
        """A matrix as 8-bit values and the scales of its rows."""
        s = x.abs().amax(1).clamp_min(1e-12) / TOP
        return padded(_pitch(x.shape[1]) - x.shape[1], (x / s[:, None]).to(E4M3)), s

    v = {}
    if c["op"].startswith("gated"):
        M, N, K = c["M"], c["N"], c["K"]
        if c["dtype"] == "e4m3":
            v["x"], v["x_scale"] = eight_bits(activations(M, K))
            v["w_gate"], v["gate_scale"] = eight_bits(normal(N, K, scale=K ** -0.5, dtype=torch.float32))
            v["w_up"], v["up_scale"] = eight_bits(normal(N, K, scale=K ** -0.5, dtype=torch.float32))
        else:
            v["x"] = padded(c["pad"], normal(M, K))
            v["w_gate"], v["w_up"] = normal(N, K, scale=K ** -0.5), normal(N, K, scale=K ** -0.5)
        if c["op"] == "gated_linear":
            o = TYPES[c["out"]]
            v["bias_gate"] = normal(N, scale=0.5, dtype=o) if c["bias"] else None
            v["bias_up"] = normal(N, scale=0.5, dtype=o) if c["bias"] else None
        else:
            v["z_gate"], v["z_up"] = normal(M, N, scale=1.5), normal(M, N, scale=1.5)
            v["dout"] = normal(M, N, scale=0.01)
        return v
    rows, cols = c["rows"], c["cols"]
    if c["op"] == "reduce_rms_norm":
        v["slots"] = [activations(rows, cols, c["W"] ** -0.5).to(t) for _ in range(c["W"])]
        v["residual"] = activations(rows, cols).to(t)
        v["weight"] = (1 + 0.2 * torch.randn(cols, generator=g, device="cuda")).to(t)
        return v
    v["weight"] = (1 + 0.2 * torch.randn(cols, generator=g, device="cuda")).to(TYPES[c["wdtype"]])
    x = padded(c["pad"], activations(rows, cols).to(t))
    if c["op"] == "rms_norm":
        v["x"] = x
        v["residual"] = activations(rows, cols).to(t) if c["res"] else None
    else:
        v["h"] = x
        v["rstd"] = (x.double().square().mean(1) + EPS).rsqrt().float()
        v["dy"] = normal(rows, cols, scale=0.01)
        v["dres"] = normal(rows, cols, scale=0.01) if c["dres"] else None
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
    if op.startswith("gated"):
        M, N, K = c["M"], c["N"], c["K"]
        act, o = getattr(arx, "ARX_ACT_" + c["act"].upper()), TYPES[c["out"]]
        if op == "gated_linear":
            out = {"out": new(M, N, dtype=o)}
            if c["save_z"]:
                out |= {"z_gate": new(M, N, dtype=o), "z_up": new(M, N, dtype=o)}
            scales = {k: v[k] for k in ("x_scale", "gate_scale", "up_scale") if k in v}
            plan = arx.arx_gated_linear_plan(v["x"], v["w_gate"], v["w_up"], out["out"], bias_gate=v["bias_gate"],
                                             bias_up=v["bias_up"], z_gate=out.get("z_gate"), z_up=out.get("z_up"),
                                             act=act, **scales)
        else:
            out = {"dx": new(M, K), "dw_gate": new(N, K), "dw_up": new(N, K)}
            if c["bias"]:
                out |= {"dbias_gate": new(N), "dbias_up": new(N)}
            ws = scratch(arx.arx_gated_linear_bwd_workspace_bytes(M, N))
            plan = arx.arx_gated_linear_bwd_plan(v["dout"], v["x"], v["w_gate"], v["w_up"], v["z_gate"], v["z_up"],
                                                 dx=out["dx"], dw_gate=out["dw_gate"], dw_up=out["dw_up"],
                                                 dbias_gate=out.get("dbias_gate"), dbias_up=out.get("dbias_up"),
                                                 act=act, workspace=ws)
        return {"case": c, "plan": plan, "out": out}
    rows, cols = c["rows"], c["cols"]
    if op == "rms_norm_bwd":
        out = {"dx": new(rows, cols), "dweight": new(cols, dtype=TYPES[c["wdtype"]])}
        ws = scratch(arx.arx_rms_norm_bwd_workspace_bytes(rows, cols))
        plan = arx.arx_rms_norm_bwd_plan(v["dy"], v["h"], v["rstd"], out["dx"], weight=v["weight"], dresidual=v["dres"],
                                         dweight=out["dweight"], workspace=ws)
        return {"case": c, "plan": plan, "out": out}
    out = {}
    if op == "reduce_rms_norm" or c["res"]:
        out["h"] = new(rows, cols)
    if c["form"] != "q":
        out["y"] = new(rows, cols)
    if c["form"] != "y":
        out["q"] = new(rows, _pitch(cols), dtype=E4M3)[:, :cols]
        out["scale"] = new(rows, dtype=torch.float32)
    if c["stats"]:
        out["rstd"] = new(rows, dtype=torch.float32)
    more = {"residual": v["residual"], "weight": v["weight"], "q": out.get("q"), "scale": out.get("scale"),
            "rstd": out.get("rstd"), "eps": EPS}
    if op == "rms_norm":
        plan = arx.arx_rms_norm_plan(v["x"], out.get("y"), h=out.get("h"), **more)
    else:
        plan = arx.arx_reduce_rms_norm_plan(v["slots"], out["h"], out.get("y"), **more)
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
    if act == "none":
        return torch.ones_like(z)
    if act == "relu":
        return (z > 0).float()
    if act == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    if act == "gelu_tanh":
        t = torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * z * z)
    s = 1 / (1 + torch.exp(-z))
    return s * (1 + z * (1 - s))


def _project(x, w, x_scale, w_scale, bias):
    z = x.float() @ w.float().t()
    if x_scale is not None:
        z = z * (x_scale[:, None] * w_scale)
    return z if bias is None else z + bias.float()


def run(state):
    if "plan" in state:
        state["plan"]()
        return state["out"]
    c, v = state["case"], state
    op, t = c["op"], TYPES[c["dtype"]]
    if op == "gated_linear":
        o = TYPES[c["out"]]
        a = _project(v["x"], v["w_gate"], v.get("x_scale"), v.get("gate_scale"), v["bias_gate"])
        b = _project(v["x"], v["w_up"], v.get("x_scale"), v.get("up_scale"), v["bias_up"])
        out = {"out": (_act(a, c["act"]) * b).to(o)}
        return {**out, "z_gate": a.to(o), "z_up": b.to(o)} if c["save_z"] else out
    if op == "gated_linear_bwd":
        a, dout, x = v["z_gate"].float(), v["dout"].float(), v["x"].float()
        da = dout * v["z_up"].float() * _act_grad(a, c["act"])
        db = dout * _act(a, c["act"])
        out = {"dx": (da @ v["w_gate"].float() + db @ v["w_up"].float()).to(t), "dw_gate": (da.t() @ x).to(t),
               "dw_up": (db.t() @ x).to(t)}
        return {**out, "dbias_gate": da.sum(0).to(t), "dbias_up": db.sum(0).to(t)} if c["bias"] else out
    if op == "rms_norm_bwd":
        dy, rstd = v["dy"].float(), v["rstd"][:, None]
        n = v["h"].float() * rstd
        p = dy * v["weight"].float()
        dx = rstd * (p - n * (p * n).mean(1, keepdim=True))
        if v["dres"] is not None:
            dx = dx + v["dres"].float()
        return {"dx": dx.to(t), "dweight": (dy * n).sum(0).to(TYPES[c["wdtype"]])}
    out = {}
    if op == "reduce_rms_norm":
        h = v["slots"][0].float()
        for p in v["slots"][1:]:
            h = h + p.float()
        h = v["residual"].float() + h
        out["h"] = h.to(t)
    else:
        h = v["x"].float()
        if c["res"]:
            h = h + v["residual"].float()
            out["h"] = h.to(t)
    rstd = 1 / torch.sqrt((h * h).mean(1, keepdim=True) + EPS)
    y = h * rstd * v["weight"].float()
    if c["form"] != "q":
        out["y"] = y.to(t)
    if c["form"] != "y":
        s = y.abs().amax(1) / TOP
        s = torch.where(s < LEAST, 1.0, s)
        out["q"], out["scale"] = (y / s[:, None]).to(E4M3), s
    if c["stats"]:
        out["rstd"] = rstd[:, 0]
    return out


# ---- the definition in 64 bits ------------------------------------------------------

def _exact_act(z, name):
    """The activation and its derivative."""
    if name == "none":
        return z, torch.ones_like(z)
    if name == "relu":
        on = (z > 0).double()
        return on * z, on
    if name == "gelu":
        p = torch.special.ndtr(z)
        return z * p, p + z * torch.exp(-z * z / 2) / (2 * math.pi) ** 0.5
    if name == "gelu_tanh":
        k = math.sqrt(8 / math.pi)
        s = torch.sigmoid(k * (z + 0.044715 * z ** 3))
        return z * s, s + z * s * (1 - s) * k * (1 + 0.134145 * z ** 2)
    s = torch.sigmoid(z)
    return z * s, s + z * s * (1 - s)


def exact(case, seed):
    c, v = case, _inputs(case, seed)
    d = {k: x.double() if isinstance(x, torch.Tensor) else x for k, x in v.items()}
    op = c["op"]
    if op == "gated_linear":
        z = []
        for which in ("gate", "up"):
            x, w = d["x"], d["w_" + which]
            if c["dtype"] == "e4m3":
                x, w = torch.einsum("mk,m->mk", x, d["x_scale"]), torch.einsum("nk,n->nk", w, d[which + "_scale"])
            z.append(torch.matmul(x, w.T))
            if c["bias"]:
                z[-1] += d["bias_" + which]
        out = {"out": _exact_act(z[0], c["act"])[0] * z[1]}
        return {**out, "z_gate": z[0], "z_up": z[1]} if c["save_z"] else out
    if op == "gated_linear_bwd":
        f, slope = _exact_act(d["z_gate"], c["act"])
        da, db = d["dout"] * d["z_up"] * slope, d["dout"] * f
        both = torch.cat([da, db], dim=1)
        out = {"dx": torch.matmul(both, torch.cat([d["w_gate"], d["w_up"]]))}
        out["dw_gate"], out["dw_up"] = torch.matmul(both.T, d["x"]).split(c["N"])
        if c["bias"]:
            out["dbias_gate"], out["dbias_up"] = both.sum(0).split(c["N"])
        return out
    if op == "rms_norm_bwd":
        unit = torch.einsum("ij,i->ij", d["h"], d["rstd"])
        into = torch.einsum("ij,j->ij", d["dy"], d["weight"])
        along = torch.einsum("ij,ij->i", into, unit) / c["cols"]
        dx = torch.einsum("ij,i->ij", into - unit * along[:, None], d["rstd"])
        return {"dx": dx + d["dres"] if c["dres"] else dx, "dweight": torch.einsum("ij,ij->j", d["dy"], unit)}
    out = {}
    h = d["x"].clone() if op == "rms_norm" else torch.zeros_like(d["residual"])
    for p in v.get("slots", ()):
        h += p
    if d["residual"] is not None:
        h += d["residual"]
        out["h"] = h
    r = (torch.einsum("ij,ij->i", h, h) / c["cols"] + EPS) ** -0.5
    y = torch.einsum("ij,i,j->ij", h, r, d["weight"])
    if c["form"] != "q":
        out["y"] = y
    if c["form"] != "y":
        out["scale"] = torch.linalg.vector_norm(y, math.inf, dim=1) / TOP
        out["q"] = y / out["scale"][:, None]
    if c["stats"]:
        out["rstd"] = r
    return out


# ---- what a pass cannot do without --------------------------------------------------

def work(case):
    c, e = case, SIZE[case["dtype"]]
    op = c["op"]
    if op.startswith("gated"):
        M, N, K = c["M"], c["N"], c["K"]
        if op == "gated_linear":
            o = SIZE[c["out"]]
            n = e * (M * K + 2 * N * K) + o * (M * N * (1 + 2 * c["save_z"]) + 2 * N * c["bias"])
            return {"bytes": n + 4 * (M + 2 * N) * (c["dtype"] == "e4m3"), "flops": 4 * M * N * K + 8 * M * N}
        n = 3 * M * N + 2 * M * K + 4 * N * K + 2 * N * c["bias"]
        return {"bytes": e * n, "flops": 8 * M * N * K + 16 * M * N}
    rows, cols = c["rows"], c["cols"]
    n = rows * cols
    if op == "rms_norm_bwd":
        return {"bytes": (3 + c["dres"]) * e * n + 2 * cols * SIZE[c["wdtype"]] + 4 * rows, "flops": 12 * n}
    res = op == "reduce_rms_norm" or c["res"]
    read = c["W"] if op == "reduce_rms_norm" else 1
    write = e * (c["form"] != "q") + (c["form"] != "y")
    w = e if op == "reduce_rms_norm" else SIZE[c["wdtype"]]
    return {"bytes": n * (e * (read + 2 * res) + write) + cols * w + 4 * rows * ((c["form"] != "y") + c["stats"]),
            "flops": (read + res + 5) * n}
