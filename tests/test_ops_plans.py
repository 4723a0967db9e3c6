"""Plans whose call needs copies that the caller did not give: where those live.

A plan holds its copies; a graph that captured a call of it is replayed after
the plan is gone.  Host-side with fakes: no GPU, no kernel launched.
"""

import contextlib
import gc

import pytest
import torch

M, N, K = 1003, 2044, 4100  # rows off 16 bytes, at a size where copies pay


@pytest.fixture
def fakes(arx, monkeypatch):
    """CPU tensors pass for CUDA ones; ``state["capturing"]`` is what the stream says; the calls are recorded."""
    from deterministic_shot_all_gb300 import _ops
    state = {"capturing": 0, "made": [], "calls": []}
    empty = torch.empty

    def on_host(*shape, device=None, **kw):
        t = empty(*shape, **kw)
        state["made"].append(t)
        return t

    def record(ref, stream):
        state["calls"].append((ref._obj.copies, ref._obj.copies_bytes, state["capturing"]))
        return 0

    monkeypatch.setattr(_ops._Marshal, "_on_device", lambda self, t, name: setattr(self, "device", 0))
    monkeypatch.setattr(torch, "empty", on_host)
    monkeypatch.setattr(torch.cuda, "stream", lambda s: contextlib.nullcontext())
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda s: s)
    monkeypatch.setattr(arx.lib, "arx_stream_capturing", lambda s: state["capturing"], raising=False)
    state["record"] = record
    return state


def _operands():
    zeros = lambda r, c: torch.zeros(r, c, dtype=torch.bfloat16)  # noqa: E731
    return zeros(M, K), zeros(N, K), zeros(M, N)


def _plan(arx, op, fakes, **more):
    x, w, out = _operands()
    if op == "linear":
        p = arx.arx_linear_plan(x, w, out, stream=7, **more)
    else:
        p = arx.arx_linear_bwd_plan(out, x, w, dx=x.clone(), dw=w.clone(), stream=7, **more)
    p._fn = fakes["record"]
    return p


@pytest.mark.parametrize("op", ["linear", "linear_bwd"])
def test_a_captured_call_does_not_use_the_plans_own_copies(arx, fakes, op):
    plan = _plan(arx, op, fakes)
    plan()
    own, n, _ = fakes["calls"][0]
    assert own == fakes["made"][0].data_ptr() and n == fakes["made"][0].numel() > 0
    fakes["capturing"] = 1
    plan()
    captured, m, _ = fakes["calls"][1]
    assert m == n and captured != own
    assert captured in [t.data_ptr() for t in fakes["made"]]
    fakes["capturing"] = 0
    plan()
    assert fakes["calls"][2][0] == own  # and the plan goes on with its own


def test_given_copies_are_used_in_a_capture_too(arx, fakes):
    n = 64 << 20
    buf = torch.zeros(n, dtype=torch.uint8)
    plan = _plan(arx, "linear", fakes, copies=buf)
    for fakes["capturing"] in (0, 1):
        plan()
    assert [c[0] for c in fakes["calls"]] == [buf.data_ptr()] * 2


def test_a_plan_without_copies_does_not_ask(arx, fakes, monkeypatch):
    plan = _plan(arx, "linear", fakes, copies=False)
    monkeypatch.setattr(arx.lib, "arx_stream_capturing", lambda s: pytest.fail("asked"))
    plan()
    assert fakes["calls"][0][0] is None and not fakes["made"]


# ---- on the GPU ---------------------------------------------------------------------------

@pytest.mark.gpu
@pytest.mark.parametrize("op", ["linear", "linear_bwd"])
def test_a_graph_outlives_its_plan(arx, op):
    make = lambda r, c, s: torch.randn(r, c, generator=torch.Generator("cuda").manual_seed(s), device="cuda").bfloat16()  # noqa: E731
    x, w, d = make(M, K, 1), make(N, K, 2), make(M, N, 3)
    outs = [torch.empty_like(t) for t in ((d,) if op == "linear" else (x, w))]
    want = [torch.empty_like(t) for t in outs]
    side = torch.cuda.Stream()

    def call(to, plan, **kw):
        f = getattr(arx, f"arx_{op}" + ("_plan" if plan else ""))
        return f(x, w, to[0], **kw) if op == "linear" else f(d, x, w, dx=to[0], dw=to[1], **kw)

    call(want, False)
    torch.cuda.synchronize()
    plan = call(outs, True, stream=side)
    n = plan._args.copies_bytes
    assert n > 0
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        assert arx.lib.arx_stream_capturing(side.cuda_stream) == 1
        plan()
    assert arx.lib.arx_stream_capturing(side.cuda_stream) == 0
    del plan
    gc.collect()
    with torch.cuda.stream(side):  # takes what the plan gave back
        others = [torch.full((n,), 0x5A, dtype=torch.uint8, device="cuda") for _ in range(3)]
    torch.cuda.synchronize()
    graph.replay()
    torch.cuda.synchronize()
    assert all(bool((o == 0x5A).all()) for o in others)
    assert all(torch.equal(a, b) for a, b in zip(outs, want))
