"""A wait of the matrix product that runs out: the kernel ends with a status, and the next call is right.

On the host: the limit's range, and a model of how a block that gave up makes
its stages' phases complete.  On the GPU: contractions so long that a wait for
a tile's products takes several milliseconds, with a limit of one.  Nothing
hangs: every wait has its limit, and the operands are ordinary ones.
"""

import ctypes
import random
import subprocess
import sys

import pytest
import torch

FAKE = 1 << 40


@pytest.mark.parametrize("op", ["linear", "linear_bwd"])
@pytest.mark.parametrize("us", [-1, 2000001, 1 << 30])
def test_limits_out_of_range(arx, op, us):
    a = getattr(arx, f"arx_{op}_args")(M=4, N=16, K=8, wait_us=us)
    for i, n in enumerate("x w out dx dout".split()):
        if hasattr(a, n):
            setattr(a, n, FAKE + (i << 32))
    for n in "ldx ldw ldout lddx lddout".split():
        if hasattr(a, n):
            setattr(a, n, 16)
    assert getattr(arx.lib, f"arx_{op}")(ctypes.byref(a), None) == arx.ARX_EINVAL
    assert f"wait_us={us}" in arx.arx_last_error()


class Barrier:
    """A shared-memory barrier's current phase: arrivals and bytes it still waits for."""

    def __init__(self, count):
        self.count = self.pending = count
        self.bytes = self.phase = 0

    def _turn(self):
        assert self.pending >= 0, "more arrivals than the phase takes"
        if self.pending == 0 and self.bytes == 0:
            self.pending, self.phase = self.count, self.phase + 1

    def expect(self, n):
        self.bytes += n

    def arrive(self):
        self.pending -= 1
        self._turn()

    def land(self, n):
        self.bytes -= n
        self._turn()


@pytest.mark.parametrize("loaders", [0, 3])
@pytest.mark.parametrize("pair", [False, True])
@pytest.mark.parametrize("copies", [True, False])
def test_a_drain_completes_every_phase_when_its_copies_have_landed(pair, loaders, copies):
    """The rule of drain_block in csrc/linear.cu, from every mix of fills that writers can have reached."""
    if not copies and not loaders:
        return
    r, stages, nbytes, blocks = random.Random(1), 4, 32, 2 if pair else 1
    for _ in range(3000):
        # Fills consumed; a writer has filled at least those and at most `stages` more.
        consumed = r.randrange(0, 9)
        writers = [(b, w) for b in range(blocks) for w in range(0 if copies else 1, 1 + loaders)]
        fills = {k: consumed + r.randrange(0, stages + 1) for k in writers}
        bars = [Barrier(copies + blocks * loaders) for _ in range(stages)]
        flying = []  # (bar, fill) of copies issued and not landed
        events = [(k, f) for k in writers for f in range(fills[k])]
        events.sort(key=lambda e: (e[1], r.random()))  # a writer fills in order
        for (b, w), f in events:
            bar = bars[f % stages]
            if w:
                bar.arrive()
                continue
            if b == 0:
                bar.expect(nbytes * blocks)
                bar.arrive()
            if f < consumed or r.random() < 0.5:
                bar.land(nbytes)
            else:
                flying.append((bar, f))
        most = max(fills.values())
        for f in range(max(0, most - stages), most):
            bar = bars[f % stages]
            assert bar.phase in (f // stages, f // stages + 1)
            whole = all(n > f for n in fills.values())
            if copies:
                own, peer = fills[0, 0] > f, pair and fills[1, 0] > f
                if own and pair and not peer:
                    bar.land(nbytes)
                elif not own and peer:
                    bar.expect(nbytes)
                    bar.arrive()
                elif not own:
                    bar.arrive()
            for (b, w), n in fills.items():
                if w and n <= f:
                    bar.arrive()
            mine = [x for x in flying if x[1] == f]
            assert (bar.phase == f // stages + 1) == (not mine), (fills, f, whole)
            for x in mine:
                bar.land(nbytes)
            assert bar.phase == f // stages + 1 and bar.bytes == 0


# ---- on the GPU ---------------------------------------------------------------------------

def _ones(rows, cols, lead=0):
    return torch.ones(rows * cols + lead, dtype=torch.bfloat16, device="cuda")[lead:].view(rows, cols)


# M, N, K, elements that x and w start off 16 bytes: the split form, tiles of a
# pair on one accumulator and on two, loading threads for one operand or both.
FORMS = {"split": (64, 128, 1 << 24, 0, 0), "split_wide": (1300, 4096, 1 << 19, 0, 0),
         "pairs": (2000, 2000, 1 << 19, 0, 0), "two_accumulators": (4096, 8192, 1 << 18, 0, 0),
         "split_threads": (64, 128, 1 << 22, 1, 1), "split_both_ways": (64, 128, 1 << 22, 0, 1),
         "pairs_threads": (5000, 5000, 1 << 18, 1, 1), "pairs_both_ways": (4096, 4096, 1 << 18, 1, 0)}


@pytest.mark.gpu
@pytest.mark.parametrize("form", FORMS)
def test_a_wait_that_runs_out_ends_with_a_status(arx, form):
    M, N, K, xlead, wlead = FORMS[form]
    x, w = _ones(M, K, xlead), _ones(N, K, wlead)
    out = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    arx.arx_linear(x, w, out, status=status, copies=False, wait_us=1000)
    torch.cuda.synchronize()
    assert int(status) & 0xFF == arx.ARX_ETIMEOUT
    # The context and the SMs' memory are in order: the same call with the default limit is right.
    for _ in range(2):
        status.zero_()
        out.zero_()
        arx.arx_linear(x, w, out, status=status, copies=False)
        torch.cuda.synchronize()
        assert int(status) == 0
        assert bool((out == float(K)).all())


@pytest.mark.gpu
@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("act", ["none", "relu", "gelu", "gelu_tanh", "silu"])
def test_what_was_not_finished_is_nan(arx, form, act):
    # Without a status word: no element keeps what was there before.
    M, N, K, xlead, wlead = FORMS[form]
    x, w = _ones(M, K, xlead), _ones(N, K, wlead)
    out, z = (torch.full((M, N), 3.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    residual = torch.zeros_like(out)
    arx.arx_linear(x, w, out, residual=residual, z=z, act=getattr(arx, "ARX_ACT_" + act.upper()), copies=False, wait_us=1000)
    torch.cuda.synchronize()
    for t in (out, z):
        nan = torch.isnan(t)
        assert bool(nan.any()) and bool((t[~nan] == float(K)).all())


@pytest.mark.gpu
def test_gradients_that_were_not_finished_are_nan(arx):
    M, N, K = 1 << 19, 512, 1024
    x, d = _ones(M, K), _ones(M, N)
    dw = torch.full((N, K), 3.0, dtype=torch.bfloat16, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    arx.arx_linear_bwd(d, x, None, dw=dw, status=status, wait_us=100)
    torch.cuda.synchronize()
    nan = torch.isnan(dw)
    assert int(status) & 0xFF == arx.ARX_ETIMEOUT
    assert bool(nan.any()) and bool((dw[~nan] == float(M)).all())


NEIGHBOUR = """
import select, sys, torch
a = torch.randn(8192, 8192, device="cuda").bfloat16()
b = torch.empty_like(a)
torch.mm(a, a, out=b)
torch.cuda.synchronize()
print("ready", flush=True)
while not select.select([sys.stdin], [], [], 0)[0]:  # until the test closes it
    for _ in range(20):
        torch.mm(a, a, out=b)
    torch.cuda.synchronize()
"""


@pytest.mark.gpu
def test_time_of_another_process_on_the_gpu_does_not_count(arx):
    # A tile's products take 2.4 ms here; beside a busy process, whose time slices
    # suspend the kernel, they take about four times that.
    M, N, K = FORMS["two_accumulators"][:3]
    x, w = _ones(M, K), _ones(N, K)
    out = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    with subprocess.Popen([sys.executable, "-c", NEIGHBOUR], stdin=subprocess.PIPE, stdout=subprocess.PIPE, text=True) as p:
        try:
            assert p.stdout.readline() == "ready\n"
            for _ in range(20):
                arx.arx_linear(x, w, out, status=status, wait_us=5000)
                torch.cuda.synchronize()
        finally:
            p.stdin.close()
    assert p.returncode == 0
    assert int(status) == 0 and bool((out == float(K)).all())
