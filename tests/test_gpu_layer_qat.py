"""The layer-wise QAT operators together, as the driver runs them, and how they may
be called: streams, graphs, views, in sequence and at once."""
import math
import os
import subprocess
import sys
import threading

import pytest
import torch

import layer_reference as ref
from bcjr_sum_product_b200 import inputs as I
from bcjr_sum_product_b200 import lib, qat

pytestmark = pytest.mark.gpu
DEV = "cuda"
E4M3, E5M2 = torch.float8_e4m3fn, torch.float8_e5m2


def randn(*shape, seed=0, scale=1.0):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)) * scale


def finished():
    torch.cuda.synchronize()
    assert lib.get_device_error() == 0


# ---------------------------------------------------------------- loss and gradient of a layer

@pytest.mark.parametrize("tokens,out,inner", [(1, 16, 32), (70, 130, 200), (333, 256, 96), (512, 64, 1000)])
def test_layer_loss_on_its_codes(tokens, out, inner):
    """R is the product of the codes' values, to bf16; the gradient that of R's codes
    (e5m2: half a step is 2^-3 of the value, 2^-17 of the scale below the normal range,
    the scale at most 2 max|r| / 57344) with the activations' column codes."""
    x, soft, target = randn(tokens, inner, seed=1), randn(out, inner, seed=2), randn(out, inner, seed=3)
    operands = qat.layer_operands(x.to(DEV))
    r, g = qat.layer_loss(soft.to(DEV), target.to(DEV), operands)
    finished()
    d, sd = lib.fp8_quantise(soft.to(DEV), 128, minus=target.to(DEV))
    vx, vd, vxt = ref.values(operands[0], operands[1], 1), ref.values(d, sd, 128), ref.values(operands[2], operands[3], 1)
    r_ref = vx @ vd.t()
    sums = (inner / 32 + 40) * 2.0 ** -23 * (vx.abs() @ vd.abs().t())
    dr = sums + 2.0 ** -8 * (r_ref.abs() + sums)
    assert bool(((r.cpu().double() - r_ref).abs() <= dr).all())
    most = r_ref.abs().max(dim=0, keepdim=True).values + dr.max(dim=0, keepdim=True).values
    dq = dr + 2.0 ** -3 * (r_ref.abs() + dr) + 2.0 ** -17 * 2 * most / 57344
    g_ref = 2.0 / tokens * (r_ref.t() @ vxt.t())
    # alpha = 2 / tokens is rounded to fp32, as is the result
    tol = 2.0 / tokens * (dq.t() @ vxt.abs().t()) + (tokens / 32 + 42) * 2.0 ** -23 * 2.0 / tokens * ((r_ref.abs() + dq).t() @ vxt.abs().t())
    assert bool(((g.cpu().double() - g_ref).abs() <= tol).all())


def test_layer_gradient_against_differences():
    """Activations and residuals that their codes hold exactly, so that only R's own
    e5m2 codes (2^-3 of the value) stand between the gradient and the loss's central
    differences, which are exact for a quadratic."""
    g = torch.Generator().manual_seed(4)
    tokens, out, inner = 48, 24, 16
    x = torch.randint(-2, 3, (tokens, inner), generator=g).double()
    d = torch.randint(-2, 3, (out, inner), generator=g).double() / 4
    target = randn(out, inner, seed=5).mul(256).round().div(256)      # soft = target + d is exact
    soft = target.double() + d
    _, grad = qat.layer_loss(soft.float().to(DEV), target.to(DEV), qat.layer_operands(x.float().to(DEV)))
    finished()
    loss = lambda e: float((x @ (d + e).t()).square().sum()) / tokens  # noqa: E731
    r = x @ d.t()
    for seed in range(4):
        v = randn(out, inner, seed=10 + seed).double()
        v /= v.norm()
        slope = (loss(v) - loss(-v)) / 2
        bound = 2.0 / tokens * float((2.0 ** -3 * r.abs() * (x @ v.t()).abs()).sum()) + 1e-5 * abs(slope)
        assert abs(float((grad.cpu().double() * v).sum()) - slope) <= bound


def test_gradients_of_a_product():
    """Forward, input gradient and weight gradient of y = x w^T, each as one call on codes
    of one pass over each operand."""
    x, w, dy = randn(100, 300, seed=6), randn(140, 300, seed=7), randn(100, 140, seed=8)
    qx = lib.fp8_quantise(x.to(DEV), 1, E4M3, layout="both")
    qw = lib.fp8_quantise(w.to(DEV), 128, E4M3, layout="both")
    qy = lib.fp8_quantise(dy.to(DEV), 1, E5M2, layout="both")
    y = lib.fp8_matmul(*qx[:2], *qw[:2], out_dtype=torch.float32)
    dx = lib.fp8_matmul(*qy[:2], *qw[2:], out_dtype=torch.float32)
    dw = lib.fp8_matmul(*qy[2:], *qx[2:], out_dtype=torch.float32)
    finished()
    vx, vw, vy = ref.values(*qx[:2], 1), ref.values(*qw[:2], 128), ref.values(*qy[:2], 1)
    vxt, vwt, vyt = ref.values(*qx[2:], 1), ref.values(*qw[2:], 128), ref.values(*qy[2:], 1)
    assert torch.equal(vwt, vw.t())                  # one scale for a block whichever way it is read
    for got, p, q in ((y, vx, vw), (dx, vy, vwt), (dw, vyt, vxt)):
        tol = (p.shape[1] / 32 + 41) * 2.0 ** -23 * (p.abs() @ q.abs().t())
        assert bool(((got.cpu().double() - p @ q.t()).abs() <= tol).all())


# ---------------------------------------------------------------- the driver

@pytest.mark.parametrize("optimizer,layer", [("muon", False), ("muon", True), ("sgd", True)])
def test_driver_runs_the_operators(optimizer, layer):
    """Two steps of the driver are the two steps written out."""
    shape, L, k, V, lr, lr_c = (64, 128), 8, 2, 1, 1e-2, 1e-3
    target, c, _ = I.random_case(L, k, V, 128, 64, seed=41)
    t, cb = target.to(DEV), c.to(DEV)
    x = randn(96, shape[1], seed=42).to(DEV) if layer else None
    out = qat.run(t, cb, L, k, V, 0.3, 0.1, 2, lr, lr_c, x=x, shape=shape, optimizer=optimizer, mu=0.9, weight_decay=0.05)
    w, cc, m = t.clone(), cb.clone(), torch.zeros_like(t)
    losses = []
    for T in qat.anneal(0.3, 0.1, 2):
        soft, _ = lib.soft_codeword(w, cc, L, k, V, T)
        if layer:
            r, g = qat.layer_loss(soft.view(shape), t.view(shape), qat.layer_operands(x))
            losses.append(float(r.float().square().sum()) / 96)
        else:
            g = 2 * (soft - t)
            losses.append(float((soft - t).square().sum()))
        gw, gc = lib.vjp(w, cc, L, k, V, T, g.view(w.shape))
        if optimizer == "muon":
            lib.muon_step(w.view(shape), gw.view(shape), m.view(shape), lr, mu=0.9, weight_decay=0.05)
        else:
            w.mul_(1 - lr * 0.05).sub_(gw, alpha=lr)
        cc.sub_(gc, alpha=lr_c)
    finished()
    # the same calls on the same values: the same bits
    assert torch.equal(out["w"], w) and torch.equal(out["codebook"], cc)
    assert out["loss"] == pytest.approx(losses, rel=1e-5)
    assert out["drift_budget"] >= out["max_drift"]
    assert ("hard_layer_mse_qat" in out) == layer


def test_driver_on_another_stream():
    target, c, _ = I.random_case(8, 2, 1, 128, 64, seed=43)
    t, cb, x = target.to(DEV), c.to(DEV), randn(40, 128, seed=44).to(DEV)
    kw = dict(x=x, shape=(64, 128), optimizer="muon")
    a = qat.run(t, cb, 8, 2, 1, 0.3, 0.1, 2, 1e-2, **kw)
    b = qat.run(t, cb, 8, 2, 1, 0.3, 0.1, 2, 1e-2, stream=torch.cuda.Stream(), **kw)
    finished()
    assert torch.equal(a["w"], b["w"]) and a["loss"] == b["loss"]


def test_command_with_layer_loss_and_muon(capsys):
    import json
    assert qat.main(["--workload", "tiny", "--loss", "layer", "--tokens", "33", "--optimizer", "muon", "--steps", "2"]) == 0
    rep = json.loads(capsys.readouterr().out.strip().splitlines()[-1])
    assert rep["steps"] == 2 and math.isfinite(rep["hard_layer_mse_qat"])


# ---------------------------------------------------------------- streams, graphs, repeats

def cases(seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.randn(300, 520, generator=g, device=DEV)
    return x, torch.randn(700, 520, generator=g, device=DEV)


def chain(x, w, momentum):
    """Every operator once, each on what the one before it gave."""
    qx, qw = lib.fp8_quantise(x, layout="both"), lib.fp8_quantise(w, 128)
    y = lib.fp8_matmul(*qx[:2], *qw)
    o = lib.orthogonalise(y)
    h = lib.orthogonalise(y[:100, :90], out_dtype=torch.float16)
    lib.muon_step(x, x * 0.5, momentum, 0.1, weight_decay=0.1)
    return qx[2], qx[3], y, o, h, x, momentum


def bits(ts):
    return [t.clone().view(torch.uint8) if t.element_size() == 1 else t.clone() for t in ts]


def same(a, b):
    return all(torch.equal(p, q) for p, q in zip(a, b))


def test_repeats_are_the_same_bits():
    runs = []
    for _ in range(3):
        x, w = cases(1)
        runs.append(bits(chain(x, w, torch.ones_like(x))))
    finished()
    assert same(runs[0], runs[1]) and same(runs[0], runs[2])


def test_large_products_repeat_the_same_bits():
    x = torch.randn(2100, 4096, generator=torch.Generator(device=DEV).manual_seed(2), device=DEV)
    q = lib.fp8_quantise(x)
    a, b = lib.fp8_matmul(*q, *q, out_dtype=torch.float32), lib.fp8_matmul(*q, *q, out_dtype=torch.float32)
    o, p = lib.orthogonalise(x), lib.orthogonalise(x)
    finished()
    assert torch.equal(a, b) and torch.equal(o, p)


def test_streams_at_once():
    """Calls on two streams at once do not share scratch."""
    want = []
    for seed in (3, 4):
        x, w = cases(seed)
        want.append(bits(chain(x, w, torch.zeros_like(x))))
    finished()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    data = [cases(3), cases(4)]
    torch.cuda.synchronize()
    for _ in range(4):
        got = []
        for (x, w), s in zip(data, streams):
            with torch.cuda.stream(s):
                x = x.clone()
                got.append(bits(chain(x, w, torch.zeros_like(x))))
    finished()
    assert same(got[0], want[0]) and same(got[1], want[1])


def test_two_host_threads():
    want, data = [], [cases(8), cases(9)]
    for x, w in data:
        want.append(bits(chain(x.clone(), w, torch.zeros_like(x))))
    finished()
    got = [None, None]

    def work(i):
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(5):
                x = data[i][0].clone()
                got[i] = bits(chain(x, data[i][1], torch.zeros_like(x)))
            torch.cuda.current_stream().synchronize()

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join(120)
    finished()
    assert same(got[0], want[0]) and same(got[1], want[1])


def test_stream_argument():
    x, w = cases(5)
    want_q = lib.fp8_quantise(x, layout="both")
    b = lib.fp8_quantise(w, 128)
    want = lib.fp8_matmul(*want_q[:2], *b), lib.orthogonalise(x)
    finished()
    for s in (torch.cuda.Stream(), torch.cuda.Stream().cuda_stream):
        stream = s if isinstance(s, torch.cuda.Stream) else torch.cuda.ExternalStream(s)
        stream.wait_stream(torch.cuda.current_stream())
        q = lib.fp8_quantise(x, layout="both", stream=s)
        y, o = lib.fp8_matmul(*q[:2], *b, stream=s), lib.orthogonalise(x, stream=s)
        stream.synchronize()
        assert torch.equal(q[2].view(torch.uint8), want_q[2].view(torch.uint8))
        assert torch.equal(y, want[0]) and torch.equal(o, want[1])
    finished()


def test_graphs():
    """Two captured graphs, replayed in turn and at once on two streams, on new values."""
    graphs = []
    for seed in (6, 7):
        x, w = cases(seed)
        m = torch.zeros_like(x)
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            chain(x.clone(), w, m.clone())                # first use outside the capture
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = chain(x, w, m)
        graphs.append((graph, x, w, m, out))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for turn in range(3):
        want = []
        for i, (graph, x, w, m, out) in enumerate(graphs):
            nx, nw = cases(20 + 2 * turn + i)
            x.copy_(nx)
            w.copy_(nw)
            m.fill_(0.25)
            want.append(bits(chain(nx, nw, torch.full_like(nx, 0.25))))
        torch.cuda.synchronize()
        for (graph, *_), s in zip(graphs, streams):
            if turn < 2:
                graph.replay()
            else:
                with torch.cuda.stream(s):
                    graph.replay()
        finished()
        for (_, _, _, _, out), wt in zip(graphs, want):
            assert same(bits(out), wt)


def test_first_calls_inside_a_capture():
    """Nothing that a first call sets up (attributes, entry points, the scratch pool)
    disturbs a capture; in a process of its own, where they are the first."""
    code = """
import torch
from bcjr_sum_product_b200 import lib
x, w = torch.randn(300, 520, device="cuda"), torch.randn(300, 520, device="cuda")
m = torch.zeros_like(x)
big = torch.randn(2048, 2048, device="cuda")
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    q = lib.fp8_quantise(x, layout="both")
    y = lib.fp8_matmul(*q[:2], *q[:2])
    o = lib.orthogonalise(x)
    p = lib.orthogonalise(big)
    lib.muon_step(w, x, m, 0.1)
g.replay()
torch.cuda.synchronize()
assert lib.get_device_error() == 0
assert torch.equal(o, lib.orthogonalise(x)) and torch.equal(p, lib.orthogonalise(big)) and torch.equal(y, lib.fp8_matmul(*q[:2], *q[:2]))
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    run = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert run.returncode == 0, run.stderr[-2000:]


def test_offsets_past_32_bits():
    """Codes and outputs of more than 2^32 bytes: the last rows."""
    free, _ = torch.cuda.mem_get_info()
    if free < 60 << 30:
        pytest.skip("needs 60 GB of device memory")
    rows, cols = 66000, 66000
    x = torch.zeros(rows, cols, dtype=torch.bfloat16, device=DEV)
    tail = torch.randn(70, cols, generator=torch.Generator(device=DEV).manual_seed(9), device=DEV).to(torch.bfloat16)
    x[-70:] = tail
    q, s, qt, st = lib.fp8_quantise(x, layout="both")
    small, ssmall = lib.fp8_quantise(tail)
    finished()
    assert torch.equal(q[-70:].view(torch.uint8), small.view(torch.uint8))
    assert torch.equal(s[-70:].view(torch.uint8), ssmall.view(torch.uint8))
    assert int(q[:-70].view(torch.uint8).max()) == 0
    # down the columns the last block of rows is all that is not zero
    want, _ = lib.fp8_quantise(x[rows // 128 * 128 - 128:, -300:], layout="cols")
    assert torch.equal(qt[-300:, rows // 128 * 128 - 128:].view(torch.uint8), want.view(torch.uint8))
    del x, qt, st
    y = lib.fp8_matmul(q, s, small, ssmall, out_dtype=torch.float32)
    z = lib.fp8_matmul(q[-70:], s[-70:], small, ssmall, out_dtype=torch.float32)
    assert float(y[:-70].abs().max()) == 0.0
    tol = (cols / 32 + 40) * 2.0 ** -22 * float(z.diagonal().max())
    assert float((y[-70:] - z).abs().max()) <= tol
    del y
    k = lib.fp8_matmul(q[:, :64], s[:, :1], q[:, :64], s[:, :1])     # 66000 x 66000 outputs
    last = lib.fp8_matmul(q[-70:, :64], s[-70:, :1], q[-70:, :64], s[-70:, :1])
    finished()
    assert torch.equal(k[-70:, -70:], last)
    assert float(k[:-70, :1000].abs().max()) == 0.0


# ---------------------------------------------------------------- waits that run out

@pytest.mark.parametrize("m,n,k", [(20, 256, 8192), (300, 400, 1024), (2048, 2048, 1024), (2048, 4096, 2048)])
def test_products_whose_waits_run_out_store_nothing(monkeypatch, m, n, k):
    """With BCJR_DENSE_TEST_NOFILL=1 one block of each cluster fetches a single stage.  The
    waits for the rest run out after 1 s; no block stores sums that lack it, its peers
    neither; the next call is right."""
    x, w = randn(m, k, seed=61).to(DEV), randn(n, k, seed=62).to(DEV)
    a, b = lib.fp8_quantise(x), lib.fp8_quantise(w, 128)
    want = lib.fp8_matmul(*a, *b, out_dtype=torch.float32)
    finished()
    out = torch.full((m, n), 7.0, device=DEV)
    monkeypatch.setenv("BCJR_DENSE_TEST_NOFILL", "1")
    lib.fp8_matmul(*a, *b, out=out)
    torch.cuda.synchronize()
    assert lib.get_device_error() == lib.BCJR_ERR_TIMEOUT
    assert bool((out == 7).all())
    monkeypatch.delenv("BCJR_DENSE_TEST_NOFILL")
    assert lib.get_device_error() == 0
    assert torch.equal(lib.fp8_matmul(*a, *b, out_dtype=torch.float32), want)
    finished()


@pytest.mark.parametrize("rows,cols", [(512, 2048), (2048, 2048)])
def test_a_muon_step_whose_waits_run_out_leaves_the_weights(monkeypatch, rows, cols):
    w, g = randn(rows, cols, seed=63).to(DEV), randn(rows, cols, seed=64).to(DEV)
    before = w.clone()
    monkeypatch.setenv("BCJR_DENSE_TEST_NOFILL", "1")
    lib.muon_step(w, g, torch.zeros_like(g), 0.1, steps=1)
    torch.cuda.synchronize()
    assert lib.get_device_error() == lib.BCJR_ERR_TIMEOUT
    assert torch.equal(w, before)
    monkeypatch.delenv("BCJR_DENSE_TEST_NOFILL")
    lib.muon_step(w, g, torch.zeros_like(g), 0.1, steps=1)
    finished()
    assert not torch.equal(w, before)
