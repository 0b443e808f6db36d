"""Calls of the layer-wise QAT operators that their arguments allow or exclude: shared
memory, gradients, numbers, streams and graphs."""
import pytest
import torch

from bcjr_sum_product_b200 import inputs as I
from bcjr_sum_product_b200 import lib, qat

pytestmark = pytest.mark.gpu
DEV = "cuda"


def randn(*shape, seed=0):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(DEV)


def finished():
    torch.cuda.synchronize()
    assert lib.get_device_error() == 0


# ---------------------------------------------------------------- shared memory

def test_outputs_apart_from_inputs():
    """The momentum is written before the gradient is read for the last time, the weights are read with the
    others still needed: shared memory would give wrong results without a word."""
    w, g = randn(40, 60, seed=1), randn(40, 60, seed=2)
    m = torch.zeros_like(w)
    for bad in ((w, g, g), (w, w, m), (w, g, w)):
        before = [t.clone() for t in bad]
        with pytest.raises(ValueError, match="share memory"):
            lib.muon_step(*bad, 0.1)
        assert all(torch.equal(t, b) for t, b in zip(bad, before))
    room = randn(41, 60, seed=3)
    with pytest.raises(ValueError, match="share memory"):
        lib.muon_step(room[:40], g, room[1:], 0.1)
    # codes and a product in the same buffer
    buffer = torch.zeros(40 * 48 * 4, dtype=torch.uint8, device=DEV)
    q, s = lib.fp8_quantise(randn(40, 48, seed=4))
    codes = buffer[:40 * 48].view(q.dtype).view(40, 48)
    codes.copy_(q)
    out = buffer.view(torch.float32)[:1600].view(40, 40)
    for a, b in ((codes, q), (q, codes)):
        with pytest.raises(ValueError, match="share memory"):
            lib.fp8_matmul(a, s, b, s, out=out)
    assert torch.equal(codes.view(torch.uint8), q.view(torch.uint8))
    apart = buffer.view(torch.float32)[480:480 + 1600 - 160].view(36, 40)
    assert torch.equal(lib.fp8_matmul(codes[:36], s[:36], codes, s, out=apart), lib.fp8_matmul(q[:36], s[:36], q, s, out_dtype=torch.float32))
    finished()


def test_matrices_between_one_anothers_rows_are_apart():
    """Weights, gradient and momentum side by side in one buffer."""
    room = randn(30, 120, seed=5)
    w, g, m = room[:, :40], room[:, 40:80], room[:, 80:]
    want = lib.muon_step(w.clone(), g.clone(), m.clone(), 0.1)
    lib.muon_step(w, g, m, 0.1)
    finished()
    assert torch.equal(w, want[0]) and torch.equal(m, want[1])


# ---------------------------------------------------------------- autograd

def test_results_without_a_gradient_are_refused():
    x = randn(20, 40, seed=6).requires_grad_()
    y = x.detach()
    q, s = lib.fp8_quantise(y)
    for call in (lambda: lib.fp8_quantise(x), lambda: lib.fp8_quantise(y, minus=x), lambda: lib.orthogonalise(x),
                 lambda: lib.fp8_matmul(q, s, q, s, out=torch.zeros(20, 20, device=DEV, requires_grad=True))):
        with pytest.raises(RuntimeError, match="no derivative"):
            call()
    with torch.no_grad():
        assert torch.equal(lib.fp8_quantise(x)[0].view(torch.uint8), q.view(torch.uint8))
        assert torch.equal(lib.orthogonalise(x), lib.orthogonalise(y))
    finished()


def test_a_step_on_a_parameter_is_seen_by_autograd():
    """A graph that saved the weights does not go back with the changed ones."""
    w = torch.nn.Parameter(randn(20, 40, seed=7))
    m = torch.zeros(20, 40, device=DEV)
    loss = (w * w).sum()
    loss.backward()
    kept = (w * w).sum()
    before = (w._version, m._version)
    lib.muon_step(w, w.grad, m, 0.1)
    assert w._version > before[0] and m._version > before[1] and w.requires_grad and w.is_leaf
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        kept.backward()
    q, s = lib.fp8_quantise(m)
    out = torch.zeros(20, 20, device=DEV)
    lib.fp8_matmul(q, s, q, s, out=out)
    assert out._version > 0
    with torch.inference_mode():
        v = torch.ones(20, 40, device=DEV)
        lib.muon_step(v, v * 2, torch.zeros_like(v), 0.1)
    finished()


# ---------------------------------------------------------------- numbers

def test_no_values_of_k_give_zeros_in_rows_of_any_length():
    """Rows of more than 2^31 bytes too, and rows apart from one another."""
    n = (1 << 29) + 8
    for m, cols, keep in ((2, n, 0), (5, 33, 7), (1, 1 << 29, 0)):
        a, b = (lib.fp8_quantise(torch.zeros(r, 0, device=DEV)) for r in (m, cols))
        room = torch.full((m, cols + keep), 3.0, device=DEV)
        lib.fp8_matmul(*a, *b, out=room[:, :cols])
        finished()
        assert not bool(room[:, :cols].any()) and bool((room[:, cols:] == 3).all())
        del room
        torch.cuda.empty_cache()


def test_numbers_of_steps():
    g = randn(20, 30, seed=8)
    want = lib.orthogonalise(g, steps=3)
    assert torch.equal(lib.orthogonalise(g, steps=3.0), want)
    for bad in (2.5, float("nan")):
        with pytest.raises(ValueError):
            lib.orthogonalise(g, steps=bad)
        with pytest.raises(ValueError):
            lib.muon_step(g.clone(), g, torch.zeros_like(g), 0.1, steps=bad)
    # what a 32-bit number would wrap around to one in range
    for many in (65, 2 ** 31, 2 ** 32 + 5, 2 ** 70):
        for coeffs in (None, (1.875, -1.25, 0.375)):
            with pytest.raises(lib.BcjrError) as e:
                lib.orthogonalise(g, steps=many, coeffs=coeffs)
            assert e.value.status == lib.BCJR_ERR_UNSUPPORTED
    for few in (0, -1, -2 ** 32 + 5):
        with pytest.raises(lib.BcjrError) as e:
            lib.orthogonalise(g, steps=few)
        assert e.value.status == lib.BCJR_ERR_INVALID_ARG
    finished()


# ---------------------------------------------------------------- precision of a layer's loss

def test_products_of_a_layers_loss():
    """Against 64 bits: fp32; and 8-bit operands, whose errors are those of their codes: x and the residual off by at
    most 2^-4 of an entry in e4m3 (in the 2-norm 2^-4 / sqrt(3) of the whole), R by 2^-9 as bf16 and by 2^-3 or 2^-4 as
    codes; errors of a product's two sides add up as independent ones."""
    tokens, out, inner = 512, 640, 1024
    x, soft, target = randn(tokens, inner, seed=9), randn(out, inner, seed=10), randn(out, inner, seed=11)
    r64 = x.double() @ (soft.double() - target.double()).t()
    g64 = 2.0 / tokens * (r64.t() @ x.double())
    off = lambda got, want: float((got.double() - want).norm() / want.norm())  # noqa: E731
    r, g = qat.layer_loss_fp32(soft, target, x)
    assert off(r, r64) <= 2.0 ** -18 and off(g, g64) <= 2.0 ** -18
    operands = qat.layer_operands(x)
    errors = {}
    for r_dtype, step in ((torch.float8_e5m2, 2.0 ** -3), (torch.float8_e4m3fn, 2.0 ** -4)):
        r, g = qat.layer_loss(soft, target, operands, r_dtype=r_dtype)
        code = 2.0 ** -4 / 3 ** 0.5
        assert off(r, r64) <= code * 2 ** 0.5
        assert off(g, g64) <= (2 * code ** 2 + (step / 3 ** 0.5) ** 2 + code ** 2) ** 0.5
        errors[r_dtype] = off(g, g64)
    assert errors[torch.float8_e4m3fn] < errors[torch.float8_e5m2]
    finished()


@pytest.mark.parametrize("products", ["e5m2", "e4m3", "fp32"])
def test_driver_with_either_products(products):
    shape, L, k, V = (64, 128), 8, 2, 1
    target, c, _ = I.random_case(L, k, V, 128, 64, seed=45)
    t, cb, x = target.to(DEV), c.to(DEV), randn(96, shape[1], seed=46)
    out = qat.run(t, cb, L, k, V, 0.3, 0.1, 2, 1e-2, x=x, shape=shape, optimizer="muon", products=products)
    w, m, losses = t.clone(), torch.zeros_like(t), []
    for T in qat.anneal(0.3, 0.1, 2):
        soft, _ = lib.soft_codeword(w, cb, L, k, V, T)
        if products == "fp32":
            r, g = qat.layer_loss_fp32(soft.view(shape), t.view(shape), x)
        else:
            r, g = qat.layer_loss(soft.view(shape), t.view(shape), qat.layer_operands(x),
                                  r_dtype=torch.float8_e4m3fn if products == "e4m3" else torch.float8_e5m2)
        losses.append(float(r.float().square().sum()) / 96)
        gw, _ = lib.vjp(w, cb, L, k, V, T, g.reshape(w.shape))
        lib.muon_step(w.view(shape), gw.view(shape), m.view(shape), 1e-2)
    finished()
    assert torch.equal(out["w"], w) and out["loss"] == pytest.approx(losses, rel=1e-5)


# ---------------------------------------------------------------- values of codes and scales

E8M0 = torch.float8_e8m0fnu


def scaled(q, block_rows):
    """Scales of 1 for codes of any value."""
    rows, cols = q.shape
    return torch.full((-(-rows // block_rows), -(-cols // 128)), 127, dtype=torch.uint8, device=DEV)


@pytest.mark.parametrize("m,n,k", [(5, 40, 300), (70, 140, 300), (1030, 2000, 600)])
def test_scales_that_are_nan_spoil_what_they_enter(m, n, k):
    """Over finite codes, and over zeros."""
    a, b = (randn(r, k, seed=s).to(torch.float8_e4m3fn) for r, s in ((m, 12), (n, 13)))
    room = [torch.zeros(t.shape[0], 608, dtype=torch.uint8, device=DEV) for t in (a, b)]
    for r, t in zip(room, (a, b)):
        r[:, :k] = t.view(torch.uint8)
    a, b = (r.view(torch.float8_e4m3fn)[:, :k] for r in room)
    room[0][3, 128:256] = 0
    sa, sb = scaled(a, 1), scaled(b, 128)
    sa[3, 1] = 255
    sb[n // 128, k // 128] = 255                       # the last rows' last values
    y = lib.fp8_matmul(a, sa.view(E8M0), b, sb.view(E8M0), out_dtype=torch.float32)
    finished()
    want = torch.zeros(m, n, dtype=torch.bool, device=DEV)
    want[3] = True
    want[:, n // 128 * 128:] = True
    assert torch.equal(torch.isnan(y), want)
    assert bool(torch.isfinite(y[~want]).all())


@pytest.mark.parametrize("m,n", [(5, 40), (1030, 2000)])
def test_scales_at_the_ends_of_their_range(m, n):
    """2^-127 and 2^127 are scales like any other; what the products' sums make of them stays in fp32."""
    k = 256
    x, w = randn(m, k, seed=14), randn(n, k, seed=15)
    a, b = x.to(torch.float8_e4m3fn), w.to(torch.float8_e4m3fn)
    one = torch.full((m, 2), 127, dtype=torch.uint8, device=DEV), torch.full((-(-n // 128), 2), 127, dtype=torch.uint8, device=DEV)
    plain = lib.fp8_matmul(a, one[0].view(E8M0), b, one[1].view(E8M0), out_dtype=torch.float32)
    for low, high in ((0, 254), (254, 0)):
        sa, sb = torch.full_like(one[0], low), torch.full_like(one[1], high)
        y = lib.fp8_matmul(a, sa.view(E8M0), b, sb.view(E8M0), out_dtype=torch.float32)
        assert torch.equal(y, plain)
    finished()


def test_infinite_codes():
    """e5m2 has infinities: theirs is the sum's, and with a zero or the other sign NaN."""
    a, b = torch.ones(3, 16, device=DEV), torch.ones(4, 16, device=DEV)
    a[1, 5] = float("inf")
    b[2, 5] = 0.0
    b[3, 5] = -1.0
    q, r = a.to(torch.float8_e5m2), b.to(torch.float8_e4m3fn)
    y = lib.fp8_matmul(q, scaled(q, 1).view(E8M0), r, scaled(r, 1).view(E8M0), out_dtype=torch.float32)
    finished()
    inf = float("inf")
    assert torch.equal(y[0], torch.tensor([16.0, 16.0, 15.0, 14.0], device=DEV)) and torch.equal(y[0], y[2])
    assert y[1, 0] == inf and y[1, 1] == inf and torch.isnan(y[1, 2]) and y[1, 3] == -inf


# ---------------------------------------------------------------- streams and graphs

def test_a_graph_of_two_streams():
    """Calls on both sides of a fork inside a capture, and after the join; replayed with new values."""
    x, w, m = randn(300, 520, seed=16), randn(700, 520, seed=17), torch.zeros(300, 520, device=DEV)
    big = randn(1100, 1200, seed=18)

    def work(side):
        main = torch.cuda.current_stream()
        qx = lib.fp8_quantise(x)
        side.wait_stream(main)
        with torch.cuda.stream(side):
            o = lib.orthogonalise(big)
            qw = lib.fp8_quantise(w, 128)
        p = lib.orthogonalise(x)
        main.wait_stream(side)
        y = lib.fp8_matmul(*qx, *qw)
        lib.muon_step(x, p, m, 0.1)
        return o, p, y

    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = work(side)
    for turn in range(3):
        start = randn(300, 520, seed=20 + turn)
        x.copy_(start)
        m.fill_(0.5)
        big.copy_(randn(1100, 1200, seed=30 + turn))
        want = [t.clone() for t in work(torch.cuda.Stream())] + [x.clone(), m.clone()]
        x.copy_(start)
        m.fill_(0.5)
        torch.cuda.synchronize()
        graph.replay()
        finished()
        for got, wanted in zip((*out, x, m), want):
            assert torch.equal(got, wanted)


def test_a_batch_of_one_matrix_again_and_again():
    """A broadcast batch, windows that overlap, and rows of one matrix of a batch apart from the next."""
    g = randn(40, 90, seed=19)
    one = lib.orthogonalise(g)
    many = lib.orthogonalise(g.expand(5, 40, 90))
    windows = lib.orthogonalise(g.as_strided((3, 20, 90), (10 * 90, 90, 1)))
    apart = lib.orthogonalise(torch.stack([g, g], 1).transpose(0, 1))
    finished()
    # (the number of blocks that sum a norm depends on the batch)
    for got in (*many, *apart):
        assert float((got.float() - one.float()).norm()) <= 2.0 ** -8 * float(one.float().norm())
    for i in range(3):
        assert float((windows[i].float() - lib.orthogonalise(g[10 * i:10 * i + 20]).float()).norm()) <= 2.0 ** -8 * 20 ** 0.5
