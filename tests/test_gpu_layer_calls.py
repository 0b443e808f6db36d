"""Calls of the layer-wise QAT operators that their arguments allow or exclude: shared
memory, gradients, numbers, streams and graphs."""
import pytest
import torch

from bcjr_sum_product_b200 import lib

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
