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
