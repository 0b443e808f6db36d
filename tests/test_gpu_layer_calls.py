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
