"""How near the orthogonalisation and the Muon step come to their 64-bit forms, on
updates of every kind: few directions, many, nearly orthogonal, thin, long, and the
sizes of whole layers."""
import math

import pytest
import torch

import layer_reference as ref
from bcjr_sum_product_b200 import lib

pytestmark = pytest.mark.gpu
DEV = "cuda"
HALF_STEP = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}


def randn(*shape, seed=0):
    return torch.randn(*shape, generator=torch.Generator(device=DEV).manual_seed(seed), device=DEV)


def low_rank(rows, cols, rank, seed):
    return randn(rows, rank, seed=seed) @ randn(rank, cols, seed=seed + 1)


def finished():
    torch.cuda.synchronize()
    assert lib.get_device_error() == 0


def relative(got, want):
    err = torch.linalg.vector_norm(got.double() - want, dim=(-2, -1)) / torch.linalg.vector_norm(want, dim=(-2, -1))
    return float(err.max())


def orthogonal_part(u, **kw):
    """What muon_step adds to weights of zero, from momentum zero without nesterov: -orthogonalise(u) in fp32."""
    w = torch.zeros(u.shape, device=DEV)
    lib.muon_step(w, u, torch.zeros(u.shape, device=DEV), 1.0, mu=0.0, nesterov=False, scale=1.0, **kw)
    return -w


# ---------------------------------------------------------------- few directions

def bound(steps, paired):
    """2-norm of the error over that of the result.  P and B are rounded to 11 bits, their diagonals to 22: independent
    errors of at most 2^-11 / sqrt(3) of each in the 2-norm.  B x changes in proportion to B's; P's enters through
    b + 2 c t, up to twice the value of a + b t + c t^2 where singular values end up (t from 0.5 to 1.3), so 1 + 4
    squares a step; the first two steps at once round three products more, each counted like P.  The last step's X, one plane of
    11 bits, grows at most 3.4445 times (on its own, so the sum); 22 bits at most 485 times."""
    one = 2.0 ** -11 / math.sqrt(3)
    squares = 5 * steps + (12 if paired else 0)
    return math.sqrt(squares) * one + 3.4445 * one + 485 * 2.0 ** -11 * one


def rounded(tol, dtype):
    """With the result's own rounding, at most half a step / sqrt(3) in the 2-norm and independent of what came before."""
    return math.hypot(tol, HALF_STEP[dtype] / math.sqrt(3))


SHAPES = [(512, 512), (200, 700), (333, 130), (16, 1000), (64, 64), (129, 129), (1100, 900), (1536, 6145), (6200, 1500)]


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("rank", [1, 8, 60, 250])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_updates_of_few_directions(rows, cols, rank, dtype):
    """A gradient summed over few tokens has few directions; the others hold nothing but
    roundings, and every step multiplies those by 3.4445.  (A bf16 update has its own roundings in them, which are
    part of the matrix.)"""
    g = low_rank(rows, cols, min(rank, rows, cols), seed=rows + cols + rank).to(dtype)
    want = ref.newton_schulz(g)
    tol = bound(5, min(rows, cols) >= 1500)
    out, u = lib.orthogonalise(g), orthogonal_part(g)
    finished()
    assert relative(u, want) <= tol
    assert relative(out, want) <= rounded(tol, torch.bfloat16)


def test_few_directions_in_a_batch():
    g = torch.stack([low_rank(130, 333, r, seed=50 + r) for r in (1, 2, 5, 17, 60, 130)])
    for x in (g, g.mT.contiguous()):
        out = lib.orthogonalise(x)
        finished()
        assert relative(out, ref.newton_schulz(x)) <= rounded(bound(5, False), torch.bfloat16)


@pytest.mark.parametrize("coeffs", [(1.875, -1.25, 0.375), [(3.0, -3.2, 1.2), (2.0, -1.5, 0.5), (0.9, 0.05, 0.0), (3.4445, -4.7750, 2.0315)],
                                    [(0.5, 0.0, 0.0), (3.0, -3.2, 1.2), (2.0, -1.5, 0.5), (1.0, 0.0, 0.0)]])
def test_few_directions_with_other_coefficients(coeffs):
    """Steps that amplify less, or nothing, take the second plane of X or leave it in any order."""
    co = coeffs if isinstance(coeffs, list) else [coeffs] * 4
    for g in (low_rank(150, 400, 3, seed=70), low_rank(400, 150, 3, seed=71)):
        u = orthogonal_part(g, steps=4, coeffs=coeffs)
        finished()
        # any X whose second plane is left out may grow four times
        tol = 3 * 4 * 2.0 ** -12 + 4 * 4 * 2.0 ** -11 / math.sqrt(3)
        assert relative(u, ref.newton_schulz(g, 4, co)) <= tol


# ---------------------------------------------------------------- nearly constant diagonals

@pytest.mark.parametrize("rows,cols", [(33, 5000), (160, 6788), (5632, 165), (16, 100), (64, 300), (400, 30000), (20000, 300), (257, 6000),
                                       (520, 12000), (1, 50), (40, 1)])
def test_thin_and_long_updates(rows, cols):
    """Rows that are nearly orthogonal: the diagonals of P and B are nearly constant, and their roundings would go one
    way.  Weights of fp32 show all of it."""
    g = randn(rows, cols, seed=rows + cols)
    want = ref.newton_schulz(g)
    out, u = lib.orthogonalise(g), orthogonal_part(g)
    finished()
    assert relative(u, want) <= bound(5, min(rows, cols) >= 512)
    assert relative(out, want) <= rounded(bound(5, min(rows, cols) >= 512), torch.bfloat16)


@pytest.mark.parametrize("side", [40, 130, 500, 700])
def test_updates_that_are_orthogonal_already(side):
    g, _ = torch.linalg.qr(randn(side, side, seed=side).double())
    g = g.float().contiguous()
    u = orthogonal_part(g)
    finished()
    assert relative(u, ref.newton_schulz(g)) <= bound(5, False)


@pytest.mark.parametrize("rows,cols", [(200, 700), (1536, 6145)])
def test_the_default_coefficients_are_those_given(rows, cols):
    g = randn(rows, cols, seed=72)
    assert torch.equal(lib.orthogonalise(g), lib.orthogonalise(g, coeffs=lib.MUON_COEFFS))
    finished()


@pytest.mark.parametrize("shape", [(32767, 3, 5), (1, 1, 65536), (1, 65536, 1), (1, 65536, 9), (2, 7, 65536)])
@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float16])
def test_largest_extents(shape, out_dtype):
    g = randn(*shape, seed=73)
    out = lib.orthogonalise(g, out_dtype=out_dtype)
    finished()
    # single matrices of a batch this large may have roundings that agree: of at most five values of k
    assert relative(out, ref.newton_schulz(g)) <= 3 * rounded(bound(5, False), out_dtype)


# ---------------------------------------------------------------- few rows

@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 7), (2, 2), (2, 5), (5, 2), (3, 3), (4, 9), (8, 8), (30, 8), (16, 16), (31, 31),
                                       (7, 1100), (3000, 5)])
def test_every_matrix_of_few_rows(rows, cols):
    """Too few entries for roundings to average out: the worst of thousands of matrices.  An entry of 22 bits is off
    by at most 2^-22, sums over few values of k by five steps of 2^-23, and what is added to X grows by what is
    left of the five steps, 682 times in all; the Gram matrix of a long one has X's 11 bits averaged along it, counted
    three times a step as above."""
    n = min(32767, 1000000 // (rows * cols))
    g = randn(n, rows, cols, seed=rows + 40 * cols)
    want = ref.newton_schulz(g)
    long_side = max(rows, cols)
    tol = 682 * (2.0 ** -22 + 5 * 2.0 ** -23) + (15 * 2.0 ** -11 / math.sqrt(3 * long_side) if long_side >= 1024 else 0.0)
    out, fine = lib.orthogonalise(g), lib.orthogonalise(g, out_dtype=torch.float16)
    finished()
    assert relative(out, want) <= tol + HALF_STEP[torch.bfloat16]
    assert relative(fine, want) <= tol + HALF_STEP[torch.float16]
    for i in range(0, n, max(1, n // 40)):
        assert relative(orthogonal_part(g[i]), want[i]) <= tol


@pytest.mark.parametrize("rows,cols", [(512, 512), (200, 700), (1536, 6145), (6200, 1500), (333, 130)])
@pytest.mark.parametrize("strong,ratio", [(1, 1e2), (1, 1e4), (6, 30.0), (40, 1e3)])
def test_few_directions_far_above_the_rest(rows, cols, strong, ratio):
    """The rest of full rank below them: where the result lives after five steps depends on how far."""
    g = low_rank(rows, cols, strong, seed=91)
    rest = randn(rows, cols, seed=93)
    g = g + rest * float(torch.linalg.vector_norm(g) / torch.linalg.vector_norm(rest)) / ratio
    want = ref.newton_schulz(g)
    u = orthogonal_part(g)
    finished()
    assert relative(u, want) <= bound(5, min(rows, cols) >= 1500)


def test_power_law_spectra():
    """Singular values i^-p."""
    for rows, cols in ((300, 500), (1100, 1000)):
        k = min(rows, cols)
        q, _ = torch.linalg.qr(randn(rows, k, seed=94).double())
        r, _ = torch.linalg.qr(randn(cols, k, seed=95).double())
        for p in (0.25, 0.5, 1.0, 2.0, 4.0):
            g = ((q * torch.arange(1, k + 1, device=DEV).double() ** -p) @ r.mT).float().contiguous()
            u = orthogonal_part(g)
            finished()
            assert relative(u, ref.newton_schulz(g)) <= bound(5, False)


@pytest.mark.parametrize("batch,rows,cols", [(3, 640, 1000), (3, 1000, 640), (2, 513, 513), (5, 512, 600), (2, 700, 530)])
@pytest.mark.parametrize("rank", [1, 30, 300, None])
def test_batches_of_512_rows_and_more(batch, rows, cols, rank):
    """Where X's second plane meets B's diagonal alone: each matrix of a batch its own, in single blocks and pairs."""
    g = torch.stack([randn(rows, cols, seed=200 + i) if rank is None else low_rank(rows, cols, rank + i, seed=200 + i) for i in range(batch)])
    out = lib.orthogonalise(g)
    finished()
    assert relative(out, ref.newton_schulz(g)) <= rounded(bound(5, False), torch.bfloat16)


@pytest.mark.parametrize("rows,cols", [(600, 900), (900, 600), (2048, 2048), (1536, 6145)])
@pytest.mark.parametrize("coeffs", [(1.875, -1.25, 0.375), [(0.5, 0.0, 0.0), (3.0, -3.2, 1.2), (2.0, -1.5, 0.5), (1.0, 0.0, 0.0)]])
def test_other_coefficients_of_large_matrices(rows, cols, coeffs):
    co = coeffs if isinstance(coeffs, list) else [coeffs] * 4
    for g in (low_rank(rows, cols, 3, seed=96), randn(rows, cols, seed=98)):
        u = orthogonal_part(g, steps=4, coeffs=coeffs)
        finished()
        # as for small ones: any X whose second plane is left out may grow four times
        tol = 3 * 4 * 2.0 ** -12 + 4 * 4 * 2.0 ** -11 / math.sqrt(3)
        assert relative(u, ref.newton_schulz(g, 4, co)) <= tol
