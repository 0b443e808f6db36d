"""The layer-wise QAT operators against their plain 64-bit forms."""
import math

import numpy as np
import pytest
import torch

import layer_reference as ref
from bcjr_sum_product_b200 import lib

pytestmark = pytest.mark.gpu
DEV = "cuda"
E4M3, E5M2 = torch.float8_e4m3fn, torch.float8_e5m2
HALF_STEP = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}


def randn(*shape, seed=0, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(*shape, generator=g) * scale


def finished():
    torch.cuda.synchronize()
    assert lib.get_device_error() == 0


# ---------------------------------------------------------------- quantisation

def check_codes(got_q, got_s, v, block_rows, dtype):
    q, s = ref.quantise(v, block_rows, dtype)
    assert tuple(got_q.shape) == q.shape and tuple(got_s.shape) == s.shape
    np.testing.assert_array_equal(got_s.cpu().float().double().numpy(), s)
    np.testing.assert_array_equal(got_q.cpu().double().numpy(), q)


@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 128), (16, 2048), (3, 130), (127, 129), (128, 128), (130, 257), (257, 4)])
@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("x_dtype,dtype", [(torch.float32, E4M3), (torch.bfloat16, E4M3), (torch.float16, E5M2)])
def test_quantise_equals_the_definition(rows, cols, block_rows, x_dtype, dtype):
    x = randn(rows, cols, seed=rows * 1000 + cols)
    x *= torch.exp2(torch.randint(-14, 4, (rows, cols), generator=torch.Generator().manual_seed(1)).float())
    x = x.to(x_dtype)
    q, s, qt, st = lib.fp8_quantise(x.to(DEV), block_rows, dtype, layout="both")
    finished()
    check_codes(q, s, x.float(), block_rows, dtype)
    check_codes(qt, st, x.float().t(), block_rows, dtype)


@pytest.mark.parametrize("layout", ["rows", "cols"])
@pytest.mark.parametrize("dtype", [E4M3, E5M2])
def test_quantise_one_layout_and_a_difference(layout, dtype):
    x, m = randn(150, 200, seed=3), randn(150, 200, seed=4)
    q, s = lib.fp8_quantise(x.to(DEV), 1, dtype, minus=m.to(DEV), layout=layout)
    finished()
    v = x - m
    check_codes(q, s, v if layout == "rows" else v.t(), 1, dtype)


def test_quantise_extreme_blocks():
    """Zeros, subnormals, the largest values, exact borders of the scale, ties of the
    rounding, and values that are not finite, which spoil their own block only."""
    x = torch.zeros(12, 256)
    x[1] = 1e-45
    x[2] = torch.finfo(torch.float32).max
    x[3, 0] = 448.0                                   # scale 1 exactly
    x[4, 0] = float(np.nextafter(np.float32(448.0), np.float32(1e9)))
    x[5, 0] = 0.875 * 2.0 ** -120
    x[6, :4] = torch.tensor([448.0, 17.0, 19.0, -0.0009765625])     # ties to even; half of the least subnormal
    x[7, 5] = math.inf
    x[8, 200] = math.nan
    x[9] = -2.0 ** -149
    x[10, 0], x[10, 1] = 2.0 ** -118, 2.0 ** -149
    x[11, 130] = -math.inf
    q, s, qt, st = lib.fp8_quantise(x.to(DEV), 1, E4M3, layout="both")
    finished()
    check_codes(q, s, x, 1, E4M3)
    check_codes(qt, st, x.t(), 1, E4M3)
    q, s = lib.fp8_quantise(x.to(DEV), 128, E4M3)
    finished()
    check_codes(q, s, x, 128, E4M3)


@pytest.mark.parametrize("rows,cols,x_dtype,minus", [(3200, 3205, torch.float32, True), (1000, 9996, torch.bfloat16, False),
                                                     (9999, 1002, torch.float32, False), (2500, 4000, torch.bfloat16, True)])
def test_quantise_many_tiles(rows, cols, x_dtype, minus):
    """Matrices of many tiles take a path of their own; it has to give the codes that
    their parts give, with row starts on 16-byte boundaries and off them."""
    g = torch.Generator(device=DEV).manual_seed(7)
    room = torch.randn(rows, cols + 15, generator=g, device=DEV).to(x_dtype)
    room = torch.nn.functional.pad(room, (0, -room.shape[1] % 8))
    m = torch.randn(rows, cols, generator=g, device=DEV) if minus else None
    for at in (0, 3, 8):
        x = room[:, at:at + cols]
        whole = lib.fp8_quantise(x, 1, E4M3, minus=m, layout="both")
        blocks = lib.fp8_quantise(x, 128, E4M3, minus=m, layout="both")
        for r in range(0, rows, 1280):                       # 128-row borders
            sub, msub = x[r:r + 1280, :512], None if m is None else m[r:r + 1280, :512]
            q, s, qt, st = lib.fp8_quantise(sub, 1, E4M3, minus=msub, layout="both")
            assert torch.equal(q.view(torch.uint8), whole[0][r:r + 1280, :512].view(torch.uint8))
            assert torch.equal(s.view(torch.uint8), whole[1][r:r + 1280, :4].view(torch.uint8))
            assert torch.equal(qt.view(torch.uint8), whole[2][:512, r:r + 1280].view(torch.uint8))
            assert torch.equal(st.view(torch.uint8), whole[3][:512, r // 128:(r + 1280) // 128].view(torch.uint8))
            q, s, qt, st = lib.fp8_quantise(sub, 128, E4M3, minus=msub, layout="both")
            assert torch.equal(q.view(torch.uint8), blocks[0][r:r + 1280, :512].view(torch.uint8))
            assert torch.equal(qt.view(torch.uint8), blocks[2][:512, r:r + 1280].view(torch.uint8))
            assert torch.equal(s.view(torch.uint8), blocks[1][r // 128:r // 128 + 10, :4].view(torch.uint8))
        finished()
        # the ragged corner against the definition
        r, c = rows // 128 * 128, cols // 128 * 128
        v = (x[r:, c:].float() if m is None else x[r:, c:].float() - m[r:, c:]).cpu()
        check_codes(whole[0][r:, c:], whole[1][r:, c // 128:], v, 1, E4M3)
        check_codes(whole[2][c:, r:], whole[3][c:, r // 128:], v.t(), 1, E4M3)
        check_codes(blocks[0][r:, c:], blocks[1][r // 128:, c // 128:], v, 128, E4M3)


def test_quantise_strided_and_unaligned_inputs():
    room = randn(140, 300, seed=5).to(DEV)
    for view in (room[:, 1:270], room[3:, 4:204], room.to(torch.bfloat16)[1::2, 3:132]):
        q, s, qt, st = lib.fp8_quantise(view, 1, E4M3, layout="both")
        finished()
        check_codes(q, s, view.float().cpu(), 1, E4M3)
        check_codes(qt, st, view.float().cpu().t(), 1, E4M3)


def test_quantise_leaves_what_lies_behind_the_rows():
    x = randn(5, 130, seed=6).to(DEV)
    q = torch.full((9, 160), 77, dtype=torch.uint8, device=DEV)
    s = torch.full((9, 8), 77, dtype=torch.uint8, device=DEV)
    rc = lib.load().bcjr_fp8_quantise(lib._ptr(x), 0, 5, 130, 130, None, 0, 3, 1, lib._ptr(q), 160, lib._ptr(s), 8,
                                      None, 0, None, 0, lib._stream(None))
    assert rc == 0
    finished()
    assert (q[5:] == 77).all() and (q[:, 130:] == 77).all() and (s[5:] == 77).all() and (s[:, 2:] == 77).all()
    check_codes(q[:5, :130].view(E4M3), s[:5, :2].view(torch.float8_e8m0fnu), x.cpu(), 1, E4M3)


# ---------------------------------------------------------------- the 8-bit product

def operand(rows, k, block_rows, dtype, seed):
    x = randn(rows, k, seed=seed)
    x *= torch.exp2(torch.randint(-3, 4, (rows, 1), generator=torch.Generator().manual_seed(seed)).float())
    x *= torch.exp2(torch.randint(-3, 4, (1, -(-k // 128)), generator=torch.Generator().manual_seed(seed + 1)).float()).repeat_interleave(128, 1)[:, :k]
    return lib.fp8_quantise(x.to(DEV), block_rows, dtype)


def check_product(y, a, sa, ra, b, sb, rb, alpha):
    """Products of 8-bit values are exact in fp32.  One instruction adds 32 of them to
    the sum, so no term passes more than K / 32 + 32 additions, each off by at most a
    whole step (2^-23, should the adder truncate) of sums no larger than the sum of
    absolute values; splitting k adds at most 8 more.  Then alpha (a power of two) and
    one rounding to the output's type."""
    va, vb = ref.values(a, sa, ra), ref.values(b, sb, rb)
    want = alpha * va @ vb.t()
    size = abs(alpha) * va.abs() @ vb.abs().t()
    tol = (va.shape[1] / 32 + 40) * 2.0 ** -23 * size + HALF_STEP[y.dtype] * want.abs() + torch.finfo(y.dtype).tiny
    err = (y.cpu().double() - want).abs()
    assert bool((err <= tol).all()), f"worst {float((err / tol).max()):.3g} of the tolerance"
    return want


@pytest.mark.parametrize("m,n,k", [(1, 16, 16), (1, 512, 2048), (3, 130, 129), (17, 128, 128), (37, 512, 2000), (64, 64, 640),
                                   (65, 257, 1000), (130, 384, 4096), (200, 1000, 72), (300, 5, 256), (1, 1, 1), (513, 300, 515)])
@pytest.mark.parametrize("ra,rb", [(1, 128), (128, 1)])
def test_matmul(m, n, k, ra, rb):
    a, sa = operand(m, k, ra, E4M3, 11)
    b, sb = operand(n, k, rb, E4M3, 12)
    y = lib.fp8_matmul(a, sa, b, sb, out_dtype=torch.float32)
    finished()
    check_product(y, a, sa, ra, b, sb, rb, 1.0)


@pytest.mark.parametrize("da", [E4M3, E5M2])
@pytest.mark.parametrize("db", [E4M3, E5M2])
@pytest.mark.parametrize("out_dtype", [torch.float32, torch.float16, torch.bfloat16])
def test_matmul_types(da, db, out_dtype):
    a, sa = operand(70, 300, 1, da, 13)
    b, sb = operand(140, 300, 128, db, 14)
    y = lib.fp8_matmul(a, sa, b, sb, alpha=0.25, out_dtype=out_dtype)
    finished()
    check_product(y, a, sa, 1, b, sb, 128, 0.25)


@pytest.mark.parametrize("m,n,k", [(2048, 2048, 1024), (1111, 4096, 896), (4096, 640, 2048)])
def test_matmul_large(m, n, k):
    a, sa = operand(m, k, 1, E4M3, 15)
    b, sb = operand(n, k, 128, E4M3, 16)
    y = lib.fp8_matmul(a, sa, b, sb, out_dtype=torch.float32)
    finished()
    check_product(y, a, sa, 1, b, sb, 128, 1.0)


def test_matmul_padding_is_not_read():
    """Codes and scales behind the rows hold NaN; rows of the output behind N stay."""
    m, n, k = 20, 150, 200
    x, w = randn(m, k, seed=17), randn(n, k, seed=18)
    ops = []
    for v in (x, w):
        room = torch.full((v.shape[0] + 3, 256), 0x7F, dtype=torch.uint8, device=DEV)
        srow = torch.full((v.shape[0] + 3, 7), 0xFF, dtype=torch.uint8, device=DEV)
        q, s = lib.fp8_quantise(v.to(DEV), 1, E4M3)
        room[: v.shape[0], :k] = q.view(torch.uint8)
        srow[: v.shape[0], :2] = s.view(torch.uint8)
        ops += [room.view(E4M3)[: v.shape[0], :k], srow.view(torch.float8_e8m0fnu)[: v.shape[0], :2]]
    room = torch.full((m + 2, n + 9), 7.0, device=DEV)
    y = lib.fp8_matmul(*ops, out=room[:m, 3:3 + n])
    finished()
    check_product(y, ops[0], ops[1], 1, ops[2], ops[3], 1, 1.0)
    assert (room[m:] == 7).all() and (room[:, :3] == 7).all() and (room[:, 3 + n:] == 7).all()


@pytest.mark.parametrize("up,down", [(100, -100), (-110, 110), (60, 10)])
@pytest.mark.parametrize("m,n", [(20, 150), (2048, 2400)])
def test_matmul_scales_of_any_size(up, down, m, n):
    """Scales far from one another: powers of two on the operands are the same powers on
    the result."""
    x, w = randn(m, 300, seed=36).to(DEV), randn(n, 300, seed=37).to(DEV)
    plain = lib.fp8_matmul(*lib.fp8_quantise(x), *lib.fp8_quantise(w, 128), out_dtype=torch.float32)
    far = lib.fp8_matmul(*lib.fp8_quantise(x * 2.0 ** up), *lib.fp8_quantise(w * 2.0 ** down, 128), out_dtype=torch.float32)
    finished()
    assert torch.equal(far, plain * 2.0 ** (up + down))


def test_matmul_not_finite_values_stay_in_their_rows():
    x, w = randn(40, 300, seed=19), randn(140, 300, seed=20)
    x[5, 3] = math.nan
    w[7, 290] = math.inf
    a, sa = lib.fp8_quantise(x.to(DEV))
    b, sb = lib.fp8_quantise(w.to(DEV))
    y = lib.fp8_matmul(a, sa, b, sb, out_dtype=torch.float32)
    finished()
    bad = torch.isnan(y.cpu())
    want = torch.zeros_like(bad)
    want[5] = True
    want[:, 7] = True
    assert torch.equal(bad, want)


def test_matmul_empty():
    a, sa = lib.fp8_quantise(torch.zeros(4, 0, device=DEV))
    b, sb = lib.fp8_quantise(torch.zeros(6, 0, device=DEV))
    assert torch.equal(lib.fp8_matmul(a, sa, b, sb), torch.zeros(4, 6, dtype=torch.bfloat16, device=DEV))
    a, sa = lib.fp8_quantise(torch.zeros(0, 32, device=DEV))
    b, sb = lib.fp8_quantise(torch.zeros(6, 32, device=DEV))
    assert lib.fp8_matmul(a, sa, b, sb).shape == (0, 6)
    finished()


# ---------------------------------------------------------------- Newton-Schulz

def check_orthogonal(out, g, steps=5, coeffs=None, noise=15.0):
    """2-norm of the difference against that of the result.  Each step rounds X, A and
    B to fp16: three relative errors of at most 2^-11 a step, `noise` of them in all,
    and they may grow twice as fast as the matrix itself where its singular values
    lie within a factor of a few of one another (the polynomial's slope there against
    its mean slope); then one rounding to the output's type."""
    want = ref.newton_schulz(g, steps, coeffs).cpu()
    tol = 2 * noise * 2.0 ** -11 + HALF_STEP[out.dtype]
    err = out.cpu().double() - want
    rel = torch.linalg.vector_norm(err, dim=(-2, -1)) / torch.linalg.vector_norm(want, dim=(-2, -1))
    assert float(rel.max()) <= tol, f"relative error {float(rel.max()):.3g} > {tol:.3g}"


@pytest.mark.parametrize("rows,cols", [(16, 48), (64, 128), (128, 512), (130, 333), (333, 130), (1, 40), (40, 1), (1, 1), (8, 1000),
                                       (512, 100), (257, 1025), (300, 130)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_orthogonalise(rows, cols, dtype):
    g = randn(rows, cols, seed=rows + cols, scale=1e-3).to(dtype)
    out = lib.orthogonalise(g.to(DEV))
    finished()
    check_orthogonal(out, g)


@pytest.mark.parametrize("rows,cols", [(512, 1536), (1536, 512), (700, 2100), (1300, 2700), (2700, 1300)])
def test_orthogonalise_large(rows, cols):
    g = randn(rows, cols, seed=21)
    out = lib.orthogonalise(g.to(DEV))
    finished()
    check_orthogonal(out, g)


@pytest.mark.parametrize("rows,cols", [(1536, 6145), (6200, 1500)])
@pytest.mark.parametrize("steps,coeffs", [(1, None), (2, None), (3, None), (4, None), (5, None), (2, (1.875, -1.25, 0.375)),
                                          (2, [(6.5, -17.0, 12.0), (2.5, -2.2, 0.6)])])
def test_orthogonalise_long_matrices(rows, cols, steps, coeffs):
    """Long enough that steps are taken two at a time (but for the last case, whose
    polynomials' product would leave fp16's headroom).  A pair rounds X once and P, B, P
    again, B and two products between them: five relative errors of 2^-11 more than the
    six of two single steps."""
    g = randn(rows, cols, seed=25).to(DEV)
    co = None if coeffs is None else [coeffs] * steps if isinstance(coeffs, tuple) else coeffs
    out = lib.orthogonalise(g, steps=steps, coeffs=coeffs)
    finished()
    check_orthogonal(out, g, steps, co, noise=3.0 * steps + 5.0 * (steps // 2))


@pytest.mark.parametrize("rows,cols", [(1, 40), (30, 30), (130, 333), (333, 130), (512, 700), (1300, 1400), (1500, 1300)])
def test_orthogonalise_two_planes(rows, cols):
    """An fp16 result: operands of 22 bits.  Three roundings a step of at most 2^-22, and
    sums of n terms in fp32 of at most (n / 16 + 16) whole steps of sums of absolute
    values, which the norms bound by sqrt(n) times the result; the smallest singular
    values of a square matrix grow 485 times while the norm grows sqrt(rank), so errors
    grow at most 485 / sqrt(rank) times against the result."""
    g = randn(rows, cols, seed=rows + 2 * cols)
    out = lib.orthogonalise(g.to(DEV), out_dtype=torch.float16)
    finished()
    want = ref.newton_schulz(g)
    rel = float(torch.linalg.vector_norm(out.cpu().double() - want) / torch.linalg.vector_norm(want))
    n = max(rows, cols)
    assert rel <= 485 / math.sqrt(min(rows, cols)) * (15 * 2.0 ** -22 + 15 * (n / 16 + 16) * 2.0 ** -23) + HALF_STEP[torch.float16]
    # and, since those are worst cases: closer than operands of 11 bits could come (3e-4 or more)
    assert rel <= 2.5e-4


@pytest.mark.parametrize("rows,cols", [(16, 100), (16, 16), (40, 40), (3652, 16), (64, 300), (33, 5000), (160, 6788), (5632, 165)])
def test_orthogonalise_roundings_do_not_add_up(rows, cols):
    """Of thin and long matrices the diagonals of P and B are nearly constant, so that plain
    roundings to 11 bits (2^-12 on average, fifteen of them) would all go one way: up to
    15 * 2^-12 = 3.7e-3.  Independent ones add up to sqrt(15) * 2^-12 / sqrt(3) * 2 =
    1.1e-3 (twice for the growth of small singular values), and with the result's own
    rounding, at most 2^-8 / sqrt(3) = 2.3e-3 in the 2-norm, to 2.5e-3."""
    g = randn(rows, cols, seed=27) + randn(rows, 4, seed=28) @ randn(4, cols, seed=29)
    out = lib.orthogonalise(g.to(DEV))
    finished()
    want = ref.newton_schulz(g)
    rel = float(torch.linalg.vector_norm(out.cpu().double() - want) / torch.linalg.vector_norm(want))
    assert rel <= 2.5e-3


@pytest.mark.parametrize("batch,rows,cols", [(64, 128, 128), (200, 128, 250), (40, 130, 900), (40, 700, 100), (300, 32, 96),
                                             (500, 17, 9), (1000, 1, 3), (37, 129, 129)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_orthogonalise_many_small_matrices(batch, rows, cols, dtype):
    """Batches large enough for every kernel that the tile rule knows, on both sides of 128 rows."""
    g = randn(batch, rows, cols, seed=31).to(dtype)
    out = lib.orthogonalise(g.to(DEV))
    finished()
    check_orthogonal(out, g)


def test_orthogonalise_batch_strides_and_zeros():
    g = randn(5, 60, 200, seed=22).to(DEV)
    g[2] = 0
    view = g[:, ::2, 7:150]
    out = lib.orthogonalise(view)
    finished()
    check_orthogonal(out[[0, 1, 3, 4]], view[[0, 1, 3, 4]].cpu())
    assert (out[2] == 0).all()


def test_orthogonalise_not_finite_matrix_stays_alone():
    g = randn(3, 40, 90, seed=23).to(DEV)
    g[1, 3, 4] = math.nan
    out = lib.orthogonalise(g)
    finished()
    check_orthogonal(out[[0, 2]], g[[0, 2]].cpu())
    assert torch.isnan(out[1]).all()


@pytest.mark.parametrize("exponent", [-130, -60, 60, 110])
def test_orthogonalise_does_not_depend_on_scale(exponent):
    """A power of two on the matrix moves neither the norm's rounding nor any other while
    its entries stay normal numbers; with eps = 0 the result is the same bits."""
    g = randn(70, 200, seed=26).to(torch.bfloat16).float()
    if exponent == -130:
        g = torch.where(g.abs() < 2.0 ** -4, torch.zeros(()), g.sign() * torch.exp2(g.abs().log2().floor()))   # powers of two: exact below 2^-126 too
    one = lib.orthogonalise(g.to(DEV), eps=0.0)
    out = lib.orthogonalise((g.double() * 2.0 ** exponent).float().to(DEV), eps=0.0)
    finished()
    assert torch.equal(out, one)
    check_orthogonal(one, g)


@pytest.mark.parametrize("rows,cols", [(70, 200), (201, 70), (130, 333), (13, 13), (517, 600), (1537, 6145)])
@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float16])
def test_orthogonalise_after_not_finite_values(rows, cols, out_dtype):
    """What an earlier call left in the scratch memory (NaN here) does not matter."""
    g = randn(rows, cols, seed=30).to(DEV)
    want = lib.orthogonalise(g, out_dtype=out_dtype)
    for bad in (math.nan, math.inf):
        spoilt = lib.orthogonalise(torch.full_like(g, bad), out_dtype=out_dtype)
        assert torch.isnan(spoilt).all()
        assert torch.equal(lib.orthogonalise(g, out_dtype=out_dtype), want)
    finished()


def test_orthogonalise_coefficients_of_each_step():
    g = randn(50, 140, seed=24)
    coeffs = [(3.0, -3.2, 1.2), (2.0, -1.5, 0.5), (1.875, -1.25, 0.375)]
    out = lib.orthogonalise(g.to(DEV), steps=3, coeffs=coeffs)
    finished()
    check_orthogonal(out, g, 3, coeffs)
    one = lib.orthogonalise(g.to(DEV), steps=2, coeffs=(1.875, -1.25, 0.375))
    finished()
    check_orthogonal(one, g, 2, [(1.875, -1.25, 0.375)] * 2)


# ---------------------------------------------------------------- Muon

@pytest.mark.parametrize("rows,cols", [(64, 200), (300, 130), (1, 50), (128, 128 * 3)])
@pytest.mark.parametrize("nesterov", [True, False])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_muon_step(rows, cols, nesterov, dtype):
    w, m = randn(rows, cols, seed=31), randn(rows, cols, seed=32, scale=1e-3)
    g = randn(rows, cols, seed=33, scale=1e-3).to(dtype)
    lr, mu, decay = 0.05, 0.9, 0.1
    wd, md = w.to(DEV), m.to(DEV)
    out = lib.muon_step(wd, g.to(DEV), md, lr, mu=mu, nesterov=nesterov, weight_decay=decay)
    finished()
    assert out[0] is wd and out[1] is md
    g64, m64 = g.double(), m.double()
    m_ref = mu * m64 + g64
    # mu is rounded to fp32 (2^-24 of it), then one fused multiply-add
    assert bool(((md.cpu().double() - m_ref).abs() <= 2.0 ** -23 * ((mu * m64).abs() + m_ref.abs())).all())
    u = g64 + mu * m_ref if nesterov else m_ref
    o = ref.newton_schulz(u)
    scale = math.sqrt(max(1.0, rows / cols))
    w_ref = (1 - lr * decay) * w.double() - lr * scale * o
    # the orthogonalised part as above (30 half steps of fp16 in the 2-norm); w in fp32: the
    # factor's rounding, the product, the sum
    err = torch.linalg.vector_norm(wd.cpu().double() - w_ref)
    tol = lr * scale * 30 * 2.0 ** -11 * torch.linalg.vector_norm(o) + 4 * 2.0 ** -24 * torch.linalg.vector_norm(w_ref)
    assert float(err) <= float(tol)


def test_muon_step_on_views():
    room = randn(100, 300, seed=34).to(DEV)
    w = room[10:90, 5:205]
    before = room.clone()
    g, m = randn(80, 200, seed=35).to(DEV), torch.zeros(80, 320, device=DEV)[:, :200]
    lib.muon_step(w, g, m, 0.1, scale=1.0)
    finished()
    assert torch.equal(m, g)
    keep = torch.ones_like(room, dtype=torch.bool)
    keep[10:90, 5:205] = False
    assert torch.equal(room[keep], before[keep])
    o = ref.newton_schulz(g.cpu().double() * 1.95)
    err = torch.linalg.vector_norm((before[10:90, 5:205] - w).cpu().double() - 0.1 * o)
    assert float(err) <= 0.1 * 30 * 2.0 ** -11 * float(torch.linalg.vector_norm(o)) + 2.0 ** -22 * float(torch.linalg.vector_norm(w))
