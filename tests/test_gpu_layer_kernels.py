"""Every kernel of the layer-wise QAT operators on values, over several blocks of k, several
tiles and ragged ends, with the kernel that each case takes read from the profiler: a
change of the rules that choose them does not silently leave one untested."""
import pytest
import torch

import layer_reference as ref
from bcjr_sum_product_b200 import lib
from test_gpu_layer_accuracy import bound, rounded

pytestmark = pytest.mark.gpu
DEV = "cuda"
E4M3, E5M2 = torch.float8_e4m3fn, torch.float8_e5m2
F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
HALF_STEP = {F32: 2.0 ** -24, F16: 2.0 ** -11, BF16: 2.0 ** -8}
OUT, GRAM, POLY, ITER, LAST, STEP = range(6)


def randn(*shape, seed=0):
    return torch.randn(*shape, generator=torch.Generator(device=DEV).manual_seed(seed), device=DEV)


def finished():
    torch.cuda.synchronize()
    assert lib.get_device_error() == 0


def launched(call):
    """call's result and the names of the kernels that it launched ("pair_kernel<1, 256, false, false, 0>")."""
    with torch.profiler.profile(activities=[torch.profiler.ProfilerActivity.CUDA]) as prof:
        out = call()
        torch.cuda.synchronize()
    names = {e.key.split("gemm::", 1)[1].split("(")[0] for e in prof.key_averages() if "gemm::" in e.key}
    assert names, "no kernel was recorded"
    return out, names


def kernel(name, kind, width, r_mn, c_mn, end):
    return f"{name}_kernel<{kind}, {width}, {str(r_mn).lower()}, {str(c_mn).lower()}, {end}>"


# ---------------------------------------------------------------- 8-bit products

def operand(rows, k, block_rows, dtype, seed):
    x = randn(rows, k, seed=seed)
    x *= torch.exp2(torch.randint(-3, 4, (rows, 1), generator=torch.Generator().manual_seed(seed)).float()).to(DEV)
    x *= torch.exp2(torch.randint(-3, 4, (1, -(-k // 128)), generator=torch.Generator().manual_seed(seed + 1)).float()).to(DEV).repeat_interleave(128, 1)[:, :k]
    return lib.fp8_quantise(x, block_rows, dtype)


def check_product(y, a, sa, ra, b, sb, rb, alpha):
    """Entry by entry: no term passes more than K / 32 + 40 additions, each off by at most a whole step of a sum no
    larger than that of the absolute values; then the rounding of the result."""
    va, vb = ref.values(a, sa, ra).to(DEV), ref.values(b, sb, rb).to(DEV)
    want = alpha * (va @ vb.t())
    size = abs(alpha) * (va.abs() @ vb.abs().t())
    tol = (va.shape[1] / 32 + 40) * 2.0 ** -23 * size + HALF_STEP[y.dtype] * want.abs() + torch.finfo(y.dtype).tiny
    err = (y.double() - want).abs()
    assert bool((err <= tol).all()), f"worst {float((err / tol).max()):.3g} of the tolerance"


PRODUCTS = [  # m, n, k, kernel, its tile's width
    (9, 1000, 4100, "tile", 16), (30, 600, 3000, "tile", 32), (60, 2000, 1111, "tile", 64), (400, 400, 5000, "tile", 64),
    (512, 2048, 8192, "tile", 128), (1500, 1600, 700, "tile", 128),
    (700, 1111, 1500, "pair", 128), (513, 2000, 777, "pair", 128), (1900, 2048, 8161, "pair", 224), (3000, 5000, 1030, "pair", 224),
    (2048, 2048, 8192, "pair", 256), (2047, 1999, 6001, "pair", 256)]


@pytest.mark.parametrize("m,n,k,name,width", PRODUCTS)
@pytest.mark.parametrize("ra,rb,da,db,out_dtype,alpha", [(1, 1, E5M2, E4M3, F32, 2.0), (1, 128, E4M3, E4M3, BF16, 1.0),
                                                         (128, 128, E4M3, E5M2, F16, 2.0 ** -6), (128, 1, E5M2, E5M2, F32, 1.0)])
def test_products_on_each_kernel(m, n, k, name, width, ra, rb, da, db, out_dtype, alpha):
    """Several groups of scales (512 values of k each) and rounds of the stages, types of either side, one scale for a
    row or for 128 rows of either side."""
    a, sa = operand(m, k, ra, da, 11)
    b, sb = operand(n, k, rb, db, 13)
    y, names = launched(lambda: lib.fp8_matmul(a, sa, b, sb, alpha=alpha, out_dtype=out_dtype))
    finished()
    assert names == {kernel(name, 1, width, False, False, OUT)}
    check_product(y, a, sa, ra, b, sb, rb, alpha)


def test_products_in_bands():
    """An operand of more than 48 MB is taken in bands of 16 tiles: two whole ones and a ragged one."""
    m, n, k = 1024, 8322, 8176
    a, sa = operand(m, k, 1, E4M3, 15)
    b, sb = operand(n, k, 128, E4M3, 17)
    y, names = launched(lambda: lib.fp8_matmul(a, sa, b, sb, out_dtype=BF16))
    finished()
    assert names == {kernel("pair", 1, 256, False, False, OUT)}
    check_product(y, a, sa, 1, b, sb, 128, 1.0)


# ---------------------------------------------------------------- Newton-Schulz

def relative(got, want):
    return float(torch.linalg.vector_norm(got.double() - want) / torch.linalg.vector_norm(want))


def muon_case(rows, cols, nesterov, dtype, offset, expect, strong=0):
    """w, momentum and gradient in rows of odd or even strides, against 64 bits; the ragged last rows and columns by
    themselves too (their errors are random shares of the whole's: three times its bound)."""
    def room(seed):
        return randn(rows, cols + 5 if offset else -(-cols // 8) * 8, seed=seed)[:, offset:offset + cols]
    w, m = room(81), room(82) * 1e-3
    if offset:
        m = torch.cat([m, m[:, :5]], 1)[:, :cols]
    g = randn(rows, cols, seed=83) * 1e-3
    if strong:
        g += 1e-2 * randn(rows, strong, seed=84) @ randn(strong, cols, seed=85)
    g = g.to(dtype)
    lr, mu, decay = 0.05, 0.9, 0.1
    g64, m64, w64 = g.double(), m.double(), w.double()
    _, names = launched(lambda: lib.muon_step(w, g, m, lr, mu=mu, nesterov=nesterov, weight_decay=decay, scale=1.0))
    finished()
    assert expect <= names, names
    m_ref = mu * m64 + g64
    assert bool(((m.double() - m_ref).abs() <= 2.0 ** -23 * ((mu * m64).abs() + m_ref.abs())).all())
    o = ref.newton_schulz(g64 + mu * m_ref if nesterov else m_ref)
    tol = bound(5, True)
    got = ((1 - lr * decay) * w64 - w.double()) / lr
    # w's own roundings: the factor, the product and the sum, 2^-24 of an entry each, over lr
    tiny = 3 * 2.0 ** -24 / lr * float(torch.linalg.vector_norm(w64) / torch.linalg.vector_norm(o))
    assert relative(got, o) <= tol + tiny
    for part in (slice(-(rows % 128 or 128), None), slice(None)), (slice(None), slice(-(cols % 128 or 128), None)):
        assert relative(got[part], o[part]) <= 3 * (tol + tiny)


PAIR_STEP = {False: kernel("pair", 0, 256, True, False, STEP), True: kernel("pair", 0, 256, False, False, STEP)}   # by rows > cols


@pytest.mark.parametrize("rows,cols", [(1300, 2700), (2700, 1300), (1537, 6145), (6200, 1500), (2048, 2048)])
@pytest.mark.parametrize("nesterov,dtype,offset", [(True, F32, 0), (False, BF16, 3), (True, F16, 0)])
def test_muon_steps_on_pairs(rows, cols, nesterov, dtype, offset):
    """The sizes of whole layers: pairs of SMs for every product, the first two steps at once where one side is long."""
    gram = kernel("pair", 0, 128, rows > cols, rows > cols, GRAM)
    muon_case(rows, cols, nesterov, dtype, offset, {gram, kernel("pair", 0, 128, False, False, POLY), PAIR_STEP[rows > cols],
                                                    kernel("pair", 0, 256, rows <= cols, False, ITER)}, strong=4)


@pytest.mark.parametrize("rows,cols,expect", [
    (20000, 100, kernel("tile", 0, 128, False, False, STEP)), (700, 300, kernel("tile", 0, 64, False, False, STEP)),
    (300, 700, kernel("tile", 0, 64, True, False, STEP)), (100, 6000, kernel("tile", 0, 64, True, False, STEP))])
@pytest.mark.parametrize("dtype", [F32, F16])
def test_muon_steps_on_single_blocks(rows, cols, expect, dtype):
    muon_case(rows, cols, True, dtype, 0, {expect})


def test_two_steps_at_once_or_one():
    """A long matrix takes five products with X fewer one (and three more of its shorter side)."""
    for rows, cols, products in ((1536, 6145, 4), (1536, 1700, 5)):
        g = randn(rows, cols, seed=86)
        with torch.profiler.profile(activities=[torch.profiler.ProfilerActivity.CUDA]) as prof:
            lib.orthogonalise(g)
            torch.cuda.synchronize()
        count = {e.key.split("gemm::", 1)[1].split("(")[0]: e.count for e in prof.key_averages() if "gemm::" in e.key}
        ends = {end: sum(n for name, n in count.items() if name.endswith(f" {end}>")) for end in (GRAM, POLY, ITER, LAST)}
        assert ends[ITER] + ends[LAST] == products and ends[POLY] == 5 and ends[GRAM] == products + (3 if products == 4 else 0)


@pytest.mark.parametrize("batch,rows,cols,widths", [
    (200, 128, 128, {(GRAM, 128, False), (POLY, 128, False), (ITER, 128, True), (LAST, 128, True)}),
    (200, 250, 128, {(GRAM, 128, True), (POLY, 128, False)}), (300, 96, 40, {(GRAM, 128, True), (POLY, 128, False), (ITER, 128, False)})])
@pytest.mark.parametrize("out_dtype", [BF16, F16])
def test_batches_on_wide_single_blocks(batch, rows, cols, widths, out_dtype):
    g = randn(batch, rows, cols, seed=87)
    out, names = launched(lambda: lib.orthogonalise(g, out_dtype=out_dtype))
    finished()
    for end, width, r_mn in widths:
        assert kernel("tile", 0, width, r_mn, end == GRAM and r_mn, end) in names, names
    assert relative(out, ref.newton_schulz(g)) <= rounded(bound(5, False), out_dtype)


@pytest.mark.parametrize("out_dtype", [BF16, F16])
def test_orthogonalise_in_bands(out_dtype):
    """X of 67 MB as the operand along r: two bands."""
    g = randn(4096, 8192, seed=88).to(BF16)
    out, names = launched(lambda: lib.orthogonalise(g, out_dtype=out_dtype))
    finished()
    assert kernel("pair", 0, 256, True, False, ITER) in names
    assert relative(out, ref.newton_schulz(g)) <= rounded(bound(5, True), out_dtype)
