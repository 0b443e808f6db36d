"""Refusals and host logic of the layer-wise QAT operators (no GPU): the C ABI on
null and host pointers, the binding's checks, the driver's arguments."""
import ctypes

import pytest
import torch

from bcjr_sum_product_b200 import lib, qat

INVALID, UNSUPPORTED, OK = lib.BCJR_ERR_INVALID_ARG, lib.BCJR_ERR_UNSUPPORTED, lib.BCJR_OK


def quantise(x=None, x_type=0, rows=4, cols=130, ld_x=130, minus=None, ld_minus=0, q_type=3, block_rows=1, q=None,
             ld_q=144, scale=None, ld_scale=2, qt=None, ld_qt=16, scale_t=None, ld_scale_t=1):
    return lib.load().bcjr_fp8_quantise(x, x_type, rows, cols, ld_x, minus, ld_minus, q_type, block_rows, q, ld_q, scale,
                                        ld_scale, qt, ld_qt, scale_t, ld_scale_t, None)


def test_quantise_refusals():
    room = torch.zeros(1 << 14)
    p = ctypes.c_void_p((room.data_ptr() + 15) // 16 * 16)        # a host pointer: refused, but after the sizes
    both = dict(x=p, q=p, scale=p, qt=p, scale_t=p)
    n0 = lib.launch_count()
    for bad in (dict(rows=-1), dict(cols=-1), dict(x_type=3), dict(x_type=9), dict(q_type=0), dict(q_type=5), dict(block_rows=2),
                dict(block_rows=0), dict(q=None), dict(scale=None), dict(scale_t=None), dict(ld_x=129), dict(minus=p, ld_minus=129),
                dict(ld_q=130), dict(ld_q=128), dict(ld_scale=1), dict(ld_qt=0), dict(ld_qt=20), dict(ld_scale_t=0)):
        assert quantise(**{**both, **bad}) == INVALID, bad
    assert quantise(x=p) == INVALID                               # nothing to write
    assert quantise(**both) == INVALID                            # host memory
    assert quantise(**{**both, "x": None}) == INVALID
    assert quantise(rows=(1 << 30) + 1) == UNSUPPORTED
    assert quantise(rows=0) == OK and quantise(cols=0) == OK
    assert lib.launch_count() == n0


def matmul(a=None, a_type=3, ld_a=256, sa=None, ld_sa=2, a_rows=1, b=None, b_type=3, ld_b=256, sb=None, ld_sb=2, b_rows=128,
           M=4, N=8, K=256, alpha=1.0, out=None, out_type=2, ld_out=8):
    return lib.load().bcjr_fp8_matmul(a, a_type, ld_a, sa, ld_sa, a_rows, b, b_type, ld_b, sb, ld_sb, b_rows, M, N, K, alpha,
                                      out, out_type, ld_out, None)


def test_matmul_refusals():
    n0 = lib.launch_count()
    for bad in (dict(M=-1), dict(N=-1), dict(K=-1), dict(a_type=0), dict(b_type=2), dict(out_type=3), dict(out_type=7), dict(a_rows=64),
                dict(b_rows=0), dict(alpha=float("nan")), dict(alpha=float("inf")), dict(ld_out=7), dict()):
        assert matmul(**bad) == INVALID, bad                      # the last: null pointers
    assert matmul(M=(1 << 30) + 1) == UNSUPPORTED and matmul(K=(1 << 30) + 1) == UNSUPPORTED
    assert matmul(M=0) == OK and matmul(N=0) == OK
    room = torch.zeros(1 << 12)
    p = ctypes.c_void_p((room.data_ptr() + 15) // 16 * 16)
    assert matmul(a=p, sa=p, b=p, sb=p, out=p) == INVALID         # host memory
    assert lib.launch_count() == n0


def orthogonalise(g=None, g_type=0, batch=1, rows=4, cols=8, ld=8, stride=32, steps=5, coeffs=None, eps=1e-7, out=None,
                  out_type=2, ld_out=8, stride_out=32):
    co = None if coeffs is None else (ctypes.c_float * len(coeffs))(*coeffs)
    return lib.load().bcjr_orthogonalise(g, g_type, batch, rows, cols, ld, stride, steps, co, eps, out, out_type, ld_out,
                                         stride_out, None)


def muon(w=None, ld_w=8, g=None, g_type=0, ld_g=8, m=None, ld_m=8, rows=4, cols=8, lr=0.1, mu=0.9, decay=0.0, scale=1.0,
         steps=5, coeffs=None, eps=1e-7):
    co = None if coeffs is None else (ctypes.c_float * len(coeffs))(*coeffs)
    return lib.load().bcjr_muon_step(w, ld_w, g, g_type, ld_g, m, ld_m, rows, cols, lr, mu, 1, decay, scale, steps, co, eps,
                                     None)


def test_orthogonalise_and_muon_refusals():
    n0 = lib.launch_count()
    nan, inf = float("nan"), float("inf")
    for bad in (dict(rows=-1), dict(cols=-1), dict(steps=0), dict(steps=-3), dict(eps=-1.0), dict(eps=nan), dict(eps=inf), dict(g_type=3)):
        assert orthogonalise(**bad) == INVALID, bad
        assert muon(**bad) == INVALID, bad
    assert orthogonalise(batch=-1) == INVALID and orthogonalise(out_type=0) == INVALID and orthogonalise(out_type=3) == INVALID
    assert orthogonalise(ld=7) == INVALID and orthogonalise(ld_out=7) == INVALID
    assert orthogonalise(batch=2, stride_out=31) == INVALID and orthogonalise(batch=2, stride=-1) == INVALID
    for bad in (dict(lr=nan), dict(mu=inf), dict(decay=nan), dict(scale=inf), dict(ld_w=7), dict(ld_g=7), dict(ld_m=7), dict()):
        assert muon(**bad) == INVALID, bad                        # the last: null pointers
    assert orthogonalise() == INVALID
    for big in (dict(rows=65537), dict(cols=65537), dict(steps=65)):
        assert orthogonalise(**big) == UNSUPPORTED and muon(**big) == UNSUPPORTED
    assert orthogonalise(batch=32768) == UNSUPPORTED
    assert orthogonalise(batch=0) == OK and orthogonalise(rows=0) == OK and orthogonalise(cols=0) == OK
    assert muon(rows=0) == OK and muon(cols=0) == OK
    # coefficients that do not keep the singular values near 1
    for co in ([3.0, 0.0, 0.0] * 5, [nan, 0.0, 0.0] * 5, [0.0, inf, 0.0] * 5, [1.5, 1.0, 1.0] * 5):
        assert orthogonalise(coeffs=co) == INVALID and muon(coeffs=co) == INVALID, co
    assert lib.launch_count() == n0


def test_binding_refusals():
    host = torch.zeros(4, 130)
    for call in (lambda: lib.fp8_quantise(host), lambda: lib.orthogonalise(host), lambda: lib.muon_step(host, host, host, 0.1),
                 lambda: lib.fp8_matmul(host.to(torch.float8_e4m3fn), torch.zeros(4, 2), host, host)):
        with pytest.raises(TypeError):
            call()
    with pytest.raises(ValueError):
        lib.orthogonalise(torch.zeros(3))
    with pytest.raises(ValueError):
        lib._coeffs((1.0, 2.0), 5)
    with pytest.raises(ValueError):
        lib._coeffs([(1.0, 2.0, 3.0)] * 4, 5)
    assert list(lib._coeffs((1.0, 2.0, 3.0), 2)) == [1.0, 2.0, 3.0] * 2
    assert list(lib._coeffs([(1, 2, 3), (4, 5, 6)], 2)) == [1, 2, 3, 4, 5, 6]


def test_driver_refusals():
    w, c = torch.zeros(4, 8), torch.zeros(16)
    args = (w, c, 4, 2, 1, 0.3, 0.1, 2, 1e-3)
    for bad in (dict(optimizer="adam"), dict(optimizer="muon"), dict(optimizer="muon", shape=(3, 8)), dict(x=torch.zeros(5, 8)),
                dict(x=torch.zeros(5, 7), shape=(4, 8)), dict(x=torch.zeros(0, 8), shape=(4, 8)), dict(weight_decay=0.1)):
        with pytest.raises(ValueError):
            qat.run(*args, **bad)


def test_command_refusals(capsys):
    for argv in (["--workload", "tiny", "--seqs", "16", "--loss", "layer", "--tokens", "0"],
                 ["--workload", "qtip", "--seqs", "3", "--optimizer", "muon"],
                 ["--workload", "tiny", "--weight-decay", "0.1"], ["--loss", "other"], ["--optimizer", "adam"]):
        with pytest.raises(SystemExit):
            qat.main(argv)
    capsys.readouterr()


def test_overlap_of_matrices():
    """Against the sets of bytes: equal and other row strides, types and offsets, rows between rows, single rows."""
    def bytes_of(t):
        return {t.data_ptr() + (r * t.stride(0) + c * t.stride(1)) * t.element_size() + i for r in range(t.shape[0])
                for c in range(t.shape[1]) for i in range(t.element_size())}

    room = torch.zeros(400)
    half = room.view(torch.float16)
    views = [room[at:at + 200].as_strided((r, c), (ld, 1), at) for at in (0, 3, 8, 40, 70) for r, c, ld in
             ((1, 5, 5), (4, 5, 20), (4, 15, 20), (3, 1, 7), (9, 4, 11), (0, 5, 5))]
    views += [half.as_strided((r, c), (ld, 1), at) for at in (1, 10, 81) for r, c, ld in ((4, 9, 40), (5, 30, 40), (2, 3, 11))]
    seen = set()
    for p in views:
        for q in views:
            want = bool(bytes_of(p) & bytes_of(q))
            assert lib._overlap(p, q) == want
            seen.add(want)
    assert seen == {True, False}


def test_products_of_the_driver():
    w, c = torch.zeros(4, 8), torch.zeros(16)
    with pytest.raises(ValueError):
        qat.run(w, c, 4, 2, 1, 0.3, 0.1, 2, 1e-3, x=torch.zeros(5, 8), shape=(4, 8), products="bf16")
    with pytest.raises(SystemExit):
        qat.main(["--loss", "layer", "--products", "int8"])


def test_command_without_rows(capsys):
    for seqs in ("0", "-8", "-16"):
        for argv in (["--loss", "layer"], ["--optimizer", "muon"]):
            with pytest.raises(SystemExit):
                qat.main(["--workload", "tiny", "--seqs", seqs, *argv])
    capsys.readouterr()
