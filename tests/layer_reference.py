"""Plain 64-bit forms of the layer-wise QAT operators, on the CPU, for the tests."""
import math

import numpy as np
import torch

BLOCK = 128
#: (largest value, mantissa bits, least exponent) of the 8-bit types
FORMATS = {torch.float8_e4m3fn: (448.0, 3, -6), torch.float8_e5m2: (57344.0, 2, -14)}


def quantise(v, block_rows, dtype):
    """Values of codes and scales (fp64 arrays) of a matrix of fp32 values, entry by entry
    from the definition; a block that is not finite is NaN throughout."""
    largest, digits, lowest = FORMATS[dtype]
    v = np.asarray(v, np.float64)
    rows, cols = v.shape
    q = np.empty_like(v)
    scale = np.empty((-(-rows // block_rows), -(-cols // BLOCK)))
    for i in range(scale.shape[0]):
        for j in range(scale.shape[1]):
            at = np.s_[i * block_rows:(i + 1) * block_rows, j * BLOCK:(j + 1) * BLOCK]
            b = v[at]
            if not np.isfinite(b).all():
                scale[i, j] = np.nan
                q[at] = np.nan
                continue
            most = np.abs(b).max()
            e = 0
            if most > 0:
                e = max(-127, math.frexp(most)[1] - math.frexp(largest)[1] - 1)
                while most > largest * 2.0 ** e:
                    e += 1
            scale[i, j] = 2.0 ** e
            y = b / scale[i, j]
            ex = np.maximum(np.frexp(y)[1] - 1, lowest)       # 2^ex <= |y| < 2^(ex + 1)
            unit = np.ldexp(1.0, ex - digits)
            q[at] = np.rint(y / unit) * unit
    return q, scale


def values(q, scale, block_rows):
    """What codes and scales (torch tensors) stand for, fp64."""
    q = q.detach().cpu().double()
    s = scale.detach().cpu().float().double()
    return q * s.repeat_interleave(block_rows, 0)[: q.shape[0]].repeat_interleave(BLOCK, 1)[:, : q.shape[1]]


MUON = (3.4445, -4.7750, 2.0315)


def newton_schulz(g, steps=5, coeffs=None, eps=1e-7):
    """The iteration on the last two dimensions, fp64 (on g's device)."""
    x = torch.as_tensor(g).detach().double()
    x = x / (torch.linalg.vector_norm(x, dim=(-2, -1), keepdim=True) + eps)
    for s in range(steps):
        a, b, c = coeffs[s] if coeffs is not None else MUON
        if x.shape[-2] > x.shape[-1]:
            t = x.mT @ x
            x = a * x + x @ (b * t + c * t @ t)
        else:
            t = x @ x.mT
            x = a * x + (b * t + c * t @ t) @ x
    return x
