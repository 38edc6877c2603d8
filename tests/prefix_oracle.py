"""Dense attention over whole sequences in 64 bits, and how far a bf16 / f32
result computed with f16 operands may be from it (test infrastructure)."""
import math

import numpy as np

_LEVELS = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])


def fp4_rows(codes, scales):
    """float64 values of FP4 rows (codes [n, 256], scales [n, 32] as bytes)."""
    import torch
    c = np.stack((codes & 15, codes >> 4), -1).reshape(len(codes), 512)
    v = _LEVELS[c & 7] * np.where(c & 8, -1.0, 1.0)
    s = torch.from_numpy(np.ascontiguousarray(scales)).view(torch.float8_e4m3fn).double().numpy()
    return v * np.repeat(s, 16, axis=1)


def e4m3_rows(b):
    import torch
    return torch.from_numpy(np.ascontiguousarray(b)).view(torch.float8_e4m3fn).double().numpy()


def attend(q, v, scale):
    """o, lse of q [h, 512] over rows v [n, 512], and the bounds of both.

    What the kernel rounds: scores are f32 sums of 512 exact products (at most
    512 roundings of 2^-23 of the sum of their magnitudes each, where the
    tensor core truncates, and the scaling), exp2's argument and result 2^-21;
    probabilities are f16 (2^-11, or 2^-25 absolute below 2^-14; the running
    maximum may be up to 2^8 low, so probabilities are at most 2^8 and their
    sum at least 2^-8 of that scale); the output is bf16 (2^-8)."""
    if len(v) == 0:
        z = np.zeros((len(q), 512))
        inf = np.full(len(q), -math.inf)
        return z, inf, z, np.zeros(len(q))
    s = q @ v.T * scale
    m = s.max(1, keepdims=True)
    p = np.exp(s - m)
    l = p.sum(1, keepdims=True)
    o, lse = (p / l) @ v, (m + np.log(l))[:, 0]
    es = 512 * 2.0 ** -23 * (np.abs(q) @ np.abs(v).T).max(1) * abs(scale) + 2.0 ** -21 * (np.abs(s).max(1) + 1)
    spread = (p / l) @ np.abs(v)
    tol = 2.0 ** -8 * np.abs(o) + (2.0 ** -11 + 2 * es[:, None]) * spread * 1.01 + len(v) * 2.0 ** -25 * np.abs(v).max() / np.minimum(l, 1.0)
    return o, lse, tol, 2 * es + 2.0 ** -20 * (np.abs(lse) + 1)
