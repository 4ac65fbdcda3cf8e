"""Plain 64-bit forms for rows with a scale per 128 elements, and bounds for coded results.

A code is off by at most half a step of its type relative to the value (2^-4 E4M3, 2^-3 E5M2) or, below
the normal range, half the smallest step (2^-10, 2^-17) times the scale; forming value * dyn, dyn and
1 / dyn takes three more fp32 roundings (2^-24 each, counted as 2^-22 together).
"""
import torch

import experts_ref as ref

F8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
TOP = {"e4m3": 448.0, "e5m2": 57344.0}
HALF = {"e4m3": 2.0 ** -4, "e5m2": 2.0 ** -3}
LEAST = {"e4m3": 2.0 ** -10, "e5m2": 2.0 ** -17}


def groups(n):
    return (n + 127) // 128


def spread(s, dim, n):
    return s.double().repeat_interleave(128, dim).narrow(dim, 0, n)


def rows_f64(codes, scales):
    """[R][I] codes with scales [R][ceil(I / 128)]."""
    return codes.double() * spread(scales, -1, codes.shape[-1])


def weights_f64(codes, scales, parts):
    """[E][parts * n][I] codes with scales [E][parts * ceil(n / 128)][ceil(I / 128)]."""
    E, N, I = codes.shape
    n = N // parts
    s = spread(spread(scales.view(E, parts, groups(n), groups(I)), 2, n), 3, I)
    return codes.double() * s.reshape(E, N, I)


def check_codes(codes, scales, y, err, kind, rows):
    """Codes (as float8) [cap][M] and scales [cap][ceil(M / 128)] against fp64 values off by at
    most err."""
    M = y.shape[1]
    c, s = codes[:rows].double(), scales[:rows].double()
    assert torch.isfinite(c).all() and torch.isfinite(s).all()
    pad = (0, -M % 128)
    most = torch.nn.functional.pad(y.abs(), pad).view(rows, groups(M), 128).amax(2)
    worst = torch.nn.functional.pad(err, pad).view(rows, groups(M), 128).amax(2)
    far = (s * TOP[kind] - most).abs() - (worst + 2.0 ** -22 * (most + worst))
    assert (far <= 0).all(), float(far.max())
    wide = spread(s, 1, M)
    diff = (c * wide - y).abs()
    tol = err + (HALF[kind] + 2.0 ** -22) * (y.abs() + err) + LEAST[kind] * wide
    assert (diff <= tol).all(), (int((diff > tol).sum()), float((diff / tol).nan_to_num().max()))


def product(x, xs, w, ws, ranges, swiglu, cut=True):
    return ref.product(rows_f64(x, xs), weights_f64(w, ws, 2 if swiglu else 1), ranges, swiglu, cut=cut)
