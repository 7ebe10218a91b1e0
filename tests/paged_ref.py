"""Plain 64-bit forms of the paged-cache operators (numpy, one row at a time) for the tests."""
import numpy as np


def inv_freq(rot, base=10000.0, scaling="none", factor=1.0, orig_len=4096, beta_slow=1.0, beta_fast=32.0):
    ld = np.longdouble
    i = np.arange(rot // 2, dtype=ld)
    b = ld(base) * (ld(factor) ** (ld(rot) / (rot - 2)) if scaling == "base" else 1)
    f = b ** (-2 * i / rot)
    if scaling == "linear":
        f = f / factor
    if scaling == "ramp":
        r = orig_len * f / (2 * ld(np.pi) + ld(2.4492935982947064e-16))  # 2 pi beyond its 53 bits
        g = np.clip((r - beta_slow) / (beta_fast - beta_slow), 0, 1)
        f = g * f + (1 - g) * f / factor
    return f


def rotate(x, pos, freq, interleaved=False, mscale=1.0, sign=1):
    """x [H][T][d] (float64), pos [T]; pairs turned by sign * pos * freq.  Extended precision: at a position
    of 2^31 a product in 64 bits would be off by 2^-22."""
    x = np.asarray(x, np.float64)
    r = 2 * len(freq)
    a = np.asarray(pos, np.longdouble)[:, None] * np.asarray(freq, np.longdouble)
    c, s = np.cos(a).astype(np.float64) * mscale, sign * np.sin(a).astype(np.float64) * mscale
    y = x.copy()
    i0 = np.arange(0, r, 2) if interleaved else np.arange(r // 2)
    i1 = i0 + 1 if interleaved else i0 + r // 2
    y[..., i0] = x[..., i0] * c - x[..., i1] * s
    y[..., i1] = x[..., i1] * c + x[..., i0] * s
    return y


def rotate_tol(x, y, rot, eps, interleaved=False, mscale=1.0):
    """How far the kernel's rotation may be from y: half a step of the output type, and in fp32 2^-21 of
    (|x_a| + |x_b|) mscale for each element of a pair: the half turns are rounded to fp32 (2^-25 of a half
    turn: 2^-23.3 in angle), sincospi is good to 2 units in the last place (2^-23 at 1), mscale and the
    two products add 3 roundings of 2^-24; 2^-23.3 + 2^-23 + 3 * 2^-24 < 2^-21."""
    x = np.abs(np.asarray(x, np.float64))
    t = np.zeros_like(x)
    i0 = np.arange(0, rot, 2) if interleaved else np.arange(rot // 2)
    i1 = i0 + 1 if interleaved else i0 + rot // 2
    t[..., i0] = t[..., i1] = (x[..., i0] + x[..., i1]) * abs(mscale) * 2.0 ** -21
    return t + eps / 2 * (np.abs(y) + t)
