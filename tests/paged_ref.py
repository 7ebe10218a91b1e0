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


def visible(p, window, sinks):
    """Mask over rows 0 .. p of the rows that a query at position p sees."""
    j = np.arange(p + 1)
    return (window == 0) | (j > p - window) | (j < sinks)


def attend(q, k, v, table, kv_len, new, scale, window=0, sinks=0):
    """q [H_q][T][d], pools k and v [page][H_kv][row][d], table [n_seq][pages], all float64 or int; new[s] rows of
    sequence s, one sequence after the other.  Returns O, lse and two magnitudes for the tolerances: sum_j p_j |v_j|
    [H_q][T][d] and max_j scale * sum |q_c k_jc| [H_q][T]."""
    Hq, T, d = q.shape
    G = Hq // k.shape[1]
    pr = k.shape[2]
    O, A = np.zeros((Hq, T, d)), np.zeros((Hq, T, d))
    lse, S = np.full((Hq, T), -np.inf), np.zeros((Hq, T))
    t = 0
    for s, n in enumerate(new):
        held = int(kv_len[s])
        for i in range(n):
            p = held - n + i
            if p >= 0:
                j = np.nonzero(visible(p, window, sinks))[0]
                pages, rows = np.asarray(table)[s, j // pr], j % pr
                for h in range(Hq):
                    K, V = k[pages, h // G, rows], v[pages, h // G, rows]
                    x = scale * (K @ q[h, t + i])
                    S[h, t + i] = abs(scale) * (np.abs(K) @ np.abs(q[h, t + i])).max()
                    m = x.max()
                    w = np.exp(x - m)
                    lse[h, t + i] = m + np.log(w.sum())
                    w /= w.sum()
                    O[h, t + i], A[h, t + i] = w @ V, w @ np.abs(V)
        t += n
    return O, lse, A, S


def attend_tol(O, lse, A, S, d, n, eps, p_eps):
    """How far a kernel that accumulates in fp32 may be from O and lse.  Scores: a sum of d products, each addition
    off by at most 2^-23 of what is summed so far (the tensor core may truncate), then scale, log2 e and the maximum
    subtracted: (d + 4) 2^-23 S.  A probability is off by twice that (its own score and the maximum's; the error is
    small, so expm1 is covered by the factor), 2^-22 for the exponential, and p_eps, half a step of the form in which it
    enters the second product.  That product and the sum of n probabilities add at most (n + 64) 2^-23 each.  The output
    is rounded to eps / 2."""
    x = 2.5 * (d + 4) * 2.0 ** -23 * S + 2.0 ** -21 + (n + 64) * 2.0 ** -22
    t = (x + p_eps)[..., None] * A if np.ndim(x) else (x + p_eps) * A
    # the logarithm's own rounding: 2^-22 of |lse|, and of the base-2 maximum it is added to
    return t + eps / 2 * (np.abs(O) + t), x + 2.0 ** -21 * (np.abs(np.where(np.isfinite(lse), lse, 0)) + 1)
