"""Per-head RMS norm and position rotation in 64 bits, and the bound on a
f32 computation of them (shared by tests; not collected)."""
import numpy as np

U = 2.0 ** -24  # half a unit in the last place of f32, relative


def angles(pos, freqs):
    """Angles [N, rd/2] in radians of int positions and 64-bit turn frequencies: the
    product's low 64 bits are the fraction of a turn."""
    with np.errstate(over="ignore"):
        turns = pos.astype(np.int64).view(np.uint64)[:, None] * freqs.view(np.uint64)[None, :]
    return turns.astype(np.float64) * (2.0 * np.pi / 2.0 ** 64)


def norm_rope(x, pos, freqs, *, norm=False, weight=None, offset=0.0, eps=1e-6, interleaved=False):
    """(y, bound) of x [N, H, D] (any float type) in float64.

    bound: |f32 result - y| in exact arithmetic of the inputs.  With u = 2^-24:
    the sum of squares takes 16 fused adds in a thread and up to 4 across
    threads (20 u), so r = 1/sqrt(mean + eps) is off by 10 u and 3 more roundings;
    two products and the weight's sum bring a value to 16 u.  sincospif is
    within 2 u of its f32 argument's sine, whose rounding (2^-25 of half a
    turn) adds 1.6 u: 4 u.  Two products, a sum: 3 u.  Together at most
    (16 + 4 + 3) u (|y_lo| + |y_hi|), counted as 24."""
    x = x.astype(np.float64)
    y = x
    if norm:
        y = x / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps)
        if weight is not None:
            y = y * (weight.astype(np.float64) + offset)
    z, mag = y.copy(), np.abs(y)
    rd = 2 * len(freqs)
    if rd:
        a = angles(pos, freqs)
        c, s = np.cos(a)[:, None], np.sin(a)[:, None]
        if interleaved:
            lo, hi = np.arange(0, rd, 2), np.arange(1, rd, 2)
        else:
            lo, hi = np.arange(rd // 2), np.arange(rd // 2, rd)
        z[..., lo] = y[..., lo] * c - y[..., hi] * s
        z[..., hi] = y[..., lo] * s + y[..., hi] * c
        m = np.abs(y[..., lo]) + np.abs(y[..., hi])
        mag = mag.copy()
        mag[..., lo] = mag[..., hi] = m
    return z, 24 * U * mag


def half_bound(y, bound):
    """The bound after rounding to f16: half a step, 2^-11 relative or 2^-25
    below the smallest normal."""
    return bound + np.maximum((np.abs(y) + bound) * 2.0 ** -11, 2.0 ** -25)
