"""Plain implementations (numpy, 64 bits) of the 8-bit block operators and of the router
with groups, shared by their GPU tests.

Tolerances used with them (derived from the formats, not from results):
  codes     of plain rows follow from single fp32 operations, so codes and scales have to
            be equal bit for bit.  Those of SwiGLU and its gradient come after a handful of
            fp32 roundings and an exponential, 64 * 2^-24 of the magnitude of the terms; a
            code is then off its value by half a step, 2^-4 of it (2^-10 of the scale
            below 2^-6), on top of that
  products  of codes are exact; a block's 128 are added with at most one unit in the last
            place each (2^-23 of the terms' magnitudes), and every block joins with one
            fp32 rounding of the product of its scales, one of the sum, one of the
            multiplication: (256 + 3 blocks) * 2^-24 of the sum of the terms' magnitudes
  bf16      one rounding more, 2^-8 of the element
"""

import numpy as np

import operator_refs as ref

SMALLEST = np.float32(2.0 ** -100)
FP32 = ref.FP32


def e4m3_values():
    """Value of every code."""
    c = np.arange(256)
    e, m = (c >> 3) & 15, c & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e.astype(np.float64) - 10))
    v = np.where((c & 127) == 127, np.nan, v)
    return np.where(c >= 128, -v, v)


VALUES = e4m3_values()
STEPS = VALUES[:127]                     # non-negative, ascending


def e4m3(v):
    """Codes of fp32 values: to nearest, ties to the even code, saturating."""
    v = np.asarray(v, np.float64)
    a = np.minimum(np.abs(np.nan_to_num(v)), 448.0)
    hi = np.clip(np.searchsorted(STEPS, a), 0, 126)
    lo = np.maximum(hi - 1, 0)
    up, down = STEPS[hi] - a, a - STEPS[lo]
    code = np.where(down < up, lo, np.where(up < down, hi, np.where(hi % 2 == 0, hi, lo)))
    code = code | np.where(np.signbit(v), 128, 0)
    return np.where(np.isnan(v), 127, code).astype(np.uint8)


def block_scales(top, pow2):
    """(scale, factor) in fp32 from the largest magnitudes."""
    with np.errstate(all="ignore"):
        top = np.where(np.isnan(top), top, np.maximum(top.astype(np.float32), SMALLEST))
        scale, factor = top / np.float32(448), np.float32(448) / top
        if pow2:
            fine = np.isfinite(top)
            m, e = np.frexp(np.where(fine, scale, 1))
            e = np.where(m == 0.5, e - 1, e)
            scale = np.where(fine, np.ldexp(np.float32(1), e), scale)
            factor = np.where(fine, np.ldexp(np.float32(1), -e), factor)
    return scale.astype(np.float32), factor.astype(np.float32)


def by_row(v, pow2=False):
    """fp32 [M, width] -> codes [M, width], scales [blocks, M]."""
    M, width = v.shape
    nb = (width + 127) // 128
    w = np.zeros((M, nb * 128), np.float32)
    w[:, :width] = v
    b = w.reshape(M, nb, 128)
    scale, factor = block_scales(np.abs(b).max(2) if M else np.zeros((0, nb)), pow2)
    with np.errstate(all="ignore"):
        codes = e4m3(b * factor[:, :, None]).reshape(M, -1)[:, :width]
    return codes, scale.T


def columns(offsets, M):
    """First column of each segment (and the end), and each row's column (-1: none)."""
    n = [0]
    place = np.full(M, -1)
    for e in range(len(offsets) - 1):
        lo, hi = offsets[e], offsets[e + 1]
        place[lo:hi] = n[-1] + np.arange(hi - lo)
        n.append(n[-1] + (hi - lo + 127) // 128 * 128)
    return n, place


def by_column(v, offsets, pow2=False):
    """fp32 [M, width] -> codes [width, used], scales [used / 128, width] of the columns
    that the segments take."""
    n, place = columns(offsets, v.shape[0])
    tall = np.zeros((v.shape[1], n[-1]), np.float32)
    rows = place >= 0
    tall[:, place[rows]] = v[rows].T
    return by_row(tall, pow2)


def by_tile(w, pow2=False):
    """fp32 [E, N, K] -> codes, scales [E, ceil(N/128), ceil(K/128)]."""
    E, N, K = w.shape
    nb, kb = (N + 127) // 128, (K + 127) // 128
    codes, scales = np.zeros(w.shape, np.uint8), np.zeros((E, nb, kb), np.float32)
    for e in range(E):
        for i in range(nb):
            for j in range(kb):
                at = (e, slice(128 * i, 128 * i + 128), slice(128 * j, 128 * j + 128))
                s, f = block_scales(np.abs(w[at]).max()[None], pow2)
                scales[e, i, j] = s[0]
                with np.errstate(all="ignore"):
                    codes[at] = e4m3(w[at] * f[0])
    return codes, scales


def values(codes, scales):
    """64-bit values of row codes."""
    with np.errstate(all="ignore"):
        s = np.repeat(np.asarray(scales, np.float64).T, 128, 1)[:, :codes.shape[1]]
        return VALUES[codes] * s


def tile_values(codes, scales):
    E, N, K = codes.shape
    s = np.repeat(np.repeat(np.asarray(scales, np.float64), 128, 1), 128, 2)[:, :N, :K]
    return VALUES[codes] * s


def swiglu(a, clamp=0.0):
    """64-bit (h, the magnitude that its error goes by)."""
    C = a.shape[1] // 2
    g, u = a[:, :C].astype(np.float64), a[:, C:].astype(np.float64)
    if clamp:
        g, u = np.clip(g, -clamp, clamp), np.clip(u, -clamp, clamp)
    h = g * ref.sigmoid(g) * u
    return h, np.abs(h) * (1 + np.abs(g))


def swiglu_grad(dh, a, clamp=0.0):
    C = a.shape[1] // 2
    g0, u0 = a[:, :C].astype(np.float64), a[:, C:].astype(np.float64)
    g, u, d = g0, u0, dh.astype(np.float64)
    if clamp:
        g, u = np.clip(g, -clamp, clamp), np.clip(u, -clamp, clamp)
    s = ref.sigmoid(g)
    dg, du = d * u * s * (1 + g * (1 - s)), d * g * s
    mag = np.abs(d * u * s) * (1 + np.abs(g)) ** 2, np.abs(du) * (1 + np.abs(g))
    if clamp:
        dg, du = np.where(np.abs(g0) > clamp, 0, dg), np.where(np.abs(u0) > clamp, 0, du)
    return np.concatenate([dg, du], 1), np.concatenate(mag, 1)


def check_codes(codes, scales, want, mag, what):
    """Codes [rows, K] and scales [K/128, rows] of `want`, known to FP32 * mag."""
    rows, K = want.shape
    nb = (K + 127) // 128
    pad = lambda v: np.pad(v, ((0, 0), (0, nb * 128 - K))).reshape(rows, nb, 128)
    top, off = np.abs(pad(want)).max(2), FP32 * pad(mag).max(2)
    scale = np.maximum(top, 2.0 ** -100) / 448
    assert np.all(np.abs(scales.T - scale) <= off / 448 + 2.0 ** -23 * scale), what
    got = values(codes, scales)
    step = np.repeat(scales.T.astype(np.float64), 128, 1)[:, :K]
    near = 2.0 ** -4 * (np.abs(want) + FP32 * mag) * (1 + 2.0 ** -20) + FP32 * mag
    low = 2.0 ** -10 * step * (1 + 2.0 ** -20) + FP32 * mag
    # the largest of a block may lie above 448 by what the scale is off
    assert np.all(np.abs(got - want) <= np.maximum(near, low)), what


def check_product(got, a, b, what, bf16=False, base=None):
    """got against a b^T (64-bit values [M, K], [N, K]), plus base."""
    want, mag = a @ b.T, np.abs(a) @ np.abs(b).T
    tol = (256 + 3 * ((a.shape[1] + 127) // 128)) * 2.0 ** -24 * mag
    if base is not None:
        want, tol = want + base, tol + 2.0 ** -24 * (np.abs(base) + mag)
    if bf16:
        tol = tol + 2.0 ** -8 * (np.abs(want) + tol)
    off = np.abs(np.asarray(got, np.float64) - want)
    assert np.all(off <= tol), (what, float((off - tol).max()))


# ---- router with groups --------------------------------------------------------


def group_choice(logits, k, groups, top, scoring, pair, bias=None):
    """ids by the definition, on 64-bit keys."""
    T, E = logits.shape
    size = E // groups
    l = logits.astype(np.float64)
    ids = np.empty((T, k), np.int32)
    for t in range(T):
        with np.errstate(all="ignore"):
            if scoring == "sigmoid":
                s = ref.sigmoid(l[t])
            else:
                m = np.fmax.reduce(l[t])
                s = np.exp(l[t] - m)
                s = s / s.sum()
            key = s if bias is None else s + bias.astype(np.float64)
        key = np.where(l[t] == -np.inf, -np.inf, key)
        order = l[t] if bias is None else key
        count = np.where(np.isnan(l[t] if bias is None and not pair else key), -np.inf,
                         l[t] if bias is None and not pair else key)
        best = -np.sort(-count.reshape(groups, size), 1)
        value = best[:, 0].copy()
        if pair and size > 1:
            value += np.where(best[:, 1] > -np.inf, best[:, 1], 0.0)
        kept = sorted(range(groups), key=lambda g: (-value[g], g))[:top]
        inside = [e for e in range(E) if e // size in kept]
        rank = sorted(inside, key=lambda e: (bool(np.isnan(order[e])),
                                             0.0 if np.isnan(order[e]) else -order[e], e))
        ids[t] = rank[:k]
    return ids
