"""Plain 64-bit implementations of the operators around the experts (numpy).

Shared by the GPU tests of the router, the block norms and the decode path.
Tolerances used with them (derived from the formats, not from results):
  fp32   every step is one rounding of 2^-24 relative to the terms it adds; a result
         takes some tens of them (exponentials of logits up to 2^4 included) and
         sums over rows or columns go through partial sums of at most a few hundred
         terms, so 64 * 2^-24 of the sum of the terms' magnitudes bounds the error
  bf16   one rounding to 8 significant bits, at most 2^-8 of the element (half of
         the 2^-7 spacing above a power of two), on top of the fp32 error
The gradients cancel (a projection is taken out of each row), so the references
also return `mag`: the same sums with every term's absolute value.
"""

import numpy as np

FP32 = 64 * 2.0 ** -24
BF16 = 2.0 ** -8


def check(got, want, what, mag=None, bf16=False):
    """got against want, elementwise with `mag`, else in norm for fp32 and against the
    row's rms for bf16; NaN and infinities have to be the same."""
    got, want = np.asarray(got, np.float64), np.asarray(want, np.float64)
    assert got.shape == want.shape, what
    fine = np.isfinite(want)
    assert np.array_equal(np.isnan(want), np.isnan(got)), what
    assert np.array_equal(want[~fine & ~np.isnan(want)], got[~fine & ~np.isnan(want)]), what
    if not want.size:
        return
    off = np.where(fine, np.abs(got - want), 0.0)
    size = np.where(fine, np.abs(want), 0.0)
    if mag is None and not bf16:
        assert np.linalg.norm(off) <= FP32 * np.linalg.norm(size), (
            what, np.linalg.norm(off) / max(np.linalg.norm(size), 1e-300))
        return
    if mag is None:
        mag = np.sqrt(np.mean(size ** 2, axis=-1, keepdims=True))
    over = off - (BF16 if bf16 else 0.0) * size - FP32 * np.maximum(mag, size)
    assert over.max() <= 0, (what, over.max())


# ---- router --------------------------------------------------------------------


def sigmoid(v):
    e = np.exp(-np.abs(v))
    return np.where(v >= 0, 1.0, e) / (1.0 + e)


def choose(key, k):
    """Per row the k largest, ties to the lowest index, NaN below everything."""
    out = np.empty((key.shape[0], k), np.int32)
    for t, row in enumerate(key):
        rank = sorted(range(len(row)), key=lambda e: (bool(np.isnan(row[e])),
                                                      -row[e] if not np.isnan(row[e]) else 0.0, e))
        out[t] = rank[:k]
    return out


def router_forward(logits, k, scoring, scale=1.0, bias=None, mask=None, ids=None):
    """logits: fp32 or fp64 [T, E]; the choice is made on fp32(logits) + fp32(bias)."""
    T, E = logits.shape
    l = logits.astype(np.float64)
    given = np.ones(T, bool) if mask is None else mask != 0
    if ids is None:
        key = logits.astype(np.float32)
        with np.errstate(invalid="ignore"):
            ids = choose(key if bias is None else key + bias.astype(np.float32), k)
        for t in np.nonzero(~given)[0]:
            ids[t] = (t * k + np.arange(k)) % E
    scores = np.zeros((T, k))
    p = np.zeros((T, E))
    stat = np.full(T, -np.inf)
    counts = np.zeros(E + 1, np.int64)
    for t in range(T):
        if not given[t] or np.all(l[t] == -np.inf):
            continue
        counts[E] += 1
        c = l[t, ids[t]]
        for e in ids[t][c != -np.inf]:
            counts[e] += 1
        if scoring == "sigmoid":
            s = sigmoid(l[t])
            stat[t] = np.log(s.sum())
            p[t] = s / s.sum()
            w = sigmoid(c)
        else:
            top = l[t].max()
            s = np.exp(l[t] - top)
            stat[t] = top + np.log(s.sum())
            p[t] = s / s.sum()
            w = p[t, ids[t]] if scoring == "softmax" else np.where(
                c == -np.inf, 0.0, np.exp(c - max(c.max(), -1e300)))
        if scoring != "softmax":
            w = w / w.sum() if w.sum() > 0 else np.zeros(k)
        scores[t] = scale * w
    n = max(int(counts[E]), 1)
    z = 0.0
    if scoring != "sigmoid":
        z = np.sum(stat[np.isfinite(stat)] ** 2) / n
    prob_sum = p.sum(0)
    balance = E / (k * n * n) * np.dot(counts[:E], prob_sum)
    return dict(ids=ids, scores=scores, counts=counts, prob_sum=prob_sum,
                losses=np.array([balance, z]), row_stat=stat)


def router_backward(logits, ids, counts, stat, k, scoring, scale=1.0, d_scores=None,
                    d_losses=None):
    """The gradient by the chain rule, one row at a time.  -> (gradient, mag)"""
    T, E = logits.shape
    l = logits.astype(np.float64)
    n = max(int(counts[E]), 1)
    dl, mag = np.zeros((T, E)), np.zeros((T, E))
    d_losses = np.zeros(2) if d_losses is None else np.asarray(d_losses, np.float64)
    dp = d_losses[0] * E * counts[:E].astype(np.float64) / (k * n * n)
    for t in range(T):
        if stat[t] == -np.inf:
            continue
        v = np.zeros(k) if d_scores is None else scale * d_scores[t].astype(np.float64)
        c = l[t, ids[t]]
        v = np.where(c == -np.inf, 0.0, v)
        if scoring == "sigmoid":
            s = sigmoid(l[t])
            p = s / s.sum()
            ds = (dp - np.dot(dp, p)) / s.sum()
            m = (np.abs(dp) + np.dot(np.abs(dp), p)) / s.sum()
            w = sigmoid(c)
            if w.sum() > 0:
                ds[ids[t]] += (v - np.dot(v, w) / w.sum()) / w.sum()
                m[ids[t]] += (np.abs(v) + np.dot(np.abs(v), w) / w.sum()) / w.sum()
            dl[t], mag[t] = ds * s * (1 - s), m * s
            continue
        p = np.exp(l[t] - l[t].max())
        p /= p.sum()
        g, a = dp.copy(), np.abs(dp)
        if scoring == "softmax":
            g[ids[t]] += v
            a[ids[t]] += np.abs(v)
        z = d_losses[1] * 2 * stat[t] / n
        dl[t], mag[t] = p * (g - np.dot(g, p) + z), p * (a + np.dot(a, p) + np.abs(z))
        if scoring == "softmax_topk" and np.any(c != -np.inf):
            w = np.where(c == -np.inf, 0.0, np.exp(c - c.max()))
            w /= w.sum()
            dl[t, ids[t]] += w * (v - np.dot(v, w))
            mag[t, ids[t]] += w * (np.abs(v) + np.dot(np.abs(v), w))
    return dl, mag


# ---- block norms -----------------------------------------------------------------


def block_norm_forward(res, y=None, w_post=None, gate=None, w_pre=None, alpha=1.0, eps=1e-6):
    """gate: broadcast against [T, d].  -> (out, u)"""
    out = res.astype(np.float64)
    if y is not None:
        y = y.astype(np.float64)
        n = y
        if w_post is not None:
            n = y / np.sqrt(np.mean(y * y, 1, keepdims=True) + eps) * w_post.astype(np.float64)
        out = out + alpha * (1.0 if gate is None else gate.astype(np.float64)) * n
    u = None
    if w_pre is not None:
        u = out / np.sqrt(np.mean(out * out, 1, keepdims=True) + eps) * w_pre.astype(np.float64)
    return out, u


def block_norm_backward(x, y=None, w_post=None, gate=None, w_pre=None, d_out=None, d_u=None,
                        alpha=1.0, eps=1e-6):
    """The gradient at the stream x after the block.  -> (r, mag), each a dict of
    d_residual, dy, dw_post, dw_pre and dgate_full [T, d] (to be summed over what the
    gate was broadcast over)."""
    mean = lambda v: np.mean(v, 1, keepdims=True)
    x = x.astype(np.float64)
    dr = np.zeros_like(x) if d_out is None else d_out.astype(np.float64).copy()
    r, mag = {}, {}
    big = np.abs(dr)
    if d_u is not None:
        d_u = d_u.astype(np.float64)
        inv = 1.0 / np.sqrt(mean(x * x) + eps)
        r["dw_pre"], mag["dw_pre"] = np.sum(d_u * x * inv, 0), np.sum(np.abs(d_u * x * inv), 0)
        t = d_u * w_pre.astype(np.float64)
        dr += inv * t - inv ** 3 * x * mean(t * x)
        big += inv * np.abs(t) + inv ** 3 * np.abs(x) * mean(np.abs(t * x))
    r["d_residual"], mag["d_residual"] = dr, big
    if y is not None:
        y = y.astype(np.float64)
        g = np.float64(1.0) if gate is None else gate.astype(np.float64)
        dn, bign = alpha * g * dr, np.abs(alpha * g) * big
        n = y
        if w_post is not None:
            inv = 1.0 / np.sqrt(mean(y * y) + eps)
            w = w_post.astype(np.float64)
            n = y * inv * w
            r["dw_post"], mag["dw_post"] = np.sum(dn * y * inv, 0), np.sum(bign * np.abs(y) * inv, 0)
            t, bigt = dn * w, bign * np.abs(w)
            r["dy"] = inv * t - inv ** 3 * y * mean(t * y)
            mag["dy"] = inv * bigt + inv ** 3 * np.abs(y) * mean(bigt * np.abs(y))
        else:
            r["dy"], mag["dy"] = dn, bign
        r["dgate_full"], mag["dgate_full"] = alpha * dr * n, np.abs(alpha * n) * big
    return r, mag
