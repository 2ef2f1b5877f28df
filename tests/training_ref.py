"""Plain 64-bit definitions (numpy) of the training operators, for their tests."""
import numpy as np


def softmax(z):
    with np.errstate(invalid="ignore", over="ignore"):
        m = z.max(axis=1, keepdims=True)
        p = np.exp(z - m)
        p = p / p.sum(axis=1, keepdims=True)
    p[np.all(z == -np.inf, axis=1)] = 0.0
    return p


def sequences(T, seq_offsets, mask):
    off = [0, T] if seq_offsets is None else list(seq_offsets)
    keep = np.ones(T, bool) if mask is None else mask.astype(bool)
    return [np.array([t for t in range(a, b) if keep[t]], dtype=int) for a, b in zip(off[:-1], off[1:])]


def balance(logits, idx, coef, seq_offsets=None, mask=None):
    z = logits.astype(np.float64)
    T, E = z.shape
    k = idx.shape[1]
    p = softmax(z)
    rows = sequences(T, seq_offsets, mask)
    S = len(rows)
    counts = np.zeros((S, E), np.int64)
    prob = np.zeros((S, E))
    used = sum(len(r) > 0 for r in rows)
    loss = 0.0
    for s, r in enumerate(rows):
        if len(r) == 0:
            continue
        ids = idx[r].ravel()
        counts[s] = np.bincount(ids[(ids >= 0) & (ids < E)], minlength=E)
        prob[s] = p[r].mean(axis=0)
        loss += coef / used * (E * counts[s] / (k * len(r)) * prob[s]).sum()
    return loss, counts, prob, np.array([len(r) for r in rows] + [used])


def route_backward(logits, idx, gates=None, dgates=None, dloss=None, coef=0.0, seq_offsets=None, mask=None):
    """The gradient and, entry by entry, the sum of the magnitudes it adds up."""
    z = logits.astype(np.float64)
    T, E = z.shape
    k = idx.shape[1]
    d, size = np.zeros((T, E)), np.zeros((T, E))
    if dloss is not None:
        p = softmax(z)
        _, counts, _, tokens = balance(logits, idx, coef, seq_offsets, mask)
        for s, r in enumerate(sequences(T, seq_offsets, mask)):
            if len(r) == 0:
                continue
            f = E * counts[s] / (k * len(r))
            w = dloss * coef / (tokens[-1] * len(r))
            dot = p[r] @ f
            d[r] = w * p[r] * (f - dot[:, None])
            size[r] = abs(w) * p[r] * (f + dot[:, None])
    if dgates is not None:
        g, dg = gates.astype(np.float64), dgates.astype(np.float64)
        a = g * (dg - (g * dg).sum(axis=1, keepdims=True))
        b = g * (np.abs(dg) + (g * np.abs(dg)).sum(axis=1, keepdims=True))
        for t in range(T):
            for j in range(k):
                if 0 <= idx[t, j] < E:
                    d[t, idx[t, j]] += a[t, j]
                    size[t, idx[t, j]] += b[t, j]
    return d, size


_MAG = np.array([(m * 2.0 ** -9) if e == 0 else (8 + m) * 2.0 ** (e - 10) for e in range(16) for m in range(8)])
_MAG[127] = np.nan


def ckpt_value(codes, scales):
    """The numbers a checkpoint stands for, float64."""
    v = _MAG[codes & 127] * np.where(codes & 128, -1.0, 1.0)
    s = np.where(scales == 255, np.nan, np.exp2(scales.astype(np.float64) - 127.0))
    return v * np.repeat(s, 128, axis=1)


def ckpt_pack(x):
    """Codes and scales of x [T, K] (float values of bf16 numbers)."""
    T, K = x.shape
    with np.errstate(invalid="ignore"):          # (signalling NaNs)
        b = x.astype(np.float64).reshape(T, K // 128, 128)
    fin = np.isfinite(b)
    a = np.where(fin, np.abs(b), 0.0).max(axis=2)
    e = np.full(a.shape, -127, int)
    for _ in range(400):
        low = a > 448.0 * np.exp2(e)
        if not low.any():
            break
        e = e + low
    v = np.where(fin, b, 0.0) / np.exp2(e)[:, :, None]
    v = np.where((e == 120)[:, :, None], np.clip(v, -240, 240), v)
    # nearest magnitude of the table, ties to the even code
    mags = _MAG[:127]
    m = np.abs(v)
    hi = np.searchsorted(mags, m).clip(0, 126)
    lo = np.maximum(hi - 1, 0)
    dl, dh = m - mags[lo], mags[hi] - m
    c = np.where(dl < dh, lo, np.where(dh < dl, hi, np.where(lo % 2 == 0, lo, hi)))
    c = np.where(m == mags[hi], hi, c)
    c = c + np.where(np.signbit(v), 128, 0)
    c = np.where(fin, c, 127)
    return c.reshape(T, K).astype(np.uint8), (e + 127).astype(np.uint8)


def swiglu_backward(g, u, dh):
    """dg, du, h and |g|-weighted sizes of dg's two terms."""
    g, u, dh = (a.astype(np.float64) for a in (g, u, dh))
    with np.errstate(over="ignore"):
        e = np.exp(-np.abs(g))
        s = np.where(g >= 0, 1 / (1 + e), e / (1 + e))
    q = np.where(g >= 0, e / (1 + e), 1 / (1 + e))
    return dh * u * (s + g * s * q), dh * g * s, g * s * u, np.abs(dh * u) * (s + np.abs(g) * s * q)
