"""Plain 64-bit forms of the operators between routing and combine, written
from their definitions with numpy, for the tests to compare with: MXFP4
(OCP Microscaling Formats specification v1.0), the experts' products and the
balance loss with its gradient."""
from __future__ import annotations

import numpy as np

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
E2M1 = np.concatenate([E2M1, -E2M1])


def e2m1_codes(v) -> np.ndarray:
    """Codes of the E2M1 values nearest to v (ties to the even code,
    saturated), by search over the magnitudes."""
    v = np.asarray(v, np.float64)
    mids = (E2M1[1:8] + E2M1[:7]) / 2
    a = np.abs(v)
    low = np.searchsorted(mids, a, side="left")     # a tie stays below
    high = np.searchsorted(mids, a, side="right")   # a tie goes above
    code = np.where(low % 2 == 0, low, high)
    return (code + 8 * np.signbit(v)).astype(np.uint8)


def pack(codes) -> np.ndarray:
    codes = np.asarray(codes, np.uint8)
    return (codes[..., 0::2] | (codes[..., 1::2] << 4)).astype(np.uint8)


def unpack(packed) -> np.ndarray:
    packed = np.asarray(packed, np.uint8)
    return np.stack([packed & 15, packed >> 4], axis=-1).reshape(packed.shape[:-1] + (-1,))


def mx_scale(amax) -> np.ndarray:
    """E8M0 scale of a block whose largest magnitude is amax (finite)."""
    amax = np.asarray(amax, np.float64)
    _, e = np.frexp(amax)                            # amax = f 2^e, f in [0.5, 1)
    return np.where(amax > 0, np.clip(e - 1 - 2, -127, 127) + 127, 0).astype(np.uint8)


def mx_quantize(x):
    """(packed codes, scales) of x [..., cols]."""
    x = np.asarray(x, np.float64)
    b = x.reshape(x.shape[:-1] + (-1, 32))
    bad = ~np.isfinite(b).all(-1)
    with np.errstate(invalid="ignore"):
        amax = np.where(bad, 0.0, np.abs(b).max(-1))
    s = mx_scale(amax)
    v = np.where(bad[..., None], 0.0, b) * 2.0 ** (127.0 - s[..., None])
    codes = np.where(bad[..., None], 0, e2m1_codes(v)).reshape(x.shape)
    return pack(codes), np.where(bad, 255, s).astype(np.uint8)


def mx_values(packed, scales) -> np.ndarray:
    scales = np.asarray(scales)
    s = np.where(scales == 255, np.nan, 2.0 ** (scales.astype(np.float64) - 127))
    return E2M1[unpack(packed)] * np.repeat(s, 32, axis=-1)


def e4m3_values(codes) -> np.ndarray:
    c = np.asarray(codes, np.uint8).astype(np.int64)
    e, m = (c >> 3) & 15, c & 7
    v = np.where(e == 0, m / 8.0 * 2.0 ** -6, (1 + m / 8.0) * 2.0 ** (e - 7.0))
    v = np.where((e == 15) & (m == 7), np.nan, v)
    return np.where(c & 128, -v, v)


def fp8_values(codes, scales) -> np.ndarray:
    return e4m3_values(codes) * np.repeat(np.asarray(scales, np.float64), 128, axis=-1)


def product(x, w, owner):
    """(x[r] . w[owner[r]], and the same of the magnitudes) for rows with an
    owner >= 0; zero rows elsewhere."""
    y = np.zeros((x.shape[0], w.shape[1]))
    mag = np.zeros_like(y)
    for e in np.unique(owner[owner >= 0]):
        r = owner == e
        y[r] = x[r] @ w[e].T
        mag[r] = np.abs(x[r]) @ np.abs(w[e]).T
    return y, mag


def sigmoid(x) -> np.ndarray:
    x = np.asarray(x, np.float64)
    with np.errstate(over="ignore"):
        return 1 / (1 + np.exp(-x))


def balance(logits, idx, seq, mask, k):
    """loss [S], count [S, E], ntok [S], prob [S, E]."""
    T, E = logits.shape
    S = len(seq) - 1
    loss, count, ntok, prob = np.zeros(S), np.zeros((S, E), np.int64), np.zeros(S, np.int64), np.zeros((S, E))
    for s in range(S):
        t = [i for i in range(seq[s], seq[s + 1]) if mask[i]]
        n = ntok[s] = len(t)
        if not n:
            continue
        sc = sigmoid(logits[t])
        z = sc.sum(1, keepdims=True)
        prob[s] = (sc / np.where(z == 0, 1, z)).sum(0) / n
        picks = idx[t].ravel()
        picks = picks[(picks >= 0) & (picks < E)]
        count[s] = np.bincount(picks, minlength=E)
        loss[s] = (E * count[s] / (k * n) * prob[s]).sum()
    return loss, count, ntok, prob


def balance_grad(logits, count, ntok, seq, mask, k, grad_loss):
    """(gradient [T, E], its scale: the size of the terms that cancel in it)."""
    T, E = logits.shape
    g, size = np.zeros((T, E)), np.zeros((T, E))
    for s in range(len(seq) - 1):
        n = ntok[s]
        for t in range(seq[s], seq[s + 1]):
            if not mask[t] or not n:
                continue
            c = E * count[s] / (k * n * n)
            sc, rest = sigmoid(logits[t]), sigmoid(-logits[t])
            z = sc.sum()
            if z == 0:
                continue
            p = sc / z
            m = (c * p).sum()
            g[t] = grad_loss[s] * (c - m) * p * rest
            size[t] = np.abs(grad_loss[s]) * (c + m) * p * rest
    return g, size
