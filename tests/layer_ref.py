"""Plain 64-bit forms of the operators around the balancer, in numpy: definitions only, no code of
the package.  8-bit values are decoded byte by byte from the e4m3 format."""
import numpy as np


def fp8_table():
    """The value of each e4m3 byte."""
    out = np.empty(256)
    for b in range(256):
        e, m = (b >> 3) & 15, b & 7
        v = np.nan if (e, m) == (15, 7) else m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        out[b] = -v if b & 128 else v
    return out


FP8 = fp8_table()
_LEVELS = np.array([FP8[b] for b in range(0x7F)])   # 0 .. 448, ascending with the byte


def round_fp8(v):
    """Finite |v| <= 448 to the nearest e4m3 value, ties to the even byte."""
    a = np.abs(v)
    hi = np.clip(np.searchsorted(_LEVELS, a), 1, len(_LEVELS) - 1)
    lo = hi - 1
    up, down = _LEVELS[hi] - a, a - _LEVELS[lo]
    pick = np.where(up < down, hi, np.where(down < up, lo, np.where(lo % 2 == 0, lo, hi)))
    return np.copysign(_LEVELS[pick], v)


def scale_exponent(amax):
    """The smallest e >= -126 with amax <= 448 * 2**e (e = -126 for 0)."""
    e = np.full(np.shape(amax), -126)
    for _ in range(300):
        e = np.where(amax > 448.0 * np.exp2(e.astype(float)), e + 1, e)
    return e


def quant_rows(x):
    """float64 [M][K] -> (values [M][K], exponents [M][blocks])."""
    M, K = x.shape
    kb = -(-K // 128)
    p = np.zeros((M, kb * 128))
    p[:, :K] = x
    p = p.reshape(M, kb, 128)
    e = scale_exponent(np.abs(p).max(axis=2))
    s = np.exp2(e.astype(float))[:, :, None]
    return (round_fp8(p / s) * s).reshape(M, kb * 128)[:, :K], e


def quant_blocks(w):
    """float64 [N][K] -> (values [N][K], exponents [blocks of N][blocks of K])."""
    N, K = w.shape
    nb, kb = -(-N // 128), -(-K // 128)
    p = np.zeros((nb * 128, kb * 128))
    p[:N, :K] = w
    p = p.reshape(nb, 128, kb, 128)
    e = scale_exponent(np.abs(p).max(axis=(1, 3)))
    s = np.exp2(e.astype(float))[:, None, :, None]
    return (round_fp8(p / s) * s).reshape(nb * 128, kb * 128)[:N, :K], e


def gate(logits, bias, k, groups, topk_groups, scale=1.0):
    """float arrays of the operator's input type's values -> (ids, weights), one token and one pick at a time."""
    T, E = logits.shape
    ids, w = np.full((T, k), -1, np.int32), np.zeros((T, k))
    for t in range(T):
        s = (logits[t].astype(np.float32) + (np.float32(0) if bias is None else bias.astype(np.float32)))
        s = np.where(np.isnan(s), -np.inf, s).astype(np.float64)
        if groups > 1:
            size = E // groups
            best = [max(s[g * size:(g + 1) * size]) for g in range(groups)]
            keep = sorted(range(groups), key=lambda g: (-best[g], g))[:topk_groups]
            for g in range(groups):
                if g not in keep:
                    s[g * size:(g + 1) * size] = -np.inf
        order = [e for e in sorted(range(E), key=lambda e: (-s[e], e)) if s[e] > -np.inf][:k]
        if not order:
            continue
        l = logits[t].astype(np.float64)[order]
        top = l.max()
        e = np.array([1.0 if v == top else np.exp(v - top) for v in l])
        ids[t, :len(order)] = order
        w[t, :len(order)] = scale * e / e.sum()
    return ids, w


def gate_backward(ids, weights, grad, E, scale=1.0):
    T, k = ids.shape
    out = np.zeros((T, E))
    for t in range(T):
        mean = (weights[t] * grad[t]).sum() / scale if scale else 0.0
        for j in range(k):
            if ids[t, j] >= 0:
                out[t, ids[t, j]] = weights[t, j] * (grad[t, j] - mean)
    return out


def silu(x):
    with np.errstate(over="ignore"):
        return x / (1 + np.exp(-x))


def layer(x, ids, weights, gate_w, up_w, down_w):
    """-> (out, the sum of the magnitudes that went into each output)."""
    T, H = x.shape
    out, mag = np.zeros((T, H)), np.zeros((T, H))
    for t in range(T):
        for j, e in enumerate(ids[t]):
            if e < 0:
                continue
            h = silu(gate_w[e] @ x[t]) * (up_w[e] @ x[t])
            out[t] += weights[t, j] * (down_w[e] @ h)
            mag[t] += abs(weights[t, j]) * (np.abs(down_w[e]) @ np.abs(h))
    return out, mag


def adamw(p, m, v, g, step, lr, beta1, beta2, eps, decay):
    """One step in float64."""
    m = beta1 * m + (1 - beta1) * g
    v = beta2 * v + (1 - beta2) * g * g
    p = p * (1 - lr * decay) - lr / (1 - beta1 ** step) * m / (np.sqrt(v / (1 - beta2 ** step)) + eps)
    return p, m, v
