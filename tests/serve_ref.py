"""Plain 64-bit forms of the cache append, the paged attention and the
adapters (numpy, CPU), written from the formulas in tq.h, and the error bounds
that the tests use."""
import numpy as np
import torch

E4M3_LEVELS = None


def round_e4m3(x):
    """Nearest e4m3 value, ties to the even pattern, saturating."""
    global E4M3_LEVELS
    if E4M3_LEVELS is None:
        lv = []
        for bits in range(127):  # positive finite patterns in order
            e, f = bits >> 3, bits & 7
            lv.append(f * 2.0 ** -9 if e == 0 else (8 + f) * 2.0 ** (e - 10))
        E4M3_LEVELS = np.array(lv)
    a = np.minimum(np.abs(x), 448.0)
    hi = np.clip(np.searchsorted(E4M3_LEVELS, a), 1, 126)
    lo = hi - 1
    dl, dh = a - E4M3_LEVELS[lo], E4M3_LEVELS[hi] - a
    pick = np.where(dl < dh, lo, np.where(dh < dl, hi, np.where(lo % 2 == 0, lo, hi)))
    return np.copysign(E4M3_LEVELS[pick], x)


def rotate(x, pos, freq, interleaved):
    """x [heads][d] of one token in float64."""
    half = len(freq)
    i = np.arange(half)
    lo, hi = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    c, s = np.cos(pos * freq), np.sin(pos * freq)
    out = x.copy()
    out[:, lo] = x[:, lo] * c - x[:, hi] * s
    out[:, hi] = x[:, lo] * s + x[:, hi] * c
    return out


def rotation_size(x, half, interleaved):
    """|a| + |b| of each feature's pair (0 for features that are not rotated)."""
    i = np.arange(half)
    lo, hi = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    out = np.zeros_like(x)
    out[..., lo] = out[..., hi] = np.abs(x[..., lo]) + np.abs(x[..., hi])
    return out


def attention(q, k, v, scale):
    """q [g][d], k and v [n][d] float64 -> out [g][d], and sum_j p_j |v_j| and
    max_j scale sum |q||k_j| for the bounds."""
    if len(k) == 0:
        return np.zeros_like(q), np.zeros_like(q), 0.0
    s = scale * (q @ k.T)
    p = np.exp(s - s.max(axis=1, keepdims=True))
    p /= p.sum(axis=1, keepdims=True)
    return p @ v, p @ np.abs(v), float((abs(scale) * (np.abs(q) @ np.abs(k).T)).max())


def attention_bound(out, size, score, n, vmax, out_t, cache_t):
    """Error bound of one head's outputs.  Output rounding: eps/2 of its
    value.  Weights: a score is a binary32 sum of exact products (d/16 + 8
    steps of at most 2^-23 of sum |q||k|), so exp moves by that much, plus
    2^-20 for the exponential and the running sums; a weight is rounded to
    fp16 (2^-12) for fp16 and e4m3 caches, with a floor of 2^-25 of the
    largest weight, and to two bf16 terms (2^-17) for bf16 caches."""
    d = out.shape[-1]
    rel = 2 * score * (d / 16 + 8) * 2.0 ** -23 + 2.0 ** -20 + (2.0 ** -16 if cache_t == torch.bfloat16 else 2.0 ** -11)
    tiny = n * 2.0 ** -25 * vmax if cache_t != torch.bfloat16 else 0.0
    half_ulp = torch.finfo(out_t).eps / 2 * (1 + 2.0 ** -10)
    floor = 2.0 ** -25 if out_t == torch.float16 else 0.0  # half a subnormal step
    return half_ulp * np.abs(out) + size * rel + tiny + floor


def lora(x, a, b, scale, ids, y):
    """Outputs and error bounds in float64.  A x: exact products, binary32
    sums of k/16 + 32 steps (2^-23 each, truncation included); the second
    product keeps A x to 2^-22 and sums rank/16 + 8 such steps; one rounding
    each for the scale and the final sum."""
    want = y.copy()
    bound = np.abs(y) * 2.0 ** -24
    for t, ad in enumerate(ids):
        if ad < 0 or ad >= len(a):
            bound[t] = 0.0
            continue
        d = scale[ad] * (b[ad] @ (a[ad] @ x[t]))
        size = abs(scale[ad]) * (np.abs(b[ad]) @ (np.abs(a[ad]) @ np.abs(x[t])))
        want[t] += d
        steps = x.shape[1] / 16 + 32 + a.shape[1] / 16 + 8 + 4
        bound[t] += size * steps * 2.0 ** -23 + np.abs(d) * 2.0 ** -22
    return want, bound + np.abs(want) * 2.0 ** -24
