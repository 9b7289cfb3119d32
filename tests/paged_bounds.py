"""How far attention over 16-bit keys and values may be from its definition in 64 bits where the scores themselves come without rounding,
and inputs of that kind: sums of products that are whole multiples of a power of two and fit 24 bits, in whatever order they are added.

What is left is counted one by one (a rounding of fp32 is off by at most 2^-24 of its value, the exponential by 2^-22):
  the exponent    scale * log2(e) and its product with a score's distance from the maximum in use are off by at most 2^-22 of the
                  distance, and where parts or earlier sums are brought to a later maximum by as much of its distance, which is at
                  most that of the row's own maximum and 24 more
  the weight      the exponential, at most four times; and its rounding to the type: 2^-bits of it for one number, the square of that
                  for two, and in fp16, whose weights are held times 2^3, 2^-28 of the largest weight for what lies below its numbers
  the sums        n / 8 + 32 steps one after another at most (two products of 16 keys, then parts), off by 2^-22 each: tensor cores
                  cut off
  the output      its division, and half a step of the type"""
import numpy as np

BITS = {"bf16": 8, "fp16": 11}
LEAST = {"bf16": 2.0 ** -134, "fp16": 2.0 ** -25}      # half of the type's smallest number


def half_step(x, t):
    """Half the distance of the type's numbers at |x|."""
    x = np.maximum(np.abs(x), 2.0 ** -140)
    return np.maximum(2.0 ** (np.floor(np.log2(x)) - BITS[t]), LEAST[t])


def attend_exact(q, k, v, first, window, causal, scale, t, parts):
    """Attention of rows q [n][n_q][hd], the first of them at position `first`, over k, v [keys][n_kv][hd] (64 bits), and how far a kernel's
    may be from it whose weights are `parts` numbers of the type each."""
    n, n_q, hd = q.shape
    keys, g = k.shape[0], n_q // k.shape[1]
    out, tol = np.zeros(q.shape), np.zeros(q.shape)
    at = np.arange(keys)
    eps = 2.0 ** -(BITS[t] * parts)
    for m in range(n):
        p = first + m
        sees = at <= p if causal else at >= 0
        if window:
            sees = sees & (at > p - window if causal else at >= first - window)
        j = np.nonzero(sees)[0]
        for h in range(n_q):
            kk, vv = k[j, h // g], v[j, h // g]
            a = scale * (kk @ q[m, h])
            a -= a.max()
            w = np.exp(a)
            w /= w.sum()
            out[m, h] = w @ vv
            each = np.where(w > 0, w * (eps + 2.0 ** -22 * (np.maximum(a, -1e30) * -1 + 24 + 4)), 0) + w.max() * (2.0 ** -28 if t == "fp16" else 0)
            steps = (len(j) / 8 + 32) * 2.0 ** -22
            size = w @ np.abs(vv)
            off = each @ np.abs(vv) + each.sum() * np.abs(out[m, h]) + steps * (size + np.abs(out[m, h]))
            tol[m, h] = off + half_step(np.abs(out[m, h]) + off, t)
    return out, tol


def spiked(rng, n, n_q, n_kv, keys, hd, spikes=6):
    """Queries [n][n_q][hd], keys and values [keys][n_kv][hd] whose scores come without rounding: of each head some `spikes` keys among
    the first keys - n have nearly all weight, so that nothing averages a weight's rounding away. Values are positive."""
    u = rng.choice([-1.0, 1.0], (n_kv, hd))
    k = rng.integers(-1, 2, (keys, n_kv, hd)) / 8
    base = 10 / hd ** 0.5
    for h in range(n_kv):
        some = rng.choice(max(1, keys - n), min(spikes, max(1, keys - n)), replace=False)
        k[some, h] = u[h] * (np.ceil(base * 16) + rng.integers(0, 3, (len(some), 1))) / 16
    g = n_q // n_kv
    q = u[np.arange(n_q) // g] * (1 + rng.choice([0.0, 0.0, 0.0, 0.25, -0.25], (n, n_q, hd)))
    v = 0.5 + np.abs(rng.standard_normal((keys, n_kv, hd)))
    return q, k, v


def far(rng, n, n_q, n_kv, keys, hd, unit):
    """Scores that are whole multiples of `unit`, a few hundred of them: one-hot, or shared evenly by those that tie. Every number is a power of
    two times -2 .. 2."""
    a = 2.0 ** np.floor(np.log2(unit) / 2)
    q = a * rng.integers(-1, 2, (n, n_q, hd))
    k = unit / a * rng.integers(-2, 3, (keys, n_kv, hd))
    return q, k, rng.standard_normal((keys, n_kv, hd))


def lifted(rng, n, n_q, n_kv, keys, hd, lift):
    """Scores of a few units around `lift` (a power of four, 2^18 at most), which grow along the keys by more than a maximum in use may fall behind."""
    q, k = rng.integers(-2, 3, (n, n_q, hd)) / 2.0, rng.integers(-2, 3, (keys, n_kv, hd)) / 4.0
    q[..., 0], k[..., 0] = lift ** 0.5, lift ** 0.5
    q[..., 1], k[..., 1] = 64.0, (np.arange(keys) * 6 // keys)[:, None] * round(hd ** 0.5 * 0.625) / 2
    return q, k, rng.standard_normal((keys, n_kv, hd))
