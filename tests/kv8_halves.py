"""Inputs that show whether both fp16 halves of a query and of a weight take part in the attention over the 8-bit cache, and a
bound on its error that is far below what a missing half costs.

Every block's first key is `s` (a vector of signs), the others are `s` times a lower level, and a query is `s` times a number c: all
keys of a level have the same logit, so a half that is missing shows in all of them alike and does not average out."""
import numpy as np

from kv8_plain import BLOCK

CTX = 160
KINDS = ("weights", "queries")


def levels(kind):
    """What the keys behind a block's first are of it, as codes hold it: 64 and 95 of 127."""
    return 64 / 127 if kind == "weights" else 95 / 127


def inputs(kind, hd, heads, rows, seed):
    """k, v [CTX + rows, hd] and q [rows, heads, hd], fp32."""
    rng = np.random.default_rng(seed)
    s = rng.choice([-1.0, 1.0], hd)
    level = np.where(np.arange(CTX + rows) % BLOCK == 0, 1.0, levels(kind))
    if kind == "weights":
        # a weight of 2^7 at the first keys, and halfway between two fp16 numbers at the others: 64..128 is held in steps of 1/16
        w = 64 + (2 * rng.integers(200, 800, (rows, heads)) + 1) / 32
        c = np.log(128 / w) / (1 - levels(kind)) / np.sqrt(hd)
        v = rng.uniform(0.5, 1.0, (CTX + rows, hd))
    else:
        level = np.where(np.arange(CTX + rows) % 2 == 0, 1.0, levels(kind))
        # fp16 numbers of 1..2 are 2^-10 apart: the high half of c is off by 0.48 of that
        c = 0.5 * (1 + 0.48 * 2.0 ** -10 + rng.uniform(-0.01, 0.01, (rows, heads)) * 2.0 ** -10) * np.where(hd == 64, 2, 1)
        v = np.where(level[:, None] == 1.0, 1.0, -1.0) * rng.uniform(0.8, 1.0, (CTX + rows, hd))
    f = lambda x: x.astype(np.float32)  # noqa: E731
    return f(level[:, None] * s), f(v), f(c[..., None] * s)


def half(x):
    return x.astype(np.float16).astype(np.float64)


def attend(q, k, v, coded, drop=None):
    """One row in 64 bits: the output and its bound; `drop` leaves out the low halves of the "weights" or of the "queries" of the first
    `coded` tokens."""
    hd = len(q)
    q, k, v = (np.asarray(x, np.float64) for x in (q, k, v))
    if drop == "queries":
        f = 2.0 ** (14 - np.floor(np.log2(np.abs(q).max())))
        x = np.concatenate([k[:coded] @ (half(q * f) / f), k[coded:] @ q]) * hd ** -0.5
    else:
        x = k @ q * hd ** -0.5
    w = 2.0 ** 7 * np.exp(x - x.max())
    p = w / w.sum()
    used = np.concatenate([half(w[:coded]), w[coded:]]) / w.sum() if drop == "weights" else p
    out = used @ v
    # A logit is a sum of hd / 8 products of 16 (both halves) that grows evenly to the largest one, S; each cuts off less than 2^-20 of
    # what it has reached (16 addends, 2^-24 each): S (hd / 8 + 1) / 2 2^-20 in all. Two halves hold 22 bits, and scaling and the
    # exponent's argument take 6 roundings: 2^-22 + 6 2^-24 of S. Behind it: the exponential (2^-22) of numerator and sum, a weight's
    # halves (2^-22), four products of a block (2^-20 each), and some 24 sums and factors of parts (2^-23 each).
    S = np.abs(x).max()
    d = S * ((hd / 8 + 1) / 2 * 2.0 ** -20 + 2.0 ** -22 + 6 * 2.0 ** -24)
    tol = 2 * d * (p @ np.abs(v - p @ v)) + (3 * 2.0 ** -22 + 4 * 2.0 ** -20 + 24 * 2.0 ** -23) * (p @ np.abs(v))
    return out, tol
