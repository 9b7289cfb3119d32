"""A plain model of the paged key/value cache in 64 bits (numpy), from the definitions of the dfl_paged calls, and
how far a kernel's result may be from it."""
import numpy as np

BITS = {"bf16": 8, "fp16": 11}      # a rounding to the type is off by at most 2^-BITS of the value


class Plan:
    """Pages of sequences, planned in plain Python: lists for table, held and the ring of free pages."""

    def __init__(self, n_seq, n_pages, max_pages, page):
        self.P, self.N, self.most = page, n_pages, max_pages
        self.table = [[0] * max_pages for _ in range(n_seq)]
        self.held = [0] * n_seq
        self.ring = list(range(n_pages))            # the pages that no sequence has, in their order
        self.first = 0

    def step(self, length, n, rows):
        """(cu, slots, whether something did not fit) of a plan, whose state this takes on."""
        P, S = self.P, len(self.held)
        cu, fine = [0], []
        for i in range(S):
            ok = length[i] >= 0 and n[i] >= 0
            cu.append(cu[-1] + (int(n[i]) if ok else 0))
            fine.append(ok and length[i] + n[i] <= self.most * P and cu[-1] <= rows)
        want = [-(-(int(length[i]) + int(n[i])) // P) if fine[i] else self.held[i] for i in range(S)]
        for i in range(S):
            if fine[i]:
                self.ring += self.table[i][want[i]:self.held[i]]
        asked = used = 0
        got = []
        for i in range(S):
            need = max(0, want[i] - self.held[i])
            asked += need
            got.append(fine[i] and (need == 0 or asked <= len(self.ring)))
            if got[i] and need:
                self.table[i][self.held[i]:want[i]] = self.ring[asked - need:asked]
                used = asked
            if got[i]:
                self.held[i] = want[i]
        self.ring = self.ring[used:]
        self.first = (self.first + used) % self.N
        slots = np.full(rows, -1, np.int32)
        for i in range(S):
            if got[i]:
                pos = int(length[i]) + np.arange(cu[i + 1] - cu[i])
                slots[cu[i]:cu[i + 1]] = np.array(self.table[i])[pos // P] * P + pos % P
        return np.minimum(cu, rows).astype(np.int32), slots, not all(got)


def attend(q, k, v, first, window, causal, scale, bits, old=None):
    """Attention of rows q [n][n_q][hd], the first of them at position `first`, over k, v [keys][n_kv][hd] (all 64 bits): the outputs and how
    far a kernel's may be from them. `old`: tokens held before the rows (not causal: what `window` counts back from).

    The bound: scores are fp32 sums of hd products, each sum off by at most (hd + 8) 2^-23 of its terms' magnitudes (tensor cores
    truncate), and the subtraction of the maximum, the exponential and the sums of n weights add (n + 16) 2^-23; a weight is off by twice
    the scores' error, and once more by 2^-bits where it is rounded to the type; the output is rounded once."""
    n, n_q, hd = q.shape
    keys, n_kv = k.shape[0], k.shape[1]
    g = n_q // n_kv
    old = first if old is None else old
    out, tol = np.zeros(q.shape), np.zeros(q.shape)
    at = np.arange(keys)
    for m in range(n):
        p = first + m
        sees = at <= p if causal else at >= 0
        if window:
            sees = sees & (at > p - window if causal else at >= old - window)
        j = np.nonzero(sees)[0]
        for h in range(n_q):
            kk, vv = k[j, h // g], v[j, h // g]
            with np.errstate(invalid="ignore", over="ignore"):
                a = scale * (kk @ q[m, h])
                w = np.exp(a - a.max())
                w /= w.sum()
                out[m, h] = w @ vv
                size = scale * (np.abs(kk) @ np.abs(q[m, h])).max()
                off = 2 * (hd + 8) * 2.0 ** -23 * size + (len(j) + 16) * 2.0 ** -23 + 2.0 ** -bits
                tol[m, h] = off * (w @ np.abs(vv)) + 2.0 ** -bits * np.abs(out[m, h]) + 1e-7
    return out, tol
