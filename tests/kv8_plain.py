"""A plain model of the 8-bit key/value cache in 64 bits (numpy), one head of one sequence at a time: what the
calls of dfl_kv8 do, from their definitions."""
import numpy as np

BLOCK, TAIL = 32, 48


def quantise(x):
    """Codes (int, -127..127) and the fp32 scale of one block x [32, head_dim] (fp32)."""
    x = np.asarray(x, np.float32)
    if not np.isfinite(x).all():
        return np.zeros(x.shape, np.int64), np.float32("nan")
    scale = np.float32(np.abs(x).max() / np.float32(127))
    if scale == 0:
        return np.zeros(x.shape, np.int64), scale
    return np.clip(np.rint(x.astype(np.float64) / np.float64(scale)), -127, 127).astype(np.int64), scale


class Head:
    def __init__(self, n_blocks):
        self.n_blocks = n_blocks
        self.blocks = []                       # per sealed block: (k codes, k scale, v codes, v scale)
        self.tail_k, self.tail_v = [], []      # fp32 rows behind them
        self.score = np.zeros(n_blocks)

    def _cut(self, length):
        if length < BLOCK * len(self.blocks):
            z = length // BLOCK
            kc, ks, vc, vs = self.blocks[z]
            part = length - BLOCK * z
            self.tail_k = [r for r in (kc[:part].astype(np.float32) * ks)]
            self.tail_v = [r for r in (vc[:part].astype(np.float32) * vs)]
            self.blocks = self.blocks[:z]
        have = length - BLOCK * len(self.blocks)
        assert 0 <= have <= len(self.tail_k), "tokens that no call has written"
        self.tail_k, self.tail_v = self.tail_k[:have], self.tail_v[:have]

    def _seal(self):
        kc, ks = quantise(np.stack(self.tail_k[:BLOCK]))
        vc, vs = quantise(np.stack(self.tail_v[:BLOCK]))
        self.blocks.append((kc, ks, vc, vs))
        self.tail_k, self.tail_v = self.tail_k[BLOCK:], self.tail_v[BLOCK:]

    def write(self, length, k, v, commit):
        self._cut(length)
        if not commit:
            while len(self.tail_k) >= BLOCK:
                self._seal()
        for i, (rk, rv) in enumerate(zip(k, v)):
            self.tail_k.append(np.asarray(rk, np.float32))
            self.tail_v.append(np.asarray(rv, np.float32))
            if (length + i) % BLOCK == 0:
                self.score[(length + i) // BLOCK] = 0.0
        while commit and len(self.tail_k) >= BLOCK:
            self._seal()

    def rows(self, end):
        """Keys and values of the tokens below `end`, in 64 bits."""
        hd = (self.blocks[0][0].shape[1] if self.blocks else len(self.tail_k[0])) if self.blocks or self.tail_k else 0
        n = end - BLOCK * len(self.blocks)
        k = [c.astype(np.float64) * np.float64(s) for c, s, _, _ in self.blocks] + [np.asarray(self.tail_k[:n], np.float64).reshape(n, hd)]
        v = [c.astype(np.float64) * np.float64(s) for _, _, c, s in self.blocks] + [np.asarray(self.tail_v[:n], np.float64).reshape(n, hd)]
        return np.concatenate(k), np.concatenate(v)

    def attn(self, q, length, n, window, causal, scale):
        """q [rows, group, hd] of the rows that count: out, bound on an fp32 kernel's error, and row 0's block weights with their bound."""
        k, v = self.rows(length + n)
        out, bound = np.zeros(q.shape), np.zeros(q.shape)
        add, add_bound = np.zeros(self.n_blocks), np.zeros(self.n_blocks)
        hd = q.shape[-1]
        for m in range(n):
            lo, hi = 0, length + (m + 1 if causal else n)
            if window:
                lo = max(0, (length + m if causal else length - 1) - window + 1)
            x = q[m].astype(np.float64) @ k[lo:hi].T * scale
            p = np.exp(x - x.max(-1, keepdims=True))
            p /= p.sum(-1, keepdims=True)
            out[m] = p @ v[lo:hi]
            # A logit is off by at most hd + 8 roundings of 2^-24 and the two halves' 2^-21, relative to
            # scale * sum |q||k|; the exponential's argument carries that and its own 2 roundings. Weights are then off by e^(2 d) - 1 <=
            # 4 d each (numerator and sum, d < 1/4), the sums over n keys by n + 64 roundings.
            d = (np.abs(q[m]).astype(np.float64) @ np.abs(k[lo:hi]).T * abs(scale)).max(-1, keepdims=True) * ((hd + 16) * 2.0 ** -24 + 2.0 ** -21)
            rel = 4 * d + (hi - lo + 64) * 2.0 ** -23
            # A weight has no relative precision below the smallest numbers: fp32 holds multiples of 2^-149 (or nothing below
            # 2^-126), and the halves hold weights, at 2^7 or more for the row's largest, to 2^-25: 2^-32 of it.
            low = p.max(-1, keepdims=True) * 2.0 ** -32 + 2.0 ** -126
            bound[m] = rel * (p @ np.abs(v[lo:hi])) + low * np.abs(v[lo:hi]).sum(0) + 1e-30
            if m == 0:
                at = np.arange(lo, hi) // BLOCK
                np.add.at(add, at, p.sum(0))
                np.add.at(add_bound, at, (rel * p + 2.0 ** -126).sum(0))   # the scores' sums stay fp32
        return out, bound, add, add_bound

    def evict(self, keep, sink, recent):
        n = len(self.blocks)
        keep = min(keep, n)
        safe = {b for b in range(n) if b < sink or b >= n - recent}
        value = [-np.inf if np.isnan(x) else x for x in self.score]
        kept = sorted(sorted(range(n), key=lambda b: (b not in safe, -value[b], b))[:keep])
        score = np.zeros(self.n_blocks)
        score[:keep] = self.score[kept]
        tail = self.score[n:n + 2][:max(0, self.n_blocks - keep)]
        score[keep:keep + len(tail)] = tail
        self.blocks, self.score = [self.blocks[b] for b in kept], score
        return kept, n - keep
