"""The 8-bit key/value cache (dfl_kv8_*) on the GPU against its plain model in 64 bits."""
import numpy as np
import pytest

from kv8_plain import BLOCK, TAIL, Head, quantise

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from dflash_speculative_decode_gb300 import build
    build.build()
    return torch


class Pair:
    """A cache on the GPU and the plain heads beside it, driven with the same rows. The table is shuffled at the start, so logical and
    stored blocks differ; codes, scales and tails start as garbage (NaN where the type has it)."""

    def __init__(self, torch, n_seq, n_kv, hd, n_blocks, seed=0):
        from dflash_speculative_decode_gb300 import Kv8Cache
        self.torch, self.S, self.H, self.hd, self.nb = torch, n_seq, n_kv, hd, n_blocks
        self.rng = np.random.default_rng(seed)
        self.c = Kv8Cache.empty(n_seq, n_kv, hd, n_blocks)
        self.c.table.copy_(torch.from_numpy(np.stack([[self.rng.permutation(n_blocks) for _ in range(n_kv)] for _ in range(n_seq)]).astype(np.int32)))
        for t in (self.c.k_scale, self.c.v_scale, self.c.k_tail, self.c.v_tail):
            t.fill_(float("nan"))
        self.c.k.fill_(255)
        self.c.v.fill_(3)
        self.heads = [[Head(n_blocks) for _ in range(n_kv)] for _ in range(n_seq)]
        self.len = np.zeros(n_seq, np.int32)

    def dev(self, a):
        return self.torch.from_numpy(np.ascontiguousarray(a)).cuda()

    def new_rows(self, rows, heads=None):
        return (self.rng.standard_normal((self.S, rows, heads or self.H, self.hd)) * np.exp(0.5 * self.rng.standard_normal((1, 1, heads or self.H, self.hd)))).astype(np.float32)

    def write(self, rows, cnt=None, commit=True, k=None, v=None):
        k = self.new_rows(rows) if k is None else k
        v = self.new_rows(rows) if v is None else v
        n = np.full(self.S, rows, np.int32) if cnt is None else np.clip(np.asarray(cnt, np.int32), 0, rows)
        call = self.c.append if commit else self.c.stage
        call(self.dev(k), self.dev(v), self.dev(self.len), None if cnt is None else self.dev(np.asarray(cnt, np.int32)))
        self.c.status()
        for s in range(self.S):
            for h in range(self.H):
                self.heads[s][h].write(int(self.len[s]), k[s, :n[s], h], v[s, :n[s], h], commit)
        if commit:
            self.len = self.len + n
        return n

    def check_state(self):
        c = self.c
        sealed, table = c.sealed.cpu().numpy(), c.table.cpu().numpy()
        k, v = c.k.cpu().numpy(), c.v.cpu().numpy()
        ks, vs, kt, vt = (t.cpu().numpy() for t in (c.k_scale, c.v_scale, c.k_tail, c.v_tail))
        for s in range(self.S):
            for h in range(self.H):
                m = self.heads[s][h]
                assert sealed[s, h] == len(m.blocks)
                for b, (kc, ksc, vc, vsc) in enumerate(m.blocks):
                    at = table[s, h, b]
                    got_k = k[s, h, at].transpose(1, 0, 2).reshape(BLOCK, self.hd).astype(np.int64) - 128
                    got_v = v[s, h, at].T.astype(np.int64) - 128
                    np.testing.assert_array_equal(got_k, kc)
                    np.testing.assert_array_equal(got_v, vc)
                    np.testing.assert_array_equal([ks[s, h, at], vs[s, h, at]], [ksc, vsc])
                n = len(m.tail_k)
                if n:
                    np.testing.assert_array_equal(kt[s, h, :n], np.stack(m.tail_k))
                    np.testing.assert_array_equal(vt[s, h, :, :n].T, np.stack(m.tail_v))

    def attn(self, n_q, rows, cnt=None, window=0, causal=True, scale=None, score=False):
        q = self.new_rows(rows, n_q) * np.float32(1.5)
        out = self.torch.full(q.shape, -77.0, device="cuda")
        n = np.full(self.S, rows, np.int32) if cnt is None else np.clip(np.asarray(cnt, np.int32), 0, rows)
        before = None if self.c.score is None else self.c.score.cpu().numpy().astype(np.float64)
        self.c.attn(self.dev(q), self.dev(self.len), None if cnt is None else self.dev(np.asarray(cnt, np.int32)), window=window, causal=causal, scale=scale,
                    score=score, out=out)
        self.c.status()
        got, group = out.cpu().numpy(), n_q // self.H
        after = None if self.c.score is None else self.c.score.cpu().numpy().astype(np.float64)
        for s in range(self.S):
            assert (got[s, n[s]:] == -77.0).all(), "rows behind the last one were written"
            for h in range(self.H):
                hs = slice(h * group, (h + 1) * group)
                want, bound, add, add_bound = self.heads[s][h].attn(q[s, :n[s], hs], int(self.len[s]), int(n[s]), window, causal,
                                                                    self.hd ** -0.5 if scale is None else scale)
                if n[s]:
                    err = np.abs(got[s, :n[s], hs] - want)
                    assert (err <= bound[:n[s]]).all(), f"sequence {s} head {h}: off by {np.nanmax(err / bound):.3g} of the bound"
                if after is not None:
                    if not score:
                        np.testing.assert_array_equal(after[s, h], before[s, h])
                    else:
                        tol = add_bound + 2.0 ** -23 * (np.abs(before[s, h]) + add)
                        assert (np.abs(after[s, h] - before[s, h] - add) <= tol).all()
                        self.heads[s][h].score = after[s, h].copy()   # as they are held in fp32
        return q, got


# ---- rows in -----------------------------------------------------------------------------------------
@pytest.mark.parametrize("hd", [64, 128, 256])
@pytest.mark.parametrize("held,rows", [(0, 1), (0, 32), (0, 33), (0, 200), (31, 1), (31, 2), (32, 64), (47, 17), (5, 500)])
def test_append_seals_complete_blocks(torch, hd, held, rows):
    p = Pair(torch, 2, 2, hd, 24, seed=held * 7 + rows)
    if held:
        p.write(held)
    p.write(rows)
    p.check_state()


def test_append_ragged_counts(torch):
    p = Pair(torch, 5, 3, 64, 16, seed=3)
    p.write(70, cnt=[0, 1, 70, 32, 99])      # values outside 0..rows are limited to it
    p.write(40, cnt=[40, 31, -5, 0, 1])
    p.check_state()


@pytest.mark.parametrize("hd", [64, 128, 256])
def test_append_of_many_blocks(torch, hd):
    """Enough blocks that a CTA seals several, behind contexts that end inside a block, and cut back over what was sealed."""
    p = Pair(torch, 8, 8, hd, 24, seed=hd + 1)
    p.write(47, cnt=[0, 1, 31, 32, 33, 40, 47, 47])
    p.write(700, cnt=[700, 699, 64, 65, 0, 1, 700, 333])
    p.check_state()
    p.len = np.minimum(p.len, [600, 31, 64, 70, 20, 41, 97, 380]).astype(np.int32)
    p.write(620, cnt=[100, 620, 620, 33, 500, 0, 620, 31])
    p.check_state()


@pytest.mark.parametrize("hd", [64, 256])
def test_staged_rows_roll_back_and_seal_when_committed(torch, hd):
    """A walk of stages and commits of every size: blocks are sealed by the stage after the commit that completes them."""
    p = Pair(torch, 3, 2, hd, 12, seed=hd)
    rng = np.random.default_rng(1)
    p.write(20, cnt=[0, 20, 7])
    for _ in range(24):
        rows = int(rng.integers(1, 17))
        n = p.write(rows, cnt=rng.integers(0, rows + 1, 3), commit=False)
        p.check_state()
        p.len = p.len + rng.integers(0, n + 1).astype(np.int32)
    p.write(1, cnt=[0, 0, 0], commit=False)
    p.check_state()


@pytest.mark.parametrize("commit", [True, False])
def test_cut_back(torch, commit):
    """A len below what is sealed drops the tokens behind it; the rows of a cut block return as the values of their codes."""
    p = Pair(torch, 4, 2, 128, 12, seed=9)
    p.write(150)
    p.len = np.array([64, 65, 0, 95], np.int32)
    p.write(10, commit=commit)
    p.check_state()
    p.len = np.array([3, 33, 0, 64], np.int32)
    p.write(16 if not commit else 100, commit=commit)
    p.check_state()


def test_codes_of_hard_values(torch):
    """Values on the border of two codes and next to it, zeros, subnormal scales, and blocks with an infinity or a NaN."""
    p = Pair(torch, 1, 1, 64, 16, seed=0)
    rng = np.random.default_rng(5)
    k = np.zeros((1, 32 * 9, 1, 64), np.float32)
    for b in range(6):
        x = rng.standard_normal((32, 64)).astype(np.float32)
        top = np.float32([127.0, 1.0, 3.7, 1e30, 1e-36, 3e-44][b])
        scale = np.float32(top / np.float32(127))
        half = ((rng.integers(-127, 127, (32, 64)) + 0.5) * np.float64(scale)).astype(np.float32)
        x = np.select([rng.random((32, 64)) < 0.4, rng.random((32, 64)) < 0.5], [half, np.nextafter(half, np.float32(0))], np.clip(x, -1, 1) * top)
        x[0, 0] = top
        k[0, 32 * b:32 * b + 32, 0] = np.clip(x, -top, top)
    k[0, 32 * 7 + 3, 0, 5] = np.inf
    k[0, 32 * 8 + 31, 0, 63] = np.nan
    p.write(k.shape[1], k=k, v=k[:, ::-1].copy())
    p.check_state()
    assert np.isnan(p.heads[0][0].blocks[7][1]) and p.heads[0][0].blocks[6][1] == 0


def test_rows_of_a_wider_tensor(torch):
    """q, k and v as parts of one product's rows; the rows between them are not touched."""
    S, M, H, n_q, hd = 2, 6, 2, 4, 64
    p = Pair(torch, S, H, hd, 8, seed=2)
    p.write(40)
    qkv = p.rng.standard_normal((S, M, n_q + 2 * H, hd)).astype(np.float32)
    d = p.dev(qkv)
    length = p.dev(p.len)
    p.c.stage(d[:, :, n_q:n_q + H], d[:, :, n_q + H:], length)
    wide = torch.full((S, M, n_q + 3, hd), 5.0, device="cuda")
    p.c.attn(d[:, :, :n_q], length, out=wide[:, :, :n_q])
    p.c.status()
    same = torch.empty(S, M, n_q, hd, device="cuda")
    p.c.attn(d[:, :, :n_q].contiguous(), length, out=same)
    assert torch.equal(wide[:, :, :n_q], same) and (wide[:, :, n_q:] == 5.0).all()
    for s in range(S):
        for h in range(H):
            p.heads[s][h].write(int(p.len[s]), qkv[s, :, n_q + h], qkv[s, :, n_q + H + h], False)
            want, bound, _, _ = p.heads[s][h].attn(qkv[s, :, 2 * h:2 * h + 2], int(p.len[s]), M, 0, True, hd ** -0.5)
            assert (np.abs(same[s, :, 2 * h:2 * h + 2].cpu().numpy() - want) <= bound).all()


# ---- rows out ----------------------------------------------------------------------------------------
@pytest.mark.parametrize("hd", [64, 256])
def test_read(torch, hd):
    p = Pair(torch, 3, 2, hd, 8, seed=4)
    p.write(140, cnt=[140, 33, 0])
    first = np.array([30, 0, 0], np.int32)
    out = [torch.full((3, 90, 2, hd), -1.0, device="cuda") for _ in range(2)]
    p.c.read(p.dev(p.len), 90, first=p.dev(first), out=out)
    p.c.status()
    for s in range(3):
        n = max(0, min(90, int(p.len[s]) - int(first[s])))
        for x in out:
            assert (x[s, n:] == -1.0).all()
        for h in range(2):
            if n:
                for x, rows in zip(out, p.heads[s][h].rows(int(p.len[s]))):
                    np.testing.assert_array_equal(x[s, :n, h].cpu().numpy(), rows[first[s]:first[s] + n].astype(np.float32))


# ---- attention ---------------------------------------------------------------------------------------
@pytest.mark.parametrize("n_q,n_kv,hd", [(4, 1, 64), (4, 2, 64), (12, 1, 256), (12, 2, 256), (32, 16, 128), (32, 8, 128), (16, 1, 64), (5, 5, 128),
                                         (9, 3, 256)])
@pytest.mark.parametrize("rows,causal", [(1, True), (8, True), (16, True), (8, False)])
def test_attn_head_layouts(torch, n_q, n_kv, hd, rows, causal):
    p = Pair(torch, 2, n_kv, hd, 12, seed=n_q + rows)
    p.write(300, cnt=[300, 77])
    p.write(rows, commit=False)
    p.attn(n_q, rows, causal=causal, score=True)


@pytest.mark.parametrize("held", [0, 1, 15, 31, 32, 33, 63, 64, 100, 255, 256, 257, 511, 640, 1500])
@pytest.mark.parametrize("window", [0, 1, 31, 33, 250])
def test_attn_lengths_and_windows(torch, held, window):
    p = Pair(torch, 1, 2, 64, 64, seed=held + window)
    if held:
        p.write(held)
    for rows, causal in ((1, True), (7, True), (5, False)):
        p.write(rows, commit=False)
        p.attn(8, rows, window=window, causal=causal, score=True)


@pytest.mark.parametrize("hd", [64, 128, 256])
def test_attn_ragged_batch(torch, hd):
    """Sequences of many lengths in one call, some without rows, scores kept; NaN rows of the tail and unsealed blocks stay out of it."""
    p = Pair(torch, 6, 2, hd, 80, seed=hd)
    p.write(2000, cnt=[2000, 0, 1, 64, 777, 33])
    n = p.write(9, cnt=[9, 1, 0, 4, 9, 2], commit=False)
    p.attn(8, 9, cnt=n, score=True)
    p.attn(8, 9, cnt=n, window=100)
    p.attn(8, 9, cnt=n, window=40, causal=False, score=True)


@pytest.mark.parametrize("scale", [1.0, 0.0, 8.0, -0.5])
def test_attn_scales(torch, scale):
    """Large logits (one key takes all the weight), equal weights, and a negative scale."""
    p = Pair(torch, 1, 2, 128, 16, seed=11)
    p.write(333)
    p.write(6, commit=False)
    p.attn(4, 6, scale=scale, score=True)


def test_attn_values_of_very_different_size(torch):
    """Blocks whose scales differ by many orders, blocks of zeros, and queries of very different size."""
    p = Pair(torch, 1, 1, 64, 16, seed=12)
    k, v = p.new_rows(320), p.new_rows(320)
    size = np.repeat(10.0 ** np.array([0, -6, 4, -30, 0, 0, 2, -3, 0, -10]), 32).astype(np.float32)[None, :, None, None]
    v = v * size
    k[:, 32:64] = 0
    v[:, 128:160] = 0
    p.write(320, k=k, v=v)
    p.write(4, commit=False, k=p.new_rows(4) * np.float32(0.1), v=p.new_rows(4) * np.float32(1e-5))
    for q_size in (1.0, 1e-12, 30.0):
        p.attn(4, 4, scale=0.1 * q_size)


def test_attn_masked_infinities_do_not_leak(torch):
    """A block whose scale is NaN (it held an infinity) and a NaN row of the tail: rows that do not see them are as without them."""
    p = Pair(torch, 1, 1, 64, 16, seed=13)
    k, v = p.new_rows(200), p.new_rows(200)
    k[0, 40, 0, 3], v[0, 41, 0, 9] = np.inf, np.nan
    p.write(200, k=k, v=v)
    ks, vs = p.new_rows(8), p.new_rows(8)
    ks[0, 6], vs[0, 6] = np.nan, -np.inf
    p.write(8, commit=False, k=ks, v=vs)
    q = p.dev(p.new_rows(8, 4))
    length = p.dev(p.len)
    out = p.c.attn(q, length, window=136).cpu().numpy()      # row m sees tokens 65 + m .. 200 + m
    assert np.isfinite(out[0, :6]).all() and np.isnan(out[0, 6:]).all()
    out = p.c.attn(q, length, window=140).cpu().numpy()      # rows 0..2 see a token of the poisoned block (32..63)
    assert np.isnan(out[0, :3]).all() and np.isfinite(out[0, 3:6]).all()
    p.c.status()


@pytest.mark.parametrize("hd", [64, 128, 256])
@pytest.mark.parametrize("n_q,rows", [(2, 1), (4, 2), (8, 1), (2, 4)])
def test_attn_of_few_rows(torch, hd, n_q, rows):
    """At most 4 rows a key/value head, the two halves of a query in one tile of columns: hard values, queries, masks and scales."""
    p = Pair(torch, 2, 2, hd, 24, seed=hd + n_q)
    k, v = p.new_rows(700), p.new_rows(700)
    size = np.repeat(10.0 ** np.array([0, -6, 4, -30, 0, 0, 2, -3, 0, -10, 0]), 64)[:700].astype(np.float32)[None, :, None, None]
    p.write(700, cnt=[700, 333], k=k, v=v * size)
    p.write(rows, commit=False)
    p.attn(n_q, rows, score=True)
    p.attn(n_q, rows, window=100)
    p.attn(n_q, rows, causal=False, window=33, scale=2.0, score=True)
    p.attn(n_q, rows, scale=1e-9)
    p.attn(n_q, rows, cnt=[0, rows], score=True)


@pytest.mark.parametrize("hd", [64, 128, 256])
@pytest.mark.parametrize("seqs", [1, 90])
def test_few_rows_see_no_masked_infinities(torch, hd, seqs):
    """Blocks and tail rows that hold infinities or NaN: rows that see them are NaN, and the others as without them."""
    p = Pair(torch, seqs, 2, hd, 10, seed=hd)
    k, v = p.new_rows(200), p.new_rows(200)
    k[0, 40, 0, 3], v[0, 41, 1, 9] = np.inf, np.nan
    p.write(200, k=k, v=v)
    ks, vs = p.new_rows(4), p.new_rows(4)
    ks[0, 3, 0], vs[0, 3, 1] = np.nan, -np.inf
    p.write(4, commit=False, k=ks, v=vs)
    q, length = p.dev(p.new_rows(4, 2)), p.dev(p.len)
    q[0, 1, 1] = float("inf")
    out = p.c.attn(q, length, window=136).cpu().numpy()      # row m sees tokens 65 + m .. 200 + m
    p.c.status()
    assert np.isfinite(out[0, [0, 2]]).all() and np.isfinite(out[0, 1, 0]).all() and np.isnan(out[0, 1, 1]).all() and np.isnan(out[0, 3]).all()
    assert np.isfinite(out[1:]).all()
    out = p.c.attn(q, length, window=138).cpu().numpy()      # row 0 sees a token of the poisoned block (32..63)
    p.c.status()
    assert np.isnan(out[0, [0, 3]]).all() and np.isfinite(out[0, 2]).all() and np.isfinite(out[1:]).all()


def test_attn_long_and_far(torch):
    """A long context whose stored blocks lie past 2^31 bytes of the code arrays."""
    from dflash_speculative_decode_gb300 import Kv8Cache
    nb, hd = 150_000, 256
    p = Pair(torch, 1, 1, hd, 300, seed=14)
    far = Kv8Cache.empty(1, 2, hd, nb)
    far.table.copy_(torch.arange(nb - 1, -1, -1, dtype=torch.int32).expand(1, 2, nb))      # logical block 0 is the last one stored
    k, v = p.new_rows(9000), p.new_rows(9000)
    p.write(9000, k=k, v=v)
    two = lambda a: p.dev(np.concatenate([p.new_rows(a.shape[1]), a], 2))  # noqa: E731
    far.append(two(k), two(v), torch.zeros(1, dtype=torch.int32, device="cuda"))
    k, v = p.new_rows(8), p.new_rows(8)
    p.write(8, commit=False, k=k, v=v)
    far.stage(two(k), two(v), p.dev(p.len))
    q, got = p.attn(6, 8)
    other = far.attn(p.dev(np.concatenate([q, q], 2)), p.dev(p.len)).cpu().numpy()
    far.status()
    # the same head, whatever else the cache holds and wherever it is stored: within twice the bound of one call
    _, bound, _, _ = p.heads[0][0].attn(q[0], int(p.len[0]), 8, 0, True, hd ** -0.5)
    assert (np.abs(other[0, :, 6:] - got[0]) <= 2 * bound).all()


def test_attn_does_not_depend_on_the_batch(torch):
    """A sequence's rows and scores are the same bits alone and in a batch, and from call to call."""
    p = Pair(torch, 4, 2, 128, 40, seed=15)
    p.write(1000, cnt=[1000, 400, 3, 999])
    n = p.write(8, cnt=[8, 3, 8, 8], commit=False)
    q, length, cnt = p.dev(p.new_rows(8, 8)), p.dev(p.len), p.dev(n)
    p.c.score.zero_()
    a = p.c.attn(q, length, cnt, score=True)
    first = p.c.score.clone()
    p.c.score.zero_()
    assert torch.equal(p.c.attn(q, length, cnt, score=True), a) and torch.equal(p.c.score, first)
    only = p.dev(np.array([0, 0, 0, 8], np.int32))
    p.c.score.zero_()
    b = p.c.attn(q, length, only, score=True)
    assert torch.equal(b[3], a[3]) and torch.equal(p.c.score[3], first[3]) and (b[:3] == 0).all()


# ---- eviction ----------------------------------------------------------------------------------------
@pytest.mark.parametrize("held,keep,sink,recent", [(0, 4, 0, 0), (31, 0, 0, 0), (64, 1, 0, 0), (640, 8, 2, 3), (640, 5, 2, 3), (640, 0, 0, 0), (640, 20, 1, 1),
                                                   (640, 500, 9, 30), (655, 12, 0, 12), (1000, 13, 13, 0)])
def test_evict(torch, held, keep, sink, recent):
    p = Pair(torch, 2, 3, 64, 40, seed=held + keep)
    if held:
        p.write(held)
    score = np.round(np.exp(p.rng.standard_normal((2, 3, 40))), 1).astype(np.float32)     # with equal ones among them
    score[0, 0, 3], score[1, 2, 1], score[0, 1, :4] = np.nan, np.nan, -0.0
    p.c.score.copy_(torch.from_numpy(score))
    before = p.c.table.cpu().numpy()
    length = p.c.evict(p.dev(p.len), keep, sink=sink, recent=recent)
    p.c.status()
    table, got = p.c.table.cpu().numpy(), p.c.score.cpu().numpy()
    for s in range(2):
        for h in range(3):
            m = p.heads[s][h]
            m.score = score[s, h].astype(np.float64)
            n = len(m.blocks)
            kept, gone = m.evict(keep, sink, recent)
            free = [b for b in range(n) if b not in kept]
            np.testing.assert_array_equal(table[s, h], before[s, h][kept + free + list(range(n, 40))])
            np.testing.assert_array_equal(got[s, h], m.score.astype(np.float32))
            assert int(length[s]) == p.len[s] - BLOCK * gone
    p.len = length.cpu().numpy()
    p.check_state()


@pytest.mark.parametrize("blocks", [1023, 1024, 5000])
def test_evict_many_blocks(torch, blocks):
    """More blocks than threads, most of them with equal scores, negative and infinite ones among them."""
    from dflash_speculative_decode_gb300 import Kv8Cache
    c = Kv8Cache.empty(1, 2, 64, blocks + 1)
    rng = np.random.default_rng(blocks)
    score = rng.choice(np.float32([0.0, 1.0, 1.5, -2.0, np.inf, -np.inf, 1e-40]), (1, 2, blocks + 1))
    c.score.copy_(torch.from_numpy(score))
    c.sealed.fill_(blocks)
    length = torch.full((1,), 32 * blocks + 5, dtype=torch.int32, device="cuda")
    for keep in (17, blocks // 2, blocks - 1):
        to = c.evict(length, keep, sink=3, recent=9, out={"table": torch.empty_like(c.table), "score": torch.empty_like(c.score),
                                                          "sealed": torch.empty_like(c.sealed), "len": torch.empty_like(length)})
        c.status()
        for h in range(2):
            m = Head(blocks + 1)
            m.blocks, m.score = [None] * blocks, score[0, h].astype(np.float64)
            kept, gone = m.evict(keep, 3, 9)
            np.testing.assert_array_equal(to["table"][0, h, :keep].cpu().numpy(), kept)
            np.testing.assert_array_equal(np.sort(to["table"][0, h].cpu().numpy()), np.arange(blocks + 1))
            np.testing.assert_array_equal(to["score"][0, h].cpu().numpy(), m.score.astype(np.float32))
            assert int(to["len"]) == 32 * blocks + 5 - 32 * gone and int(to["sealed"][0, h]) == keep


# ---- all of them together ------------------------------------------------------------------------------
@pytest.mark.parametrize("n_q,n_kv,hd", [(4, 2, 64), (12, 1, 256), (32, 8, 128)])
def test_decode_with_eviction(torch, n_q, n_kv, hd):
    """A prompt, then steps of staged rows, attention with scores and commits of any number of rows, and evictions between them."""
    p = Pair(torch, 2, n_kv, hd, 20, seed=21)
    rng = np.random.default_rng(22)
    p.write(333, cnt=[333, 100])
    for step in range(14):
        n = p.write(8, cnt=[8, int(rng.integers(1, 9))], commit=False)
        p.attn(n_q, 8, cnt=n, score=True)
        p.len = p.len + rng.integers(1, n + 1).astype(np.int32)
        if step % 4 == 3:
            p.len = p.c.evict(p.dev(p.len), 5, sink=1, recent=2).cpu().numpy()
            p.c.status()
            for row in p.heads:
                for m in row:
                    m.evict(5, 1, 2)
    p.write(1, cnt=[0, 0], commit=False)
    p.check_state()
    np.testing.assert_array_equal(p.c.sealed.cpu().numpy(), p.len[:, None] // BLOCK * np.ones((1, n_kv), int))


def test_captured_steps(torch):
    """Two graphs of stage and attention, captured at one position and replayed at others, give the eager calls' bits."""
    p = Pair(torch, 2, 2, 64, 40, seed=23)
    p.write(500, cnt=[500, 37])
    k, v, q = p.dev(p.new_rows(4)), p.dev(p.new_rows(4)), p.dev(p.new_rows(4, 4))
    length = p.dev(p.len)
    outs = [torch.empty_like(q) for _ in range(2)]
    p.c.stage(k, v, length)
    p.c.attn(q, length, out=outs[0], score=True)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    graphs = []
    for out, score in zip(outs, (True, False)):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            p.c.stage(k, v, length)
            p.c.attn(q, length, out=out, score=score)
        graphs.append(g)
    for add in (0, 3, 4, 2):
        length += add
        p.c.score.zero_()
        for g in graphs:
            g.replay()
        got, sums = [o.clone() for o in outs], p.c.score.clone()
        p.c.score.zero_()
        p.c.stage(k, v, length)
        want = p.c.attn(q, length, score=True)
        assert torch.equal(got[0], want) and torch.equal(got[1], want) and torch.equal(sums, p.c.score)
    p.c.status()


def test_other_stream(torch):
    p = Pair(torch, 1, 2, 128, 16, seed=24)
    p.write(400)
    p.write(8, commit=False)
    q, length = p.dev(p.new_rows(8, 8)), p.dev(p.len)
    want = p.c.attn(q, length)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = p.c.attn(q, length)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want)


# ---- faults that the device meets -----------------------------------------------------------------------
def test_faults_are_reported_and_leave_the_sequence(torch):
    from dflash_speculative_decode_gb300 import DflError, _abi
    p = Pair(torch, 3, 1, 64, 4, seed=25)
    p.write(64)

    def code():
        with pytest.raises(DflError) as e:
            p.c.status()
        p.c.status()      # the word is cleared
        return e.value.code

    k = p.dev(p.new_rows(8))
    for lens, want in (([64, 125, 64], _abi.DFL_E_CAPACITY), ([64, -1, 64], _abi.DFL_E_CAPACITY), ([64, 64 + TAIL + 1, 64], _abi.DFL_E_STATE)):
        before = [t.clone() for t in (p.c.k, p.c.v, p.c.k_tail, p.c.v_tail, p.c.sealed)]
        length = p.dev(np.array(lens, np.int32))
        p.c.stage(k, k, length)
        assert code() == want
        for t, b in zip((p.c.k, p.c.v, p.c.k_tail, p.c.v_tail, p.c.sealed), before):
            assert t[1].equal(b[1]) or torch.equal(torch.nan_to_num(t[1].float()), torch.nan_to_num(b[1].float()))
        out = torch.full((3, 8, 2, 64), 9.0, device="cuda")
        p.c.attn(p.dev(p.new_rows(8, 2)), length, out=out)
        assert code() == want
        assert (out[1] == 9.0).all() and torch.isfinite(out).all() and (out[0] != 9.0).all() and (out[2] != 9.0).all()
    length = p.dev(p.len)
    p.c.stage(k, k, length)
    p.c.status()
    for bad in (4, -1, 1 << 30):
        keep = p.c.table.clone()
        p.c.table[1, 0, 1] = bad
        out = torch.full((3, 8, 2, 64), 9.0, device="cuda")
        p.c.attn(p.dev(p.new_rows(8, 2)), length, out=out)
        assert code() == _abi.DFL_E_INVALID_ARG
        assert (out[1] == 9.0).all() and (out[0] != 9.0).all() and (out[2] != 9.0).all()
        p.c.read(length, 64)
        assert code() == _abi.DFL_E_INVALID_ARG
        p.c.append(k.repeat(1, 8, 1, 1), k.repeat(1, 8, 1, 1), torch.zeros_like(length))     # seals over blocks 0 and 1
        assert code() == _abi.DFL_E_INVALID_ARG
        p.c.table.copy_(keep)
        p.c.append(k.repeat(1, 8, 1, 1), k.repeat(1, 8, 1, 1), torch.zeros_like(length))
        p.c.stage(k, k, length)
        p.c.status()
    p.c.sealed[2, 0] = 5
    p.c.attn(p.dev(p.new_rows(8, 2)), length)
    assert code() == _abi.DFL_E_INVALID_ARG


def test_quantisation_error_is_half_a_step(torch):
    """Values read back are within scale / 2 (and the product's rounding) of the rows appended."""
    p = Pair(torch, 1, 2, 128, 8, seed=26)
    k, v = p.new_rows(256), p.new_rows(256)
    p.write(256, k=k, v=v)
    got = p.c.read(p.dev(p.len), 256)
    for x, rows in zip(got, (k, v)):
        for b in range(8):
            for h in range(2):
                want = rows[0, 32 * b:32 * b + 32, h].astype(np.float64)
                scale = np.float64(quantise(rows[0, 32 * b:32 * b + 32, h])[1])
                err = np.abs(x[0, 32 * b:32 * b + 32, h].cpu().numpy() - want)
                assert (err <= scale / 2 + 127 * scale * 2.0 ** -24).all()


# ---- more units than CTAs: the work is shared out evenly -----------------------------------------------------
@pytest.mark.parametrize("S,n_kv,n_q,hd,rows,held", [(40, 4, 8, 64, 1, 900), (21, 8, 32, 128, 3, 400), (40, 2, 24, 256, 2, 300), (52, 3, 9, 64, 16, 260),
                                                     (170, 1, 4, 64, 2, 90), (77, 2, 2, 256, 1, 150)])
def test_attn_of_many_sequences(torch, S, n_kv, n_q, hd, rows, held):
    """Sequences of very different lengths, some without rows or tokens: full and windowed, causal and not, with scores and without."""
    p = Pair(torch, S, n_kv, hd, held // BLOCK + 2, seed=S)
    cnt = p.rng.integers(0, held + 1, S)
    cnt[::5], cnt[1], cnt[-1] = 0, held, held
    p.write(held, cnt=cnt)
    n = p.rng.integers(0, rows + 1, S)
    n[-3:] = rows
    p.write(rows, cnt=n, commit=False)
    p.attn(n_q, rows, cnt=n, score=True)
    p.attn(n_q, rows, cnt=n, window=70, score=True)
    p.attn(n_q, rows, cnt=n, window=33, causal=False)


@pytest.mark.parametrize("S,n_kv,n_q,hd,rows,blocks", [(16, 8, 32, 64, 3, 514), (32, 2, 12, 256, 2, 514)])
def test_attn_shared_out_by_capacity(torch, S, n_kv, n_q, hd, rows, blocks):
    """Fewer units, but a capacity so long that whole splits would leave CTAs idle; the sequences themselves are short, and one is long."""
    p = Pair(torch, S, n_kv, hd, blocks, seed=S)
    cnt = p.rng.integers(0, 200, S)
    cnt[[0, 3, S - 1]] = 1300, 0, 31
    p.write(1300, cnt=cnt)
    n = p.rng.integers(0, rows + 1, S)
    n[[0, 3, S - 1]] = rows
    p.write(rows, cnt=n, commit=False)
    p.attn(n_q, rows, cnt=n, score=True)
    p.attn(n_q, rows, cnt=n, causal=False)


def test_attn_of_more_sequences_than_threads(torch):
    """700 sequences, a few of which have rows: the first, the last, and some on either side of 256 and 512."""
    p = Pair(torch, 700, 1, 64, 6, seed=31)
    n = np.zeros(700, np.int32)
    n[[0, 1, 255, 256, 400, 511, 512, 513, 699]] = [3, 2, 1, 3, 2, 1, 3, 2, 1]
    p.write(150, cnt=np.where(n > 0, 150 - 17 * n, 0))
    p.write(3, cnt=n, commit=False)
    p.attn(4, 3, cnt=n, score=True)
    p.attn(4, 3, cnt=np.zeros(700, np.int32), score=True)      # nothing to do at all


def test_many_sequences_give_the_same_bits_each_time(torch):
    """Eagerly, and replayed from a graph with other counts of rows than it was captured with."""
    p = Pair(torch, 90, 2, 64, 30, seed=32)
    p.write(800, cnt=p.rng.integers(0, 801, 90))
    p.write(4, commit=False)
    q, length = p.dev(p.new_rows(4, 8)), p.dev(p.len)
    p.c.score.zero_()
    want, side = p.c.attn(q, length, score=True), torch.cuda.Stream()
    sums, out, g = p.c.score.clone(), torch.empty_like(want), torch.cuda.CUDAGraph()
    n = torch.zeros(90, dtype=torch.int32, device="cuda")
    with torch.cuda.graph(g, stream=side):
        p.c.attn(q, length, n, score=True, out=out)
    n.fill_(4)
    for _ in range(3):
        p.c.score.zero_()
        out.zero_()
        g.replay()
        assert torch.equal(out, want) and torch.equal(p.c.score, sums)
    p.c.status()


def test_faults_among_many_sequences(torch):
    """A bad length, table entry or count concerns its own sequence (or head) only."""
    from dflash_speculative_decode_gb300 import DflError, _abi
    S = 80
    p = Pair(torch, S, 2, 64, 8, seed=33)
    p.write(200, cnt=p.rng.integers(64, 201, S))
    p.write(2, commit=False)
    q = p.dev(p.new_rows(2, 4))
    good = p.c.attn(q, p.dev(p.len))
    p.c.status()

    def check(bad, code, length=None):
        out = torch.full_like(q, 9.0)
        p.c.attn(q, p.dev(p.len) if length is None else length, out=out)
        with pytest.raises(DflError) as e:
            p.c.status()
        assert e.value.code == code
        for s in range(S):
            for h in range(2):
                x, want = out[s, :, 2 * h:2 * h + 2], good[s, :, 2 * h:2 * h + 2]
                if (s, h) in bad:
                    assert (x == 9.0).all()
                else:           # other cuts than before: the same numbers to a few roundings of fp32 sums of values below 16
                    assert (x - want).abs().max() < 2e-5
    length = p.dev(p.len)
    length[3], length[40] = -1, 31
    check({(3, 0), (3, 1), (40, 0), (40, 1)}, _abi.DFL_E_STATE, length)
    keep = p.c.table.clone()
    p.c.table[7, 1, 0] = 8
    p.c.table[79, 0, 1] = -1
    check({(7, 1), (79, 0)}, _abi.DFL_E_INVALID_ARG)
    p.c.table.copy_(keep)
    p.c.sealed[11, 1] = 1 if int(p.c.sealed[11, 1]) != 1 else 0
    check({(11, 1)}, _abi.DFL_E_STATE)


# ---- eviction's faults, and its place in graphs ---------------------------------------------------------------
def test_eviction_of_a_sequence_out_of_order_keeps_it(torch):
    from dflash_speculative_decode_gb300 import DflError, _abi
    p = Pair(torch, 4, 2, 64, 12, seed=34)
    p.write(300)
    p.c.score.copy_(p.dev(p.rng.random((4, 2, 12)).astype(np.float32)))
    for change, code in ((dict(len=287), _abi.DFL_E_STATE), (dict(len=9 * 32 + TAIL + 1), _abi.DFL_E_STATE), (dict(sealed=8), _abi.DFL_E_STATE),
                         (dict(sealed=13), _abi.DFL_E_INVALID_ARG), (dict(sealed=-1), _abi.DFL_E_INVALID_ARG)):
        length, sealed = p.dev(p.len), p.c.sealed.clone()
        if "len" in change:
            length[2] = change["len"]
        else:
            p.c.sealed[2, 1] = change["sealed"]
        to = {"table": torch.full_like(p.c.table, -5), "score": torch.full_like(p.c.score, -5), "sealed": torch.full_like(sealed, -5), "len": torch.full_like(length, -5)}
        p.c.evict(length, 4, sink=1, recent=1, out=to)
        with pytest.raises(DflError) as e:
            p.c.status()
        assert e.value.code == code
        assert all(torch.equal(to[name][2], getattr(p.c, name)[2]) for name in ("table", "score", "sealed")) and int(to["len"][2]) == int(length[2])
        assert to["len"][[0, 1, 3]].tolist() == [300 - 5 * 32] * 3 and (to["sealed"][[0, 1, 3]] == 4).all()
        p.c.sealed.copy_(sealed)


def test_eviction_in_place_keeps_graphs_valid(torch):
    """A graph captured before evictions attends over what they leave, and an eviction can itself be captured."""
    p = Pair(torch, 2, 2, 64, 20, seed=35)
    p.write(500)
    p.write(3, commit=False)
    q, length = p.dev(p.new_rows(3, 4)), p.dev(p.len)
    out, side, g, ge = torch.empty_like(q), torch.cuda.Stream(), torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    p.c.attn(q, length, out=out, score=True)
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=side):
        p.c.attn(q, length, out=out, score=True)
    with torch.cuda.graph(ge, stream=side):
        length.copy_(p.c.evict(length, 6, sink=1, recent=2))
    for keep, evict in ((10, lambda: length.copy_(p.c.evict(length, 10, sink=1, recent=2))), (6, ge.replay)):
        for s in range(2):
            for h in range(2):
                p.heads[s][h].score = p.c.score[s, h].cpu().numpy().astype(np.float64)
                p.heads[s][h].evict(keep, 1, 2)
        evict()
        p.c.status()
        p.len = length.cpu().numpy()
        p.check_state()
        g.replay()
        for s in range(2):
            for h in range(2):
                want, bound, _, _ = p.heads[s][h].attn(q[s, :, 2 * h:2 * h + 2].cpu().numpy(), int(p.len[s]), 3, 0, True, 0.125)
                assert (np.abs(out[s, :, 2 * h:2 * h + 2].cpu().numpy() - want) <= bound).all()
    p.c.status()


def test_memory_of_a_cache_used_on_another_stream_is_not_given_away(torch):
    """A cache is dropped while another stream still works on it: what is allocated next must not be written by that work."""
    p = Pair(torch, 1, 2, 128, 600, seed=36)
    p.write(19000)
    p.write(8, commit=False)
    q, length, side = p.dev(p.new_rows(8, 8)), p.dev(p.len), torch.cuda.Stream()
    want = p.c.attn(q, length)
    c, p.c = p.c, None
    side.wait_stream(torch.cuda.current_stream())
    out = torch.empty_like(q)
    with torch.cuda.stream(side):
        for _ in range(200):
            c.attn(q, length, out=out)
    sizes = [t.numel() * t.element_size() for t in (c.k, c.v, c.table, c._scratch)]
    del c
    taken = [torch.zeros(n, dtype=torch.uint8, device="cuda") for n in sizes]
    side.synchronize()
    assert torch.equal(out, want) and all((t == 0).all() for t in taken)
