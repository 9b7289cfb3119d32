"""The paged key/value cache (dfl_paged_*) on the GPU against its plain model in 64 bits."""
import numpy as np
import pytest

from paged_plain import BITS, Plan, attend

pytestmark = pytest.mark.gpu

# query heads, key/value heads, head dimension
HEADS = [(4, 1, 64), (4, 2, 64), (2, 2, 64), (7, 1, 64), (6, 2, 128), (32, 16, 128), (16, 1, 128), (12, 1, 256), (12, 2, 256), (3, 3, 256)]


@pytest.fixture(scope="module")
def torch():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from dflash_speculative_decode_gb300 import build
    build.build()
    return torch


def dtype_of(torch, t):
    return {"bf16": torch.bfloat16, "fp16": torch.float16}[t]


def i32(torch, v):
    return torch.tensor(np.asarray(v, np.int32), device="cuda")


def cache(torch, n_seq, n_kv, hd, n_pages=4, most=4, page=16, t="bf16"):
    from dflash_speculative_decode_gb300 import PagedCache
    c = PagedCache.empty(n_seq, n_kv, hd, n_pages, most, page, dtype_of(torch, t))
    c.k.fill_(float("nan"))
    c.v.fill_(float("nan"))
    return c


def rows_of(torch, rng, n, heads, hd, t, gain=1.0):
    """Rows of the type, and the same in 64 bits."""
    x = torch.from_numpy((rng.standard_normal((n, heads, hd)) * gain * np.exp(0.4 * rng.standard_normal((1, heads, hd)))).astype(np.float32)).to(dtype_of(torch, t))
    return x.cuda(), x.double().numpy()


def back(x):
    return x.double().cpu().numpy()


def near(got, want, tol):
    np.testing.assert_array_equal(np.isnan(got), np.isnan(want))
    bad = ~(np.abs(got - want) <= tol) & ~np.isnan(want)
    assert not bad.any(), (np.argwhere(bad)[:5], got[bad][:5], want[bad][:5], tol[bad][:5])


# ---- plans -------------------------------------------------------------------------------------------
def same_plan(c, p):
    S, N = c.n_seq, c.n_pages
    assert c.held.tolist() == p.held
    first, count, a, b = c.queue.tolist()
    assert (first, count, a, b) == (p.first, len(p.ring), 0, 0)
    ring = c.free.tolist()
    assert [ring[(first + i) % N] for i in range(count)] == p.ring
    for s in range(S):
        assert c.table[s, :p.held[s]].tolist() == p.table[s][:p.held[s]]


@pytest.mark.parametrize("n_seq,n_pages,most,page,rows", [
    (1, 1, 1, 16, 5), (1, 40, 40, 16, 700), (3, 20, 8, 32, 300), (7, 64, 30, 64, 2100), (100, 300, 9, 16, 1500), (513, 4000, 40, 128, 9000), (4096, 9000, 6, 16, 30000)])
def test_plans_of_many_steps(torch, n_seq, n_pages, most, page, rows):
    rng = np.random.default_rng(n_seq)
    c, p = cache(torch, n_seq, 1, 64, n_pages, most, page), Plan(n_seq, n_pages, most, page)
    length = np.zeros(n_seq, np.int64)
    cu, slots = i32(torch, [-5] * (n_seq + 1)), i32(torch, [-5] * rows)
    short = False
    for step in range(12):
        gone = rng.random(n_seq) < 0.3
        length = np.where(gone, 0, length)
        per = max(1, int(rows * [0.3, 1.2, 0.7][step % 3] / n_seq))
        n = np.where(gone & (rng.random(n_seq) < 0.5), 0, rng.integers(0, 2 * per + 1, n_seq))
        c.plan(i32(torch, length), i32(torch, n), out=(cu, slots))
        want_cu, want_slots, some = p.step(length, n, rows)
        short |= some
        assert cu.tolist() == want_cu.tolist()
        np.testing.assert_array_equal(slots.cpu().numpy(), want_slots)
        same_plan(c, p)
        fits = np.array([-(-int(a + b) // page) <= h for a, b, h in zip(length, n, p.held)])
        length = np.where(fits, length + rng.integers(0, n + 1), length)     # some rows are rolled back
    if short:
        with pytest.raises(RuntimeError, match="DFL_E_CAPACITY"):
            c.status()
    c.status()


@pytest.mark.parametrize("n_seq,rows,shift", [(3, 40003, 0), (300, 50001, 1), (700, 33000, 2), (4096, 70000, 3)])
def test_plans_of_many_rows(torch, n_seq, rows, shift):
    """Slots that begin anywhere (shift: int32 numbers past a 16-byte boundary), two batches of prompts in turn."""
    rng = np.random.default_rng(n_seq)
    per = 2 * rows // n_seq
    n_pages = rows // 16 + n_seq
    c, p = cache(torch, n_seq, 1, 64, n_pages, -(-per // 16) + 1, 16), Plan(n_seq, n_pages, -(-per // 16) + 1, 16)
    cu, slots = i32(torch, [-5] * (n_seq + 1)), i32(torch, [-5] * (rows + 8))[shift:shift + rows]
    for step in range(4):
        n = np.where(np.arange(n_seq) % 2 == step % 2, rng.integers(0, per - per // 8, n_seq), 0)
        c.plan(i32(torch, np.zeros(n_seq)), i32(torch, n), out=(cu, slots))
        want_cu, want_slots, _ = p.step(np.zeros(n_seq, int), n, rows)
        assert cu.tolist() == want_cu.tolist()
        np.testing.assert_array_equal(slots.cpu().numpy(), want_slots)
        same_plan(c, p)
    try:
        c.status()
    except RuntimeError as e:
        assert "DFL_E_CAPACITY" in str(e)


def test_a_plan_that_frees_all_and_one_of_no_rows(torch):
    c, p = cache(torch, 3, 1, 64, 50, 20, 16), Plan(3, 50, 20, 16)
    for length, n, rows in (([0, 0, 0], [300, 200, 250], 750), ([0, 0, 0], [0, 0, 0], 0), ([0, 0, 0], [320, 320, 160], 800), ([5, 0, 319], [0, 0, 1], 1)):
        cu, slots = i32(torch, [7] * 4), i32(torch, [7] * rows)
        c.plan(i32(torch, length), i32(torch, n), out=(cu, slots))
        want_cu, want_slots, _ = p.step(length, n, rows)
        assert cu.tolist() == want_cu.tolist() and slots.tolist() == want_slots.tolist()
        same_plan(c, p)
    c.status()


@pytest.mark.parametrize("length,n,code", [
    ([0, -1, 0], [4, 4, 4], "DFL_E_INVALID_ARG"), ([0, 0, 0], [4, -7, 4], "DFL_E_INVALID_ARG"), ([0, 2 ** 31 - 1, 0], [4, 2 ** 31 - 1, 0], "DFL_E_CAPACITY"),
    ([0, 60, 0], [4, 5, 4], "DFL_E_CAPACITY"), ([0, 0, 0], [30, 40, 40], "DFL_E_CAPACITY"), ([0, 0, 0], [64, 64, 64], "DFL_E_CAPACITY")])
def test_plans_that_cannot_be_served(torch, length, n, code):
    c, p = cache(torch, 3, 1, 64, 9, 4, 16), Plan(3, 9, 4, 16)
    for a, b in (([0, 0, 0], [16, 16, 16]), (length, n)):
        cu, slots = c.plan(i32(torch, a), i32(torch, b), 100)
        want_cu, want_slots, _ = p.step(a, b, 100)
        assert cu.tolist() == want_cu.tolist() and slots.tolist() == want_slots.tolist()
        same_plan(c, p)
    with pytest.raises(RuntimeError, match=code):
        c.status()
    c.status()


def test_a_state_out_of_order_is_reported_and_left(torch):
    for spoil in ("held", "first", "count", "more"):
        c = cache(torch, 2, 1, 64, 8, 4, 16)
        c.plan(i32(torch, [0, 0]), i32(torch, [40, 16]), 64)
        if spoil == "held":
            c.held[0] = 5
        elif spoil == "first":
            c.queue[0] = 8
        elif spoil == "count":
            c.queue[1] = -1
        else:
            c.queue[1] = 7                       # and three more come back: pages that are named twice
        state = [x.clone() for x in (c.table, c.held, c.free, c.queue)]
        cu, slots = c.plan(i32(torch, [0, 0]), i32(torch, [0, 16]), 64)
        assert cu.tolist() == [0, 0, 16]
        if spoil != "held":                      # nothing of the call is done
            assert (slots == -1).all()
        for a, b in zip(state, (c.table, c.held, c.free, c.queue)):
            assert torch.equal(a, b)
        with pytest.raises(RuntimeError, match="DFL_E_STATE"):
            c.status()


def test_ring_entries_that_are_no_pages(torch):
    c = cache(torch, 1, 1, 64, 8, 4, 16)
    c.free[1] = 8
    _, slots = c.plan(i32(torch, [0]), i32(torch, [48]), 48)
    assert slots.tolist() == list(range(16)) + [-1] * 16 + list(range(32, 48))
    with pytest.raises(RuntimeError, match="DFL_E_INVALID_ARG"):
        c.status()


# ---- rows into pages -----------------------------------------------------------------------------------
@pytest.mark.parametrize("n_kv,hd,page,rows,t", [(1, 64, 16, 1, "bf16"), (3, 64, 32, 50, "fp16"), (2, 128, 64, 333, "bf16"), (5, 256, 128, 77, "fp16"), (16, 128, 16, 1000, "bf16")])
def test_rows_into_pages(torch, n_kv, hd, page, rows, t):
    rng = np.random.default_rng(rows)
    n_pages = rows // page + 5
    c = cache(torch, 1, n_kv, hd, n_pages, 4, page, t)
    slots = rng.permutation(n_pages * page)[:rows].astype(np.int32)
    slots[rng.random(rows) < 0.2] = -1
    wide = torch.randn(rows, (2 * n_kv + 1) * hd, device="cuda").to(dtype_of(torch, t))     # keys and values as parts of wider rows
    k, v = wide[:, :n_kv * hd].view(rows, n_kv, hd), wide[:, (n_kv + 1) * hd:].view(rows, n_kv, hd)
    want = []
    for x, new in ((c.k, k), (c.v, v)):
        w = x.clone()
        for r, s in enumerate(slots):
            if s >= 0:
                w[s // page, :, s % page] = new[r]
        want.append(w)
    c.append(k, v, i32(torch, slots))
    c.status()
    for x, w in zip((c.k, c.v), want):
        assert torch.equal(x.view(torch.int16), w.view(torch.int16))


def test_a_slot_past_the_pool(torch):
    c = cache(torch, 1, 1, 64, 4, 4, 16)
    c.k.zero_(), c.v.zero_()
    k = torch.ones(3, 1, 64, dtype=torch.bfloat16, device="cuda")
    c.append(k, k, i32(torch, [64, 5, 2 ** 31 - 1]))
    assert float(c.k.sum()) == 64 and float(c.k[0, 0, 5].sum()) == 64
    with pytest.raises(RuntimeError, match="DFL_E_INVALID_ARG"):
        c.status()


# ---- prompts -------------------------------------------------------------------------------------------
class Prompts:
    """Packed prompts with spare rows behind them, and what their attention is in 64 bits."""

    def __init__(self, torch, heads, lens, t, window=0, scale=None, seed=0, spare=3, gain=1.5):
        self.torch, self.lens, self.t, self.window = torch, lens, t, window
        self.n_q, self.n_kv, self.hd = heads
        self.scale = self.hd ** -0.5 if scale is None else scale
        rng = np.random.default_rng(seed)
        self.total = sum(lens) + spare
        self.q, self.q64 = rows_of(torch, rng, self.total, self.n_q, self.hd, t, gain)
        self.k, self.k64 = rows_of(torch, rng, self.total, self.n_kv, self.hd, t)
        self.v, self.v64 = rows_of(torch, rng, self.total, self.n_kv, self.hd, t)
        self.cu = np.concatenate([[0], np.cumsum(lens)])
        self.c = cache(torch, len(lens), self.n_kv, self.hd, t=t)

    def put(self, x, row, value, channel=None):
        """A value into a row of "k" or "v" (of one head's channel, or of all)."""
        a, b = getattr(self, x), getattr(self, x + "64")
        if channel is None:
            a[row], b[row] = value, value
        else:
            a[row, 0, channel], b[row, 0, channel] = value, value

    def want(self):
        out, tol = np.full(self.q64.shape, -77.0), np.zeros(self.q64.shape)
        for a, b in zip(self.cu[:-1], self.cu[1:]):
            if b > a:
                out[a:b], tol[a:b] = attend(self.q64[a:b], self.k64[a:b], self.v64[a:b], 0, self.window, True, self.scale, BITS[self.t])
        return out, tol

    def run(self, **more):
        out = self.torch.full_like(self.q, -77.0)
        got = self.c.prompt(self.q, self.k, self.v, i32(self.torch, self.cu), window=self.window, scale=more.get("scale", self.scale), out=out)
        assert got is out
        self.c.status()
        return back(out)

    def check(self):
        want, tol = self.want()
        near(self.run(), want, tol)


@pytest.mark.parametrize("t", ["bf16", "fp16"])
@pytest.mark.parametrize("heads", HEADS)
def test_prompts(torch, heads, t):
    for lens, window in (([1], 0), ([37, 0, 1, 150], 0), ([129, 64], 20)):
        Prompts(torch, heads, lens, t, window).check()


@pytest.mark.parametrize("lens", [[2], [15, 16, 17], [31, 32, 33], [63, 64, 65], [127, 128, 129], [255, 1, 257], [0, 0, 5, 0], [1] * 40, [383, 384, 385], [700]])
def test_lengths_of_prompts(torch, lens):
    Prompts(torch, (4, 2, 64), lens, "bf16", seed=sum(lens)).check()
    Prompts(torch, (2, 2, 128), lens, "fp16", seed=sum(lens)).check()


@pytest.mark.parametrize("heads", [(4, 2, 64), (2, 1, 128), (2, 2, 256)])
@pytest.mark.parametrize("window", [1, 2, 31, 64, 100, 128, 129, 300, 511, 600, 2 ** 31 - 1])
def test_windows_of_prompts(torch, heads, window):
    Prompts(torch, heads, [520, 90], "bf16", window, seed=window % 1000).check()


@pytest.mark.parametrize("heads", [(4, 2, 64), (1, 1, 128), (6, 1, 256)])
def test_long_prompts(torch, heads):
    Prompts(torch, heads, [1500, 1100], "fp16", seed=3).check()


@pytest.mark.parametrize("t", ["bf16", "fp16"])
@pytest.mark.parametrize("scale,gain", [(1.0, 4.0), (0.001, 1.0), (20.0, 1.0)])
def test_scales_of_prompts(torch, t, scale, gain):
    """Weights that one key takes nearly all of, and weights that are nearly equal."""
    Prompts(torch, (4, 2, 64), [200, 140], t, scale=scale, gain=gain).check()


@pytest.mark.parametrize("heads", [(4, 2, 64), (2, 2, 128), (12, 1, 256)])
def test_maxima_that_grow_and_fall_along_a_prompt(torch, heads):
    """Scores whose largest comes later and later, and then ever smaller ones: earlier sums are scaled down, or later weights nearly nothing."""
    for up in (1.0, -1.0):
        p = Prompts(torch, heads, [600], "bf16", seed=11)
        ramp = np.linspace(-30 * up, 30 * up, p.total).astype(np.float32)
        q = np.abs(p.q64) * 0 + 1.0
        k = np.repeat((ramp / (p.hd * p.scale))[:, None, None], p.n_kv, 1).repeat(p.hd, 2)
        p.q.copy_(torch.from_numpy(q)), p.k.copy_(torch.from_numpy(k))
        p.q64, p.k64 = back(p.q), back(p.k)
        p.check()


@pytest.mark.parametrize("heads", [(4, 2, 64), (2, 2, 128), (12, 1, 256)])
@pytest.mark.parametrize("window", [0, 50])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
def test_values_that_are_not_finite_reach_the_rows_that_see_them_alone(torch, heads, window, value):
    p = Prompts(torch, heads, [300, 90], "bf16", window)
    p.put("v", 200, value, 5)
    p.put("v", 389, value, 7)
    for row in (390, 391, 392):                  # spare rows
        for x in ("k", "v"):
            p.put(x, row, value)
    want, tol = p.want()
    got = p.run()
    sees = np.zeros(got.shape, bool)             # what is not finite there may be infinite or NaN
    g = p.n_q // p.n_kv
    sees[200:(300 if not window else 250), :g, 5] = True
    sees[389, :g, 7] = True
    assert not np.isfinite(got[sees]).any()
    near(np.where(sees, 0, got), np.where(sees, 0, want), np.where(sees, 0, tol))


@pytest.mark.parametrize("heads", [(4, 2, 64), (2, 2, 128), (12, 1, 256)])
def test_keys_and_queries_that_are_not_finite(torch, heads):
    """A NaN key makes NaN of the rows that see it, a NaN query of its own."""
    for window in (0, 40):
        p = Prompts(torch, heads, [260, 70], "bf16", window)
        p.put("k", 100, float("nan"), 3)
        p.q[300, 0, 2], p.q64[300, 0, 2] = float("nan"), float("nan")
        want, tol = p.want()
        got, g = p.run(), p.n_q // p.n_kv
        assert np.isnan(got[100:(260 if not window else 140), :g]).all() and np.isnan(got[300, 0]).all()
        near(got, want, tol)


def some_rows(p, rows, got, first=0):
    """Rows of the first sequence, alone against the definition."""
    for m in rows:
        want, tol = attend(p.q64[m:m + 1], p.k64[:m + 1], p.v64[:m + 1], m, p.window, True, p.scale, BITS[p.t])
        near(got[m:m + 1], want, tol)


@pytest.mark.parametrize("heads,n,window", [((12, 1, 256), 9000, 0), ((12, 2, 256), 6000, 512), ((4, 2, 64), 12000, 0), ((8, 4, 128), 10000, 0), ((16, 8, 128), 8000, 700)])
def test_prompts_of_many_items(torch, heads, n, window):
    """Many items a CTA and long rows of keys: some rows of each, several times over."""
    p = Prompts(torch, heads, [n], "bf16", window, seed=n)
    got = p.run()
    some_rows(p, [0, 1, 9, 10, 63, 64, 127, 128, 129, 1000, 2047, n // 2, n - 130, n - 65, n - 2, n - 1], got)
    for _ in range(6):
        np.testing.assert_array_equal(got, p.run())


@pytest.mark.parametrize("n_seq", [33, 256, 257, 900, 4096])
@pytest.mark.parametrize("heads", [(4, 2, 64), (2, 1, 128), (12, 1, 256)])
def test_prompts_of_many_sequences(torch, n_seq, heads):
    rng = np.random.default_rng(n_seq)
    lens = [int(x) for x in rng.integers(0, 4 if n_seq > 300 else 12, n_seq)]
    lens[n_seq // 2], lens[-1] = 150, 0
    Prompts(torch, heads, lens, "fp16", 0 if n_seq % 2 else 3, seed=n_seq).check()


@pytest.mark.parametrize("heads", [(4, 2, 64), (2, 2, 128), (12, 1, 256)])
@pytest.mark.parametrize("window", [0, 130])
def test_values_that_are_not_finite_in_long_prompts(torch, heads, window):
    """Found in the middle of long rows of keys, of which some of a tile's rows see them and others do not."""
    p = Prompts(torch, heads, [1100, 300], "bf16", window, seed=7)
    for row, ch in ((500, 0), (501, 33), (777, 63), (1099, 8), (1100, 9), (1399, 10)):
        p.put("v", row, float("inf") if row % 2 else float("nan"), ch)
    want, tol = p.want()
    got, g = p.run(), p.n_q // p.n_kv
    sees = np.zeros(got.shape, bool)
    for row, ch in ((500, 0), (501, 33), (777, 63), (1099, 8), (1100, 9), (1399, 10)):
        sees[row:min(row + (window or 10 ** 6), 1100 if row < 1100 else 1400), :g, ch] = True
    assert not np.isfinite(got[sees]).any()
    near(np.where(sees, 0, got), np.where(sees, 0, want), np.where(sees, 0, tol))


@pytest.mark.parametrize("value", [2.0 ** 90, -2.0 ** 90])
def test_large_values(torch, value):
    """Sums stay finite, also where the maximum in use falls behind."""
    p = Prompts(torch, (4, 2, 64), [400], "bf16", seed=3)
    ramp = torch.linspace(-10, 10, p.total, device="cuda")[:, None, None]
    p.q.fill_(1.0), p.k.copy_((ramp / (64 * p.scale)).expand(-1, 2, 64)), p.v.fill_(value)
    p.q64, p.k64, p.v64 = back(p.q), back(p.k), back(p.v)
    p.check()
    a = Pages(torch, (4, 2, 64), [400], [3], 16, "bf16", seed=3)
    a.c.v.fill_(value), a.v64[0].fill(float(value))
    a.check(3)


def test_rows_in_the_gaps_of_a_wide_buffer(torch):
    """Queries, keys, values and outputs as parts of one buffer's rows."""
    p = Prompts(torch, (4, 2, 64), [70, 20], "fp16", seed=5)
    wide = torch.zeros(p.total, 12 * 64, dtype=p.q.dtype, device="cuda")
    q, k, v, out = (wide[:, a * 64:b * 64].view(p.total, b - a, 64) for a, b in ((8, 12), (4, 6), (6, 8), (0, 4)))
    for x, y in ((q, p.q), (k, p.k), (v, p.v)):
        x.copy_(y)
    out.fill_(-77.0)
    p.c.prompt(q, k, v, i32(torch, p.cu), out=out)
    want, tol = p.want()
    near(back(out), want, tol)
    from dflash_speculative_decode_gb300 import DflError
    with pytest.raises(DflError):
        p.c.prompt(q, k, v, i32(torch, p.cu), out=q)


def test_rows_far_apart(torch):
    """Offsets that pass 32 bits: rows of 160 KiB, some 5 GiB of them."""
    p = Prompts(torch, (4, 2, 64), [32000, 200], "bf16", seed=6)
    wide = torch.empty(p.total, 80 * 1024, dtype=p.q.dtype, device="cuda")
    n = p.total
    q, k, v, out = (wide[:, a * 64:b * 64].view(n, b - a, 64) for a, b in ((0, 4), (6, 8), (1000, 1002), (1100, 1104)))
    for x, y in ((q, p.q), (k, p.k), (v, p.v)):
        x.copy_(y)
    out.fill_(-77.0)
    p.c.prompt(q, k, v, i32(torch, p.cu), window=300, out=out)
    p.c.status()
    got, p.window = back(out), 300
    some_rows(p, [0, 5000, 27000, 31999], got)
    a, b = 32000, 32200
    want, tol = attend(p.q64[a:b], p.k64[a:b], p.v64[a:b], 0, 300, True, p.scale, BITS["bf16"])
    near(got[a:b], want, tol)
    assert (got[b:] == -77).all()


def test_every_value_nan(torch):
    p = Prompts(torch, (4, 2, 128), [700], "bf16")
    p.v[:700].fill_(float("nan"))
    assert np.isnan(p.run()[:700]).all()


@pytest.mark.parametrize("heads", [(4, 2, 64), (2, 1, 128), (12, 2, 256)])
def test_prompts_as_parts_of_wider_rows(torch, heads):
    p = Prompts(torch, heads, [140, 61], "bf16", seed=2)
    n_q, n_kv, hd = heads
    wide = torch.zeros(p.total, (n_q + 2 * n_kv) * hd + 8, dtype=p.q.dtype, device="cuda")
    parts = [wide[:, a * hd:b * hd].view(p.total, b - a, hd) for a, b in ((0, n_q), (n_q, n_q + n_kv), (n_q + n_kv, n_q + 2 * n_kv))]
    for x, y in zip(parts, (p.q, p.k, p.v)):
        x.copy_(y)
    p.q, p.k, p.v = parts
    out = torch.full((p.total, n_q * hd + 16), -77.0, dtype=p.q.dtype, device="cuda")
    p.c.prompt(p.q, p.k, p.v, i32(torch, p.cu), out=out[:, 8:8 + n_q * hd].view(p.total, n_q, hd))
    want, tol = p.want()
    near(back(out[:, 8:8 + n_q * hd].reshape(p.total, n_q, hd)), want, tol)
    assert (out[:, :8] == -77).all() and (out[:, -8:] == -77).all()


def test_a_prompt_is_the_same_wherever_it_stands(torch):
    """A sequence's rows do not depend on the others of the call, and a call gives the same bits each time."""
    p = Prompts(torch, (8, 2, 128), [300, 77, 200], "bf16")
    whole = p.run()
    np.testing.assert_array_equal(whole, p.run())
    for a, b in zip(p.cu[:-1], p.cu[1:]):
        alone = cache(torch, 1, 2, 128).prompt(p.q[a:b], p.k[a:b], p.v[a:b], i32(torch, [0, b - a]))
        np.testing.assert_array_equal(back(alone), whole[a:b])


@pytest.mark.parametrize("cu", [[0, 50, 20, 90], [0, 50, 60, 91], [-1, 50, 60, 90], [0, 2 ** 31 - 1, 60, 90]])
def test_rows_out_of_order_are_reported(torch, cu):
    """Sequences whose bounds are sound have their rows, the others' keep what was there."""
    p = Prompts(torch, (4, 2, 64), [50, 10, 30], "bf16", spare=0)
    good = np.zeros(90, bool)
    p.cu = np.array(cu)
    for i in range(3):
        if 0 <= cu[i] <= cu[i + 1] <= 90:
            good[cu[i]:cu[i + 1]] = True
    out = torch.full_like(p.q, -77.0)
    p.c.prompt(p.q, p.k, p.v, i32(torch, cu), out=out)
    assert (back(out)[~good] == -77).all()
    with pytest.raises(RuntimeError, match="DFL_E_INVALID_ARG"):
        p.c.status()
    p.c.status()


# ---- attention over pages --------------------------------------------------------------------------------
class Pages:
    """Sequences of given lengths in pages in any order, the rows of a step behind them, and their attention in 64 bits."""

    def __init__(self, torch, heads, lens, counts, page, t, seed=0, spare=2, gain=1.5, wide=0):
        self.torch, self.lens, self.counts, self.t = torch, np.asarray(lens), np.asarray(counts), t
        self.n_q, self.n_kv, self.hd = heads
        rng = np.random.default_rng(seed)
        S = len(lens)
        need = [-(-(a + b) // page) for a, b in zip(lens, counts)]
        n_pages, most = sum(need) + 2, max(need) + 1 + wide
        self.c = c = cache(torch, S, self.n_kv, self.hd, n_pages, most, page, t)
        order = rng.permutation(n_pages)
        table = np.full((S, most), 2 ** 30, np.int32)              # entries that no call may follow
        at, self.k64, self.v64 = 0, [], []
        for s in range(S):
            mine = order[at:at + need[s]]
            table[s, :need[s]] = mine
            at += need[s]
            end = int(self.lens[s] + self.counts[s])
            for x, keep in ((c.k, self.k64), (c.v, self.v64)):
                rows, r64 = rows_of(torch, rng, end, self.n_kv, self.hd, t)
                keep.append(r64)
                for i, pg in enumerate(mine):
                    part = rows[i * page:(i + 1) * page]
                    x[int(pg), :, :part.shape[0]] = part.transpose(0, 1)
        c.table.copy_(i32(torch, table))
        c.held.copy_(i32(torch, need))
        self.total = int(self.counts.sum()) + spare
        self.q, self.q64 = rows_of(torch, rng, self.total, self.n_q, self.hd, t, gain)
        self.cu = np.concatenate([[0], np.cumsum(counts)])

    def put(self, x, s, token, value, channel):
        """A value into a channel of head 0 of a token."""
        page = self.c.page
        getattr(self.c, x)[int(self.c.table[s, token // page]), 0, token % page, channel] = value
        getattr(self, x + "64")[s][token, 0, channel] = value

    def want(self, window, causal, scale):
        out, tol = np.full(self.q64.shape, -77.0), np.zeros(self.q64.shape)
        for s in range(len(self.lens)):
            a, b = self.cu[s], self.cu[s + 1]
            if b > a:
                out[a:b], tol[a:b] = attend(self.q64[a:b], self.k64[s], self.v64[s], int(self.lens[s]), window, causal, scale, BITS[self.t])
        return out, tol

    def run(self, rows, window=0, causal=True, scale=None):
        out = self.torch.full_like(self.q, -77.0)
        got = self.c.attn(self.q, i32(self.torch, self.cu), i32(self.torch, self.lens), rows, window=window, causal=causal, scale=scale, out=out)
        assert got is out
        return back(out)

    def check(self, rows, window=0, causal=True, scale=None):
        want, tol = self.want(window, causal, self.hd ** -0.5 if scale is None else scale)
        near(self.run(rows, window, causal, scale), want, tol)
        self.c.status()


@pytest.mark.parametrize("t", ["bf16", "fp16"])
@pytest.mark.parametrize("heads", HEADS)
def test_attention_over_pages(torch, heads, t):
    Pages(torch, heads, [0], [1], 16, t).check(1)
    Pages(torch, heads, [100, 0, 33, 5], [1, 1, 1, 0], 32, t).check(1)
    p = Pages(torch, heads, [70, 200, 0], [5, 8, 3], 64, t)
    for window, causal in ((0, True), (0, False), (17, True), (17, False)):
        p.check(8, window, causal)


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("rows", [1, 2, 7, 16])
@pytest.mark.parametrize("heads", [(4, 2, 64), (12, 1, 256), (32, 8, 128)])
def test_pages_and_rows(torch, page, rows, heads):
    p = Pages(torch, heads, [page - 1, page, 3 * page + 1, 0, 5 * page - rows], [rows, max(1, rows - 1), 0, rows, rows], page, "bf16")
    p.check(rows)
    p.check(rows, 2 * page - 3, True)
    p.check(16, page, False)


@pytest.mark.parametrize("length", [1, 15, 16, 17, 63, 64, 65, 127, 128, 255, 256, 257, 511, 1000, 3000])
def test_lengths_over_pages(torch, length):
    Pages(torch, (4, 2, 64), [length], [1], 16, "bf16", seed=length).check(1)
    Pages(torch, (6, 2, 128), [length, 1], [4, 4], 64, "fp16", seed=length).check(4)


@pytest.mark.parametrize("window", [1, 2, 15, 16, 63, 64, 65, 500, 999, 1000, 1001, 2 ** 31 - 1])
@pytest.mark.parametrize("causal", [True, False])
def test_windows_over_pages(torch, window, causal):
    Pages(torch, (4, 2, 64), [1000, 40], [6, 6], 16, "bf16", seed=1).check(6, window, causal)
    Pages(torch, (4, 1, 256), [700], [1], 128, "fp16", seed=1).check(1, window, causal)


def test_many_sequences_of_many_lengths(torch):
    rng = np.random.default_rng(8)
    lens = rng.integers(0, 400, 150)
    Pages(torch, (4, 2, 64), lens, rng.integers(0, 2, 150), 16, "bf16").check(1)
    Pages(torch, (4, 1, 128), lens[:60], rng.integers(0, 9, 60), 32, "bf16").check(8)


@pytest.mark.parametrize("heads", [(4, 2, 64), (32, 8, 128), (12, 1, 256)])
@pytest.mark.parametrize("lens", [[100], [0, 5, 0], [300] * 20, [900, 20, 0, 3], [5000] + [10] * 30, [60] * 400, [5000] + [70] * 400, [2000] * 40,
                                  [0] * 900 + [6000] + [0] * 1000 + [500]])
def test_short_sequences_in_a_wide_table(torch, heads, lens):
    """The capacity says nothing of the lengths: units are taken whole or cut by what the sequences hold."""
    n = [1 if (i % 7 != 6 if len(lens) < 1000 else x > 0) else 0 for i, x in enumerate(lens)]
    Pages(torch, heads, lens, n, 16, "bf16", seed=len(lens), wide=2000).check(1)
    if len(lens) < 100:
        Pages(torch, heads, lens, [3 * x for x in n], 64, "fp16", seed=len(lens), wide=500).check(3)


@pytest.mark.parametrize("heads,rows", [((12, 2, 256), 1), ((32, 8, 128), 1), ((4, 1, 64), 8), ((16, 1, 128), 16), ((16, 1, 256), 16)])
def test_long_contexts(torch, heads, rows):
    Pages(torch, heads, [9000], [rows], 64, "bf16", seed=4).check(rows)


@pytest.mark.parametrize("scale,gain", [(1.0, 4.0), (0.001, 1.0), (20.0, 1.0)])
def test_scales_over_pages(torch, scale, gain):
    Pages(torch, (4, 2, 64), [900, 30], [3, 2], 16, "bf16", gain=gain).check(3, scale=scale)
    Pages(torch, (4, 2, 128), [900, 30], [1, 1], 16, "fp16", gain=gain).check(1, scale=scale)


@pytest.mark.parametrize("heads", [(4, 2, 64), (8, 2, 128), (12, 1, 256)])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("long", [0, 3000])
def test_values_over_pages_that_are_not_finite(torch, heads, value, long):
    """A staged token that later rows alone see, one that a window has left behind for some rows, and one that all see."""
    base = 100 + long
    p = Pages(torch, heads, [base, 40], [6, 6], 16, "bf16")
    g = p.n_q // p.n_kv
    p.put("v", 0, base + 3, value, 5)            # seen by rows 3, 4, 5
    p.put("v", 0, base - 50 + 2, value, 9)       # with a window of 50 by rows 0 and 1 alone
    p.put("v", 1, 7, value, 1)
    p.put("v", 0, 1, value, 11)                  # before the window
    for window in (0, 50):
        want, tol = p.want(window, True, p.hd ** -0.5)
        got = p.run(6, window)
        sees = np.zeros(got.shape, bool)
        sees[3:6, :g, 5] = True
        sees[0:(6 if not window else 2), :g, 9] = True
        sees[6:(12 if not window else 6 + 50), :g, 1] = True
        if not window:
            sees[0:6, :g, 11] = True
        sees[12:] = False
        assert not np.isfinite(got[sees]).any()
        near(np.where(sees, 0, got), np.where(sees, 0, want), np.where(sees, 0, tol))
        p.c.status()


@pytest.mark.parametrize("window", [1, 5, 16, 17, 40, 100])
@pytest.mark.parametrize("causal", [True, False])
def test_a_token_does_not_touch_what_its_window_has_left(torch, window, causal):
    """One row: every token before its window is a NaN, and so is what lies behind the row in its page."""
    p = Pages(torch, (4, 2, 64), [200, 77], [1, 1], 32, "bf16")
    for s, length in enumerate((200, 77)):
        lo = max(0, length - window + 1 if causal else length - window)
        for token in range(lo):
            for x in ("k", "v"):
                p.put(x, s, token, float("nan"), 3)
    want, tol = p.want(window, causal, 0.125)
    got = p.run(1, window, causal)
    assert np.isfinite(got).all()
    near(got, want, tol)


def test_keys_over_pages_that_are_not_finite(torch):
    p = Pages(torch, (4, 2, 64), [100], [6], 16, "bf16")
    p.put("k", 0, 103, float("nan"), 5)
    want, tol = p.want(0, True, 0.125)
    got = p.run(6)
    assert np.isnan(got[3:6, :2]).all() and np.isfinite(got[:3]).all()
    near(got, want, tol)


def test_sequences_that_cannot_be_attended(torch):
    """More rows than the call allows, pages that are missing, a negative length: left as they are, and reported; the others are served."""
    for spoil, code in (("rows", "DFL_E_INVALID_ARG"), ("held", "DFL_E_STATE"), ("len", "DFL_E_INVALID_ARG"), ("far", "DFL_E_STATE"), ("heldmost", "DFL_E_STATE")):
        p = Pages(torch, (4, 2, 64), [40, 50, 60], [3, 4, 3], 16, "bf16")
        want, tol = p.want(0, True, 0.125)
        if spoil == "held":
            p.c.held[1] = 3
        elif spoil == "len":
            p.lens[1] = -1
        elif spoil == "far":
            p.lens[1] = 2 ** 31 - 2
        elif spoil == "heldmost":
            p.c.held[1] = p.c.max_pages + 1
            p.lens[1] = 16 * p.c.max_pages
        want[3:7], tol[3:7] = -77.0, 0.0
        near(p.run(3 if spoil == "rows" else 4), want, tol)
        with pytest.raises(RuntimeError, match=code):
            p.c.status()
        p.c.status()


def test_table_entries_that_are_no_pages(torch):
    p = Pages(torch, (4, 2, 64), [100, 100], [2, 2], 16, "bf16")
    want, tol = p.want(0, True, 0.125)
    p.c.table[1, 2] = p.c.n_pages
    want[2:4] = float("nan")
    near(p.run(2), want, tol)
    with pytest.raises(RuntimeError, match="DFL_E_INVALID_ARG"):
        p.c.status()
    p.c.table[1, 2] = -1
    near(p.run(2), want, tol)
    with pytest.raises(RuntimeError, match="DFL_E_INVALID_ARG"):
        p.c.status()
    got = p.run(2, window=30)                    # the page is out of sight
    want, tol = p.want(30, True, 0.125)
    near(got, want, tol)
    p.c.status()


@pytest.mark.parametrize("cu", [[0, 3, 2, 9], [0, 3, 7, 13], [-1, 3, 6, 9], [0, 2 ** 31 - 1, 6, 9]])
def test_rows_over_pages_out_of_order_are_reported(torch, cu):
    p = Pages(torch, (4, 2, 64), [40, 50, 60], [3, 3, 3], 16, "bf16")
    p.cu = np.array(cu)
    got = p.run(3)
    good = np.zeros(len(got), bool)
    for i in range(3):
        if 0 <= cu[i] <= cu[i + 1] <= len(got) and cu[i + 1] - cu[i] <= 3:
            good[cu[i]:cu[i + 1]] = True
    assert (got[~good] == -77).all() and np.isfinite(got).all()
    with pytest.raises(RuntimeError, match="DFL_E_INVALID_ARG"):
        p.c.status()


@pytest.mark.parametrize("n_seq,most", [(3000, 40), (4096, 3), (700, 300)])
def test_attention_of_very_many_sequences(torch, n_seq, most):
    rng = np.random.default_rng(n_seq)
    Pages(torch, (4, 2, 64), rng.integers(0, most, n_seq), rng.integers(0, 2, n_seq), 16, "bf16").check(1)


def test_pages_far_into_the_pool(torch):
    """A pool of more than 4 GiB each of keys and values, whose last pages are in use."""
    p = Pages(torch, (8, 8, 256), [300, 20], [2, 1], 128, "bf16", seed=9)
    big = cache(torch, 2, 8, 256, 1, p.c.max_pages, 128)
    from dflash_speculative_decode_gb300 import PagedCache
    N, n = 9000, p.c.n_pages
    k, v = (torch.empty(N, 8, 128, 256, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    table = torch.where(p.c.table < n, p.c.table + (N - n), p.c.table)
    c = PagedCache(k, v, table.contiguous(), p.c.held, torch.zeros(N, dtype=torch.int32, device="cuda"), big.queue)
    rows = torch.arange(n * 128, device="cuda")
    for x, y in ((k, p.c.k), (v, p.c.v)):
        x[:N - n].fill_(float("nan"))
    flat = [y.transpose(1, 2).reshape(n * 128, 8, 256) for y in (p.c.k, p.c.v)]
    c.append(*flat, ((N - n) * 128 + rows).to(torch.int32))
    assert torch.equal(k[N - n:].view(torch.int16), p.c.k.view(torch.int16)) and torch.equal(v[N - n:].view(torch.int16), p.c.v.view(torch.int16))
    p.c = c
    p.check(2)


def test_the_same_bits_each_time(torch):
    for heads, rows, lens in (((12, 2, 256), 1, [9000]), ((32, 8, 128), 2, [300, 2000, 4, 0, 900]), ((16, 1, 128), 16, [3000, 100])):
        p = Pages(torch, heads, lens, [rows] * len(lens), 32, "bf16")
        first = p.run(rows)
        for _ in range(3):
            np.testing.assert_array_equal(first, p.run(rows))


# ---- a run of them ----------------------------------------------------------------------------------------
class Server:
    """Requests that come, prefill, decode with verifies that are partly rolled back, and end, over two layers that share a plan."""

    def __init__(self, torch, heads, n_seq, n_pages, page, t, rows, seed):
        from dflash_speculative_decode_gb300 import PagedCache
        self.torch, self.heads, self.S, self.rows, self.t = torch, heads, n_seq, rows, t
        self.rng = np.random.default_rng(seed)
        c = cache(torch, n_seq, heads[1], heads[2], n_pages, n_pages, page, t)
        d = PagedCache(torch.full_like(c.k, float("nan")), torch.full_like(c.v, float("nan")), c.table, c.held, c.free, c.queue)
        self.layers = [c, d]
        self.length = np.zeros(n_seq, np.int64)
        self.past = [[[np.zeros((0, heads[1], heads[2])) for _ in range(2)] for _ in range(n_seq)] for _ in self.layers]
        self.cu, self.slots = i32(torch, [0] * (n_seq + 1)), i32(torch, [0] * rows)
        self.dev_len, self.dev_n = i32(torch, self.length), i32(torch, self.length)
        n_q, n_kv, hd = heads
        dt = dtype_of(torch, t)
        self.buf = [[torch.zeros(rows, h, hd, dtype=dt, device="cuda") for h in (n_q, n_kv, n_kv, n_q)] for _ in self.layers]

    def calls(self, prompt, most):
        self.layers[0].plan(self.dev_len, self.dev_n, out=(self.cu, self.slots))
        for c, (q, k, v, out) in zip(self.layers, self.buf):
            c.append(k, v, self.slots)
            if prompt:
                c.prompt(q, k, v, self.cu, out=out)
            else:
                c.attn(q, self.cu, self.dev_len, most, window=30 if c is self.layers[1] else 0, out=out)

    def step(self, n, prompt, kept, most=8, play=None):
        torch, (n_q, n_kv, hd) = self.torch, self.heads
        self.dev_len.copy_(i32(torch, self.length)), self.dev_n.copy_(i32(torch, n))
        new = []
        for bufs in self.buf:
            made = [rows_of(torch, self.rng, self.rows, h, hd, self.t, 1.2) for h in (n_q, n_kv, n_kv)]
            for x, (y, _) in zip(bufs, made):
                x.copy_(y)
            bufs[3].fill_(-77.0)
            new.append([y for _, y in made])
        play() if play else self.calls(prompt, most)
        for c in self.layers:
            c.status()
        cu = np.concatenate([[0], np.cumsum(n)])
        for i, ((q, k, v), bufs) in enumerate(zip(new, self.buf)):
            got = back(bufs[3])
            assert (got[cu[-1]:] == -77).all()
            for s in range(self.S):
                a, b = cu[s], cu[s + 1]
                pk, pv = self.past[i][s]
                pk, pv = (np.concatenate([x[:int(self.length[s])], y[a:b]]) for x, y in ((pk, k), (pv, v)))
                self.past[i][s] = [pk, pv]
                if b > a:
                    want, tol = attend(q[a:b], pk, pv, int(self.length[s]), 30 if i and not prompt else 0, True, hd ** -0.5, BITS[self.t])
                    near(got[a:b], want, tol)
        self.length = self.length + kept

    def end(self, s):
        self.length[s] = 0


@pytest.mark.parametrize("heads,page,t", [((4, 2, 64), 16, "bf16"), ((6, 2, 128), 32, "fp16"), ((12, 1, 256), 64, "bf16")])
def test_a_server_of_requests(torch, heads, page, t):
    z = Server(torch, heads, 3, 400 // page + 3, page, t, 150, 5)
    z.step(np.array([60, 0, 41]), True, np.array([60, 0, 41]))
    rng = np.random.default_rng(1)
    for _ in range(4):
        n = np.array([4, 0, 7])
        z.step(n, False, rng.integers(0, n + 1))
    z.end(0)
    z.length[2], held = 0, z.length[2]           # the third waits while a prompt comes in the second's place
    z.past[0][2], z.past[1][2] = [[x[:0] for x in y[2]] for y in z.past]
    z.step(np.array([0, 101, 0]), True, np.array([0, 101, 0]))
    for _ in range(3):
        n = np.array([0, 8, 0])
        z.step(n, False, rng.integers(0, n + 1))
    z.end(1)
    z.step(np.array([0, 0, 0]), False, np.zeros(3, int))
    assert z.layers[0].queue[1] == z.layers[0].n_pages and held


def test_a_captured_step_replays_at_any_lengths(torch):
    z = Server(torch, (4, 2, 64), 4, 60, 16, "bf16", 40, 9)
    z.step(np.array([5, 9, 0, 12]), True, np.array([5, 9, 0, 12]))
    z.calls(False, 8)                            # everything is allocated before the capture
    for c in z.layers:                           # (12 rows are more than a verify's 8)
        with pytest.raises(RuntimeError, match="DFL_E_INVALID_ARG"):
            c.status()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        z.calls(False, 8)
    rng = np.random.default_rng(2)
    for _ in range(6):
        n = rng.integers(0, 9, 4)
        z.step(n, False, rng.integers(0, n + 1), play=g.replay)
    p = torch.cuda.CUDAGraph()
    z.length[:] = 0
    with torch.cuda.graph(p):
        z.calls(True, 8)
    for n in ([7, 0, 30, 1], [0, 0, 0, 0], [10, 10, 10, 10]):
        z.length[:] = 0
        z.step(np.array(n), True, np.zeros(4, int), play=p.replay)


def test_on_another_stream(torch):
    side = torch.cuda.Stream()
    p, a = Prompts(torch, (4, 2, 64), [100], "bf16"), Pages(torch, (4, 2, 64), [300], [2], 16, "bf16")
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        p.check()
        a.check(2)


def test_python_refusals(torch):
    from dflash_speculative_decode_gb300 import DflError, PagedCache
    c = cache(torch, 2, 2, 64)
    q, k = torch.zeros(5, 4, 64, dtype=torch.bfloat16, device="cuda"), torch.zeros(5, 2, 64, dtype=torch.bfloat16, device="cuda")
    cu, n = i32(torch, [0, 2, 5]), i32(torch, [2, 3])
    bad = [lambda: c.append(k.float(), k, cu), lambda: c.append(k, k[:4], i32(torch, [0] * 5)), lambda: c.append(k, k, i32(torch, [0] * 4)),
           lambda: c.append(k, k, cu.long()[:0]), lambda: c.prompt(q.half(), k, k, cu), lambda: c.prompt(q, k, k, n), lambda: c.prompt(q[:4], k, k, cu),
           lambda: c.prompt(q[:, :3], k, k, cu), lambda: c.prompt(q.cpu(), k, k, cu), lambda: c.prompt(q, k, k, cu, window=-1), lambda: c.prompt(q, k, k, cu, scale=0.0),
           lambda: c.attn(q, cu, n, 0), lambda: c.attn(q, cu, n, 17), lambda: c.attn(q, cu, cu, 1), lambda: c.attn(q[:, :, :32], cu, n, 1),
           lambda: c.attn(q, cu, n, 1, out=q[:3]), lambda: c.attn(q.transpose(0, 1), cu, n, 1), lambda: c.plan(n, n), lambda: c.plan(n, cu, 5),
           lambda: c.plan(n, n, 5, out=(cu, n)), lambda: PagedCache(c.k.float(), c.v, c.table, c.held, c.free, c.queue),
           lambda: PagedCache(c.k, c.v, c.table, c.held, c.free, c.queue[:2]), lambda: PagedCache.empty(1, 1, 96, 1, 1), lambda: PagedCache.empty(1, 1, 64, 1, 1, page=48)]
    for i, f in enumerate(bad):
        with pytest.raises(DflError):
            f()
            pytest.fail(str(i))
    c.status()
    assert c.attn(q[:0], cu, n, 1).shape == (0, 4, 64) and c.prompt(q[:0], k[:0], k[:0], i32(torch, [0, 0, 0])).shape == (0, 4, 64)
