"""The paged key/value cache's attentions where they can go wrong, against derived bounds (tests/paged_bounds.py)."""
import numpy as np
import pytest

from paged_bounds import attend_exact, far, lifted, spiked
from paged_plain import Plan
from test_gpu_paged import Pages, Prompts, Server, cache, i32, near, same_plan, torch  # noqa: F401  (torch: the fixture)

pytestmark = pytest.mark.gpu


def rounded(torch, x, t):
    """x in the type on the GPU, and what it holds in 64 bits."""
    y = torch.from_numpy(np.asarray(x, np.float32)).to({"bf16": torch.bfloat16, "fp16": torch.float16}[t])
    return y.cuda(), y.double().numpy()


class ExactPrompts(Prompts):
    """Prompts of given numbers, within the bound for scores that come without rounding."""

    def __init__(self, torch, heads, lens, t, make, window=0, seed=0, scale=None):
        super().__init__(torch, heads, lens, t, window, scale, seed, spare=0)
        rng = np.random.default_rng(seed)
        n_q, n_kv, hd = heads
        made = [make(rng, n, n_q, n_kv, n, hd) for n in lens]
        for i, x in enumerate("qkv"):
            y, y64 = rounded(torch, np.concatenate([m[i] for m in made]), t)
            setattr(self, x, y), setattr(self, x + "64", y64)

    def want(self):
        out, tol = np.full(self.q64.shape, -77.0), np.zeros(self.q64.shape)
        for a, b in zip(self.cu[:-1], self.cu[1:]):
            if b > a:
                out[a:b], tol[a:b] = attend_exact(self.q64[a:b], self.k64[a:b], self.v64[a:b], 0, self.window, True, self.scale, self.t, 1)
        return out, tol


class ExactPages(Pages):
    """The same over pages. `wide`: pages of a table beyond what a sequence needs, so that the capacity does not say that its units are short."""

    def __init__(self, torch, heads, lens, counts, page, t, make, seed=0, wide=0):
        super().__init__(torch, heads, lens, counts, page, t, seed, spare=0, wide=wide)
        rng = np.random.default_rng(seed)
        n_q, n_kv, hd = heads
        made = [make(rng, b, n_q, n_kv, a + b, hd) for a, b in zip(lens, counts)]
        self.q, self.q64 = rounded(torch, np.concatenate([m[0] for m in made]), t)
        for s, m in enumerate(made):
            table = self.c.table[s].tolist()
            for x, keep, rows in ((self.c.k, self.k64, m[1]), (self.c.v, self.v64, m[2])):
                y, keep[s] = rounded(torch, rows, t)
                for i in range(-(-len(rows) // page)):
                    part = y[i * page:(i + 1) * page]
                    x[table[i], :, :part.shape[0]] = part.transpose(0, 1)

    def want(self, window, causal, scale, rows=1):
        g = self.n_q // self.n_kv
        out, tol = np.full(self.q64.shape, -77.0), np.zeros(self.q64.shape)
        for s in range(len(self.lens)):
            a, b = self.cu[s], self.cu[s + 1]
            if b > a:
                out[a:b], tol[a:b] = attend_exact(self.q64[a:b], self.k64[s], self.v64[s], int(self.lens[s]), window, causal, scale, self.t, 2 if rows * g <= 16 else 1)
        return out, tol

    def check(self, rows, window=0, causal=True, scale=None):
        want, tol = self.want(window, causal, self.hd ** -0.5 if scale is None else scale, rows)
        near(self.run(rows, window, causal, scale), want, tol)
        self.c.status()


LARGE = {"fp16": 2.0 ** 28, "bf16": 2.0 ** 60}       # units of scores whose numbers the type holds


# ---- scores so large that a rounding of theirs is worth many powers of two -----------------------------------
@pytest.mark.parametrize("t", ["bf16", "fp16"])
@pytest.mark.parametrize("heads", [(4, 2, 64), (2, 1, 128), (12, 1, 256)])
def test_prompts_of_very_large_scores(torch, heads, t):
    for unit, scale in ((LARGE[t], None), (LARGE[t], 0.3), (2.0 ** 14, None)):
        ExactPrompts(torch, heads, [300, 70], t, lambda *a: far(*a, unit), seed=1, scale=scale).check()
    ExactPrompts(torch, heads, [300], t, lambda *a: far(*a, LARGE[t]), window=40, seed=2).check()


@pytest.mark.parametrize("t", ["bf16", "fp16"])
@pytest.mark.parametrize("heads", [(4, 2, 64), (2, 1, 128), (12, 1, 256)])
@pytest.mark.parametrize("lift", [0.0, 2.0 ** 10, 2.0 ** 14, 2.0 ** 18])
def test_prompts_of_scores_around_a_large_one(torch, heads, t, lift):
    ExactPrompts(torch, heads, [400, 30], t, lambda *a: lifted(*a, lift), seed=3).check()


@pytest.mark.parametrize("t", ["bf16", "fp16"])
@pytest.mark.parametrize("heads", [(4, 2, 64), (6, 2, 128), (12, 1, 256)])
@pytest.mark.parametrize("lens,wide", [([300, 70], 0), ([1500], 2000)])
def test_pages_of_very_large_scores(torch, heads, t, lens, wide):
    """Units that are taken whole, and cut ones, whose parts have maxima of their own."""
    for unit, rows in ((LARGE[t], 1), (LARGE[t], 3), (2.0 ** 14, 3)):
        ExactPages(torch, heads, lens, [rows] * len(lens), 16, t, lambda *a: far(*a, unit), seed=1, wide=wide).check(rows, scale=0.3)


@pytest.mark.parametrize("t", ["bf16", "fp16"])
@pytest.mark.parametrize("heads", [(4, 2, 64), (6, 2, 128), (12, 1, 256)])
@pytest.mark.parametrize("lift", [0.0, 2.0 ** 10, 2.0 ** 14, 2.0 ** 18])
def test_pages_of_scores_around_a_large_one(torch, heads, t, lift):
    for lens, wide in (([300, 70], 0), ([1500], 2000)):
        p = ExactPages(torch, heads, lens, [2] * len(lens), 16, t, lambda *a: lifted(*a, lift), seed=3, wide=wide)
        p.check(2)
        p.check(2, window=200)


# ---- weights as two numbers of the type -------------------------------------------------------------------------
@pytest.mark.parametrize("t", ["bf16", "fp16"])
@pytest.mark.parametrize("heads,rows", [((4, 2, 64), 4), ((2, 1, 64), 8), ((12, 2, 128), 2), ((16, 1, 128), 1), ((12, 1, 256), 1), ((4, 2, 256), 7)])
@pytest.mark.parametrize("lens,wide", [([100, 33], 0), ([600], 2000)])
def test_both_parts_of_a_weight(torch, heads, rows, t, lens, wide):
    """Units of up to 16 rows are as near the definition as their output's rounding and fp32 let them: a bound that outputs without
    a weight's second part, or with one of the wrong sign, exceed (tests/test_paged_bounds.py). Units taken whole, and cut ones."""
    p = ExactPages(torch, heads, lens, [rows] * len(lens), 16, t, spiked, seed=5, wide=wide)
    p.check(rows)
    p.check(rows, causal=False)


# ---- keys and queries that are infinite -------------------------------------------------------------------------

@pytest.mark.parametrize("t", ["bf16", "fp16"])
@pytest.mark.parametrize("heads", [(4, 2, 64), (2, 1, 128), (12, 1, 256)])
@pytest.mark.parametrize("window", [0, 40])
def test_infinite_keys_and_queries_of_prompts(torch, heads, window, t):
    """A score of minus infinity takes no weight, and NaN is what has no other score, or one of plus infinity or NaN."""
    g = heads[0] // heads[1]
    p = ExactPrompts(torch, heads, [260, 70], t, spiked, window, seed=7)
    sign = np.sign(p.q64[:, 0])                  # (of head 0's queries: the same in all rows, and no 0)
    low, high = sign[0] * -np.inf, sign[260] * np.inf
    p.put("k", 0, low[3], 3)                     # the first row sees nothing else
    p.put("k", 100, low[5], 5)
    p.put("k", 300, high[7], 7)                  # (a row of the second prompt)
    p.q[200, heads[0] - 1, 2], p.q64[200, heads[0] - 1, 2] = float("inf"), np.inf
    with np.errstate(invalid="ignore"):
        want, tol = p.want()
    got = p.run()
    nan = np.zeros(got.shape[:2], bool)
    nan[0, :g], nan[200, -1] = True, True
    nan[300:(330 if not window else 340), :g] = True
    np.testing.assert_array_equal(np.isnan(want).all(-1), nan)
    assert np.isfinite(want[~nan]).all()
    near(got, want, tol)


@pytest.mark.parametrize("t", ["bf16", "fp16"])
@pytest.mark.parametrize("heads", [(4, 2, 64), (6, 2, 128), (12, 1, 256)])
@pytest.mark.parametrize("lens,wide", [([200, 0], 0), ([1500, 0], 2000)])
def test_infinite_keys_and_queries_over_pages(torch, heads, lens, wide, t):
    g = heads[0] // heads[1]
    n = lens[0]
    for where in (7, n // 2, n + 1):             # in a unit's first part, a middle one, and among the rows themselves
        for high in (False, True):
            p = ExactPages(torch, heads, lens, [4, 3], 16, t, spiked, seed=n, wide=wide)
            p.put("k", 0, where, np.sign(p.q64[0, 0, 5]) * (np.inf if high else -np.inf), 5)
            p.put("k", 1, 0, np.sign(p.q64[4, 0, 3]) * -np.inf, 3)        # the second sequence's first row sees nothing else
            p.q[3, heads[0] - 1, 2], p.q64[3, heads[0] - 1, 2] = float("-inf"), -np.inf
            for window in (0, 50):
                with np.errstate(invalid="ignore"):
                    want, tol = p.want(window, True, p.hd ** -0.5, 4)
                nan = np.zeros(want.shape[:2], bool)
                nan[4, :g], nan[3, -1] = True, True
                if high and (not window or where > n - 47):
                    nan[max(0, where - n):4, :g] = True
                np.testing.assert_array_equal(np.isnan(want).all(-1), nan)
                assert np.isfinite(want[~nan]).all()
                near(p.run(4, window), want, tol)
                p.c.status()


# ---- a wait that gives up ------------------------------------------------------------------------------------------
@pytest.fixture
def stall():
    from dflash_speculative_decode_gb300._abi import lib
    yield lib().dfl_paged_test_stall
    lib().dfl_paged_test_stall(0)


@pytest.mark.parametrize("heads", [(4, 2, 64), (2, 1, 128), (3, 1, 256)])
@pytest.mark.parametrize("copies", [1, 2, 5, -1, -4])
def test_a_prompt_whose_copies_do_not_come(torch, stall, heads, copies):
    """No fault and no endless wait: the copies of every item stop, in its first pass or in the one over values that are not finite; the
    waits give up after a second, the status says so, and the cache works as before."""
    from dflash_speculative_decode_gb300 import DflError
    from dflash_speculative_decode_gb300._abi import DFL_E_TIMEOUT
    p = Prompts(torch, heads, [700, 40], "bf16", seed=4)
    if copies < 0:
        for row in (1, 300, 705):                # (each item has rows that do not see one of its keys' values)
            p.put("v", row, float("nan"), 2)
    stall(copies)
    p.c.prompt(p.q, p.k, p.v, i32(torch, p.cu), out=torch.empty_like(p.q))
    with pytest.raises(DflError) as e:
        p.c.status()
    assert e.value.code == DFL_E_TIMEOUT
    p.c.status()
    stall(0)
    want, tol = p.want()
    near(p.run(), want, tol)
    p.c.status()


# ---- sizes at the limits -------------------------------------------------------------------------------------------
def test_more_tokens_than_a_call_counts(torch):
    """A table whose rows all name one page: 4096 sequences of 2^25 tokens each are as many as 2^31 granules of 64. Nothing is done, and
    the next call works."""
    from dflash_speculative_decode_gb300 import PagedCache
    S, per = 4096, 1 << 18
    z = lambda *shape: torch.zeros(*shape, dtype=torch.int32, device="cuda")  # noqa: E731
    k = torch.zeros(1, 1, 128, 64, dtype=torch.bfloat16, device="cuda")
    c = PagedCache(k, k.clone(), z(S, per), z(S) + per, z(1), z(4))
    q, cu = torch.zeros(S, 1, 64, dtype=torch.bfloat16, device="cuda"), torch.arange(S + 1, dtype=torch.int32, device="cuda")
    for n in (S, 2100):                          # (2^30 and some granules)
        length = z(S)
        length[:n] = per * 128 - 1
        out = torch.full_like(q, -77.0)
        c.attn(q, cu, length, 1, out=out)
        assert (out == -77).all()
        with pytest.raises(RuntimeError, match="DFL_E_STATE"):
            c.status()
    assert (c.attn(q, cu, z(S) + 5, 1, out=out) == 0).all()
    c.status()


def test_sizes_that_32_bits_do_not_hold(torch):
    """What ctypes would cut down to a size that the library takes is refused: windows, rows, slots, a table of 2^32 + 2 pages."""
    from dflash_speculative_decode_gb300 import DflError, PagedCache
    p, a = Prompts(torch, (4, 2, 64), [20], "bf16"), Pages(torch, (4, 2, 64), [300], [2], 16, "bf16")
    cu, length, c = i32(torch, a.cu), i32(torch, a.lens), a.c
    wide = torch.empty(2 ** 32 + 2, dtype=torch.int32, device="cuda")
    for f in (lambda: p.c.prompt(p.q, p.k, p.v, i32(torch, p.cu), window=2 ** 32 + 5), lambda: c.attn(a.q, cu, length, 2, window=2 ** 32 + 5),
              lambda: p.c.prompt(p.q, p.k, p.v, i32(torch, p.cu), window=5 - 2 ** 32), lambda: c.attn(a.q, cu, length, 2, window=5 - 2 ** 32),
              lambda: c.attn(a.q, cu, length, 2 ** 32 + 2), lambda: c.attn(a.q, cu, length, 2 - 2 ** 32), lambda: c.plan(length, i32(torch, [2]), out=(i32(torch, [0, 0]), wide)),
              lambda: PagedCache(c.k, c.v, wide[None], c.held, c.free, c.queue)):
        with pytest.raises(DflError, match="DFL_E_INVALID_ARG"):
            f()
    p.window = 2 ** 31 - 1
    p.check()
    a.check(2, window=2 ** 31 - 1)


# ---- plans ---------------------------------------------------------------------------------------------------------
def test_what_lies_behind_rows_that_do_not_fit(torch):
    """The third sequence has ended, but lies behind one whose rows reach past the buffer: it keeps its pages in this plan, and gives them back in
    the next. One before it gives its pages back at once."""
    c, p = cache(torch, 4, 1, 64, 12, 4, 16), Plan(4, 12, 4, 16)
    for length, n, rows in (([0, 0, 0, 0], [40, 16, 30, 5], 100), ([0, 16, 0, 5], [0, 20, 0, 3], 10), ([0, 16, 0, 5], [0, 4, 0, 3], 10)):
        cu, slots = c.plan(i32(torch, length), i32(torch, n), rows)
        want_cu, want_slots, short = p.step(length, n, rows)
        assert cu.tolist() == want_cu.tolist() and slots.tolist() == want_slots.tolist()
        same_plan(c, p)
        if short:
            assert c.held.tolist() == [0, 1, 2, 1]
            with pytest.raises(RuntimeError, match="DFL_E_CAPACITY"):
                c.status()
    assert c.held.tolist() == [0, 2, 0, 1]
    c.status()


@pytest.mark.parametrize("heads,t", [((4, 2, 64), "bf16"), ((12, 1, 256), "fp16")])
def test_prompts_come_in_while_others_decode(torch, heads, t):
    """As two steps each time: the prompt's rows with none of the others', then theirs with the prompt in its pages."""
    z = Server(torch, heads, 3, 40, 16, t, 100, 6)
    z.step(np.array([50, 0, 33]), True, np.array([50, 0, 33]))
    for i, n in enumerate((70, 100, 1)):
        z.step(np.array([0, n, 0]), True, np.array([0, n, 0]))
        held = z.layers[0].held.tolist()
        assert held == [-(-int(x) // 16) for x in z.length]
        z.step(np.array([3, 0, 8]), False, np.array([3, 0, 5]))
        z.step(np.array([1, 4, 1]), False, np.array([1, 2, 0]))
        z.end(1)
    z.step(np.array([2, 0, 1]), False, np.array([2, 0, 1]))
    assert z.layers[0].held[1] == 0


# ---- values at the type's end --------------------------------------------------------------------------------------
@pytest.mark.parametrize("heads", [(4, 2, 64), (2, 1, 128), (12, 1, 256)])
@pytest.mark.parametrize("value", [65504.0, -65504.0])
def test_the_largest_values_of_fp16(torch, heads, value):
    """Weights that are all rounded up by nearly half a step, and values that are all the type's largest number: so are the outputs. And where
    one value is infinite, what sees it is not finite."""
    n_q, n_kv, hd = heads
    scale = (1 - np.log2(1 + 2.0 ** -11 * 1.02)) / np.log2(np.e)       # a weight of 4 and a half step of its type, and some more, beside one of 8
    k = np.full((400, n_kv, hd), 0.0)
    k[1:, :, 0] = -1
    q = np.zeros((400, n_q, hd))
    q[..., 0] = 1
    make = lambda rng, n, *_: (q[:n], k[:n], np.full((n, n_kv, hd), value))  # noqa: E731
    p = ExactPrompts(torch, heads, [400], "fp16", make, scale=scale)
    assert (p.run() == value).all()
    p.put("v", 300, np.inf, 3)
    got, g = p.run(), n_q // n_kv
    assert not np.isfinite(got[300:, :g, 3]).any()
    got[300:, :g, 3] = value
    assert (got == value).all()
    for lens, rows, wide in (([390], 1, 0), ([390], 9, 0), ([1500], 9, 2000), ([1500], 16, 2000)):
        k = np.full((lens[0] + rows, n_kv, hd), 0.0)
        k[1:, :, 0] = -1
        many = lambda rng, n, n_q, n_kv, keys, hd: (q[:n], k, np.full((keys, n_kv, hd), value))  # noqa: E731
        a = ExactPages(torch, heads, lens, [rows], 16, "fp16", many, wide=wide)
        assert (a.run(rows, scale=scale) == value).all()
        a.put("v", 0, 200, np.inf, 3)
        got = a.run(rows, scale=scale)
        assert not np.isfinite(got[:, :g, 3]).any()
        got[:, :g, 3] = value
        assert (got == value).all()
        a.c.status()


# ---- calls that nothing else makes -----------------------------------------------------------------------------------
def test_a_graph_after_the_scratch_has_grown(torch):
    """Two captured graphs and eager calls of one cache, one after another: a call of more rows brings a larger scratch, and the graph captured
    before goes on with its own."""
    lens, few = [700, 90], i32(torch, [0, 1, 2])
    p = Pages(torch, (12, 1, 256), lens, [16, 16], 16, "bf16", seed=3, wide=2000)
    want, tol = p.want(0, True, 1 / 16)
    first = torch.stack([p.q[0], p.q[16]]).contiguous()          # each sequence's first row
    calls = [(first, few, i32(torch, lens), 1), (p.q, i32(torch, p.cu), i32(torch, lens), 16)]
    wants = [(want[[0, 16]], tol[[0, 16]]), (want, tol)]
    outs, graphs = [torch.full_like(c[0], -77.0) for c in calls], []
    torch.cuda.synchronize()
    for c, out in zip(calls, outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            p.c.attn(*c, out=out)
        graphs.append(g)
    for turn in (0, 1, 0, 1):
        for out in outs:
            out.fill_(-77.0)
        graphs[turn].replay()
        p.c.attn(*calls[1 - turn], out=outs[1 - turn])
        for out, (w, t) in zip(outs, wants):
            near(out.double().cpu().numpy(), w, t)
    p.c.status()


@pytest.mark.parametrize("heads", [(4, 2, 64), (12, 1, 256)])
def test_rows_before_the_first_sequence(torch, heads):
    """Sequences that begin behind the buffers' first rows, which are left as they were."""
    p, a = Prompts(torch, heads, [5, 60, 0, 33], "bf16"), Pages(torch, heads, [5, 100, 40], [5, 3, 2], 16, "bf16")
    for x, rows in ((p, None), (a, 3)):
        x.cu = np.array([5, *x.cu[2:]])
        if x is p:
            x.lens, x.c = x.lens[1:], cache(torch, 3, heads[1], heads[2])
        else:
            full = x.c
            x.lens, x.counts, x.k64, x.v64 = x.lens[1:], x.counts[1:], x.k64[1:], x.v64[1:]
            from dflash_speculative_decode_gb300 import PagedCache
            x.c = PagedCache(full.k, full.v, full.table[1:].contiguous(), full.held[1:].contiguous(), full.free, full.queue)
        x.check() if rows is None else x.check(rows)


@pytest.mark.parametrize("heads", [(1024, 1024, 64), (2048, 1024, 64), (4096, 256, 64)])
def test_very_many_heads(torch, heads):
    Prompts(torch, heads, [9, 3], "bf16").check()
    p = Pages(torch, heads, [5, 150], [1, 3], 16, "fp16", wide=300)
    p.check(3)
    p.check(16, window=40)
