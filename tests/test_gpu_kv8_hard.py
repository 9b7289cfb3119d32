"""The 8-bit cache where its own sums, checks and masks can go wrong."""
import numpy as np
import pytest

from test_gpu_kv8 import Pair, torch  # noqa: F401  (torch is a fixture)

pytestmark = pytest.mark.gpu


# ---- rows behind the last one -----------------------------------------------------------------------------
@pytest.mark.parametrize("hd", [64, 128, 256])
@pytest.mark.parametrize("seqs", [2, 170])
def test_query_rows_behind_the_last_one_need_no_memory(torch, hd, seqs):  # noqa: F811
    """The queries end with the last sequence's last row that counts: what would lie behind it is another tensor's."""
    p = Pair(torch, seqs, 1, hd, 4, seed=hd)
    p.write(70)
    n = p.write(16, cnt=p.rng.integers(0, 17, seqs), commit=False)
    n[-1] = 3
    q, length, cnt = p.dev(p.new_rows(16, 4)), p.dev(p.len), p.dev(n)
    want = p.c.attn(q, length, cnt)
    held = torch.empty((seqs - 1) * 16 + 3, 4, hd, device="cuda")       # the end of an allocation of its own
    held.copy_(q.reshape(-1, 4, hd)[:len(held)])
    out = torch.zeros_like(q)
    need = p.c.L.dfl_kv8_attn_scratch_bytes(p.c._c, 4, 16, 0, 0)
    scratch = torch.empty(need, dtype=torch.uint8, device="cuda")
    rc = p.c.L.dfl_kv8_attn(p.c._c, held.data_ptr(), 4 * hd, 4, 16, length.data_ptr(), cnt.data_ptr(), 0, 1, hd ** -0.5, 0, out.data_ptr(), 4 * hd,
                            scratch.data_ptr(), need, torch.cuda.current_stream().cuda_stream)
    assert rc == 0
    p.c.status()
    assert torch.equal(out, want)


# ---- values that a row does not see -----------------------------------------------------------------------
@pytest.mark.parametrize("hd", [64, 128, 256])
@pytest.mark.parametrize("n_q,rows", [(2, 1), (4, 1), (2, 4), (4, 4), (16, 2)])     # 2, 4, 8, 16 and 32 rows a head
@pytest.mark.parametrize("seqs,sizes", [(1, (20, 40, 100)), (160, (40,))])
def test_masked_values_of_any_size_cost_nothing(torch, hd, n_q, rows, seqs, sizes):  # noqa: F811
    """A value far larger than the others just before the window's edge, inside the first block that rows see, and one that only row 0
    sees: the others' outputs are held to the bound of what they see."""
    for size in sizes:
        p = Pair(torch, seqs, 1, hd, 12, seed=hd + rows)
        k, v = p.new_rows(300), p.new_rows(300)
        v[:, 140] *= np.float32(2.0 ** size)     # row m of a window of 150 sees tokens 151 + m .. 300 + m
        p.write(300, k=k, v=v)
        p.write(rows, commit=False)
        p.attn(n_q, rows, window=150)
        p.attn(n_q, rows, window=150, causal=False)
        p = Pair(torch, seqs, 1, hd, 12, seed=hd + rows + 1)
        v[:, 140], v[:, 151] = p.new_rows(1)[:, 0], v[:, 151] * np.float32(2.0 ** size)
        p.write(300, k=k, v=v)
        p.write(rows, commit=False)
        p.attn(n_q, rows, window=150)


# ---- scores where values are not finite ----------------------------------------------------------------------
@pytest.mark.parametrize("hd", [64, 256])
@pytest.mark.parametrize("n_q,rows", [(2, 1), (4, 4), (16, 2)])
def test_scores_are_weights_whatever_the_values(torch, hd, n_q, rows):  # noqa: F811
    """Weights come from queries and keys: a value that is not finite, in a block or in the tail, makes the rows that see it NaN and leaves
    what the blocks' scores get as it is."""
    for at in (41, 198, None):
        p = Pair(torch, 2, 1, hd, 10, seed=hd + rows)
        k, v = p.new_rows(200), p.new_rows(200)
        if at is not None:
            v[0, at, 0, 9] = np.nan if at == 41 else np.inf
        p.write(200, k=k, v=v)
        vs = p.new_rows(rows)
        if at is None:
            vs[0, 0, 0, hd - 1] = np.nan
        p.write(rows, commit=False, v=vs)
        p.c.score.zero_()
        q = p.new_rows(rows, n_q)
        out = p.c.attn(p.dev(q), p.dev(p.len), score=True).cpu().numpy()
        p.c.status()
        assert np.isnan(out[0]).all() and np.isfinite(out[1]).all()
        got = p.c.score.cpu().numpy()
        for s in range(2):
            with np.errstate(invalid="ignore"):
                _, _, add, bound = p.heads[s][0].attn(q[s], 200, rows, 0, True, hd ** -0.5)
            assert (np.abs(got[s, 0] - add) <= bound + 2.0 ** -23 * add).all()


# ---- table entries out of range ---------------------------------------------------------------------------
@pytest.mark.parametrize("odd", [0, 1])
@pytest.mark.parametrize("rows,commit", [(5, False), (40, True), (150, True)])
def test_a_head_left_behind_is_met_alike_in_every_batch(torch, odd, rows, commit):  # noqa: F811
    """A bad entry keeps one head of a sequence from going on with the other. Attention then leaves what differs from the first head,
    however many sequences there are, and attends the others."""
    from dflash_speculative_decode_gb300 import DflError, _abi
    left = []
    for seqs in (2, 90):
        p = Pair(torch, seqs, 2, 64, 12, seed=rows)
        p.write(32)
        for _ in range(2):
            p.write(16, commit=False)
            p.len = p.len + 16                  # 32 rows of the tail are committed: the next call seals block 1
        table = p.c.table.clone()
        p.c.table[1, odd, 1] = 12
        with pytest.raises(DflError) as e:
            p.write(rows, commit=commit)
        assert e.value.code == _abi.DFL_E_INVALID_ARG
        z = (64 + rows) // 32 if commit else 2
        assert p.c.sealed[1, odd] == 1 and p.c.sealed[1, 1 - odd] == z and (p.c.sealed[0] == z).all()
        p.c.table.copy_(table)
        length = p.dev(p.len + (rows if commit else 0))
        q, n = p.dev(p.new_rows(5, 4)), p.dev(np.full(seqs, 5 if not commit else 0, np.int32))
        if commit:
            n[:] = 1
        out = torch.full_like(q, 9.0)
        p.c.attn(q, length, n, out=out)         # (after an append the row staged is whatever the tail holds)
        with pytest.raises(DflError) as e:
            p.c.status()
        assert e.value.code == _abi.DFL_E_STATE
        left.append([[bool((out[s, 0, 2 * h:2 * h + 2] == 9.0).all()) for h in range(2)] for s in range(2)])
    assert left[0] == left[1]
    assert left[0][0] == [False, False] and left[0][1][1]      # the sequence beside it, and the head that is not the first one's like
    assert left[0][1][0] == (odd == 0 and commit)   # the first head: left only where its tail does not reach so far


def test_read_looks_at_the_blocks_of_its_range_only(torch):  # noqa: F811
    from dflash_speculative_decode_gb300 import DflError, _abi
    p = Pair(torch, 1, 2, 64, 8, seed=5)
    p.write(160)
    table = p.c.table.clone()
    length = p.dev(p.len)
    for first, rows, bad, hit in ((0, 64, 2, False), (0, 64, 3, False), (0, 65, 2, True), (33, 31, 2, False), (33, 31, 0, False), (33, 32, 2, True),
                                  (70, 20, 4, False), (40, 8, 2, False)):
        p.c.table.copy_(table)
        p.c.table[0, 1, bad] = 99
        got = p.c.read(length, rows, first=p.dev(np.array([first], np.int32)))
        if hit:
            with pytest.raises(DflError) as e:
                p.c.status()
            assert e.value.code == _abi.DFL_E_INVALID_ARG
        else:
            p.c.status()
            for x, want in zip(got, p.heads[0][1].rows(160)):
                np.testing.assert_array_equal(x[0, :, 1].cpu().numpy(), want[first:first + rows].astype(np.float32))


# ---- refusals that repeat -----------------------------------------------------------------------------------
def test_a_refused_shape_is_refused_the_same_way_again(torch):  # noqa: F811
    from dflash_speculative_decode_gb300 import DflError
    p = Pair(torch, 1, 2, 64, 4, seed=6)
    p.write(40)
    said = []
    for q, window in ((p.new_rows(17, 2), 0), (p.new_rows(1, 3), 0), (p.new_rows(1, 2), -1)):
        for _ in range(2):
            with pytest.raises(DflError) as e:
                p.c.attn(p.dev(q), p.dev(p.len), window=window)
            said.append((e.value.code, str(e.value)))
        assert said[-1] == said[-2]


def test_a_call_that_found_no_memory_for_its_scratch_can_be_made_again(torch):  # noqa: F811
    class Full:
        def __getattr__(self, name):
            return getattr(torch, name)

        def empty(self, *args, **kw):
            raise torch.cuda.OutOfMemoryError("none left")
    p = Pair(torch, 2, 2, 64, 8, seed=7)
    p.write(100)
    p.write(3, commit=False)
    p.attn(4, 1)
    p.c.torch = Full()
    with pytest.raises(torch.cuda.OutOfMemoryError):
        p.attn(32, 3)
    p.c.torch = torch
    p.attn(32, 3)
