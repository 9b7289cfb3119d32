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
