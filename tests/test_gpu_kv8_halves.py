"""Both fp16 halves of queries and of weights take part in the attention over the 8-bit cache, at every head size and number of rows, in
splits and in shares: outputs are held to a bound that a missing half would pass (test_kv8_halves_host.py)."""
import numpy as np
import pytest

from kv8_halves import CTX, KINDS, attend, inputs
from kv8_plain import Head
from test_gpu_kv8 import torch  # noqa: F401  (a fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("hd", [64, 128, 256])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("heads,rows", [(2, 1), (4, 1), (8, 1), (4, 4), (16, 2)])
@pytest.mark.parametrize("seqs", [1, 160])
def test_no_half_is_missing(torch, hd, kind, heads, rows, seqs):  # noqa: F811
    from dflash_speculative_decode_gb300 import Kv8Cache
    k, v, q = inputs(kind, hd, heads, rows, seed=hd + heads)
    c = Kv8Cache.empty(seqs, 1, hd, 8)
    dev = lambda x: torch.from_numpy(np.broadcast_to(x, (seqs, *x.shape)).copy()).cuda()  # noqa: E731
    length = torch.zeros(seqs, dtype=torch.int32, device="cuda")
    c.append(dev(k[:CTX, None]), dev(v[:CTX, None]), length)
    length += CTX
    c.stage(dev(k[CTX:, None]), dev(v[CTX:, None]), length)
    out = c.attn(dev(q), length)
    c.status()
    assert torch.allclose(out, out[:1].expand_as(out), rtol=0, atol=1e-4)     # the sequences are alike, their cuts are not
    m = Head(8)
    m.write(0, k[:CTX], v[:CTX], True)
    m.write(CTX, k[CTX:], v[CTX:], False)
    keys, values = m.rows(CTX + rows)
    got = out.cpu().numpy()
    for r in range(rows):
        for h in range(heads):
            want, tol = attend(q[r, h], keys[:CTX + r + 1], values[:CTX + r + 1], CTX)
            err = np.abs(got[:, r, h] - want)
            assert (err <= tol).all(), f"row {r} head {h}: off by {(err / tol).max():.3g} of the bound"
