"""CPU: the bound that the GPU test holds the attention to is below what a missing half costs."""
import numpy as np
import pytest

from kv8_halves import CTX, KINDS, attend, inputs
from kv8_plain import Head


@pytest.mark.parametrize("hd", [64, 128, 256])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("heads,rows", [(2, 1), (4, 1), (8, 1), (4, 4), (16, 2)])
def test_a_missing_half_is_seen(hd, kind, heads, rows):
    k, v, q = inputs(kind, hd, heads, rows, seed=hd + heads)
    m = Head(8)
    m.write(0, k[:CTX], v[:CTX], True)
    m.write(CTX, k[CTX:], v[CTX:], False)
    keys, values = m.rows(CTX + rows)
    worst = []
    for r in range(rows):
        for h in range(heads):
            n = CTX + r + 1
            want, tol = attend(q[r, h], keys[:n], values[:n], CTX)
            got, _ = attend(q[r, h], keys[:n], values[:n], CTX, drop=kind)
            worst.append((np.abs(got - want) / tol).max())
    assert min(worst) > 1.25, worst
