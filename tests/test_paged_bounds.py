"""CPU: the bound that the paged attention's tests hold a kernel's weights to, on results worked out here: weights as two numbers of the type
are within it, weights rounded once, or with a second number of the wrong sign, are not."""
import numpy as np
import pytest

from paged_bounds import attend_exact, far, lifted, spiked


def rounded(x, t):
    import torch
    return torch.from_numpy(np.asarray(x, np.float32)).to({"bf16": torch.bfloat16, "fp16": torch.float16}[t]).float().numpy()


def kernel(q, k, v, first, scale, t, second):
    """Attention in fp32 with a weight as its rounding and `second` times what that left."""
    f = np.float32
    out = np.zeros(q.shape, f)
    g = q.shape[1] // k.shape[1]
    for m in range(q.shape[0]):
        for h in range(q.shape[1]):
            s = (k[:first + m + 1, h // g].astype(f) @ q[m, h].astype(f)).astype(f)
            e = np.exp2(((s - s.max()) * f(scale * 1.4426950408889634)).astype(f) + f(3 if t == "fp16" else 0)).astype(f)
            hi = rounded(e, t)
            w = hi + second * rounded(e - hi, t)
            out[m, h] = rounded((w @ v[:first + m + 1, h // g].astype(f)) / e.sum(dtype=f), t)
    return out


@pytest.mark.parametrize("t", ["bf16", "fp16"])
@pytest.mark.parametrize("heads,rows", [((4, 2, 64), 4), ((2, 1, 64), 8), ((12, 2, 128), 2), ((16, 1, 128), 1), ((12, 1, 256), 1), ((4, 2, 256), 7)])
@pytest.mark.parametrize("length", [33, 100, 600])
def test_a_missing_part_passes_the_bound(heads, rows, t, length):
    n_q, n_kv, hd = heads
    q, k, v = (rounded(x, t).astype(np.float64) for x in spiked(np.random.default_rng(length), rows, n_q, n_kv, length + rows, hd))
    want, tol = attend_exact(q, k, v, length, 0, True, hd ** -0.5, t, 2)
    assert (np.abs(kernel(q, k, v, length, hd ** -0.5, t, 1) - want) <= tol).all()
    for second in (0, -1):
        bad = np.abs(kernel(q, k, v, length, hd ** -0.5, t, second) - want) > tol
        assert bad.sum() >= 4 and bad.mean() > 0.002, (second, bad.mean())
    once, tol = attend_exact(q, k, v, length, 0, True, hd ** -0.5, t, 1)
    assert (np.abs(kernel(q, k, v, length, hd ** -0.5, t, 0) - once) <= tol).all()


@pytest.mark.parametrize("hd", [64, 128, 256])
def test_scores_come_without_rounding(hd):
    rng = np.random.default_rng(hd)
    for t, unit in (("fp16", 2.0 ** 28), ("bf16", 2.0 ** 60), ("fp16", 2.0 ** 14)):
        for q, k, v in (spiked(rng, 3, 4, 2, 400, hd), lifted(rng, 3, 4, 2, 400, hd, 2.0 ** 18), far(rng, 3, 4, 2, 400, hd, unit)):
            for x in (q, k):
                np.testing.assert_array_equal(rounded(x, t), x.astype(np.float32))
            terms = q[:, None, [0, 2]] * k[None]
            least = 2.0 ** np.floor(np.log2(np.abs(terms[terms != 0]).min()))
            while (terms % least).any():
                least /= 2
            assert np.abs(terms).sum(-1).max() < least * 2.0 ** 24
