"""CPU: the inputs of the paged attention's tests whose scores come without rounding."""
import numpy as np
import pytest

from paged_bounds import far, lifted, spiked


def rounded(x, t):
    import torch
    return torch.from_numpy(np.asarray(x, np.float32)).to({"bf16": torch.bfloat16, "fp16": torch.float16}[t]).float().numpy()


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
