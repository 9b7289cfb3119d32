"""The paged key/value cache's attentions where they can go wrong, against derived bounds (tests/paged_bounds.py)."""
import numpy as np
import pytest

from paged_bounds import attend_exact, far, lifted
from test_gpu_paged import Prompts, torch  # noqa: F401  (torch: the fixture)

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
