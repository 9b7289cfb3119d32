"""The engine with the full layers' planes in 8 bits (dfl_config.kv8): speculative decode in lockstep with the oracle, whose
full planes are rounded to the same codes, block by block, before the pass that follows their commit."""
import numpy as np
import pytest

import gen
import oracle
from kv8_plain import BLOCK, quantise

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def weights():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from dflash_speculative_decode_gb300 import build
    build.build()
    return {name: (pc, gen.generate(pc)) for name, pc in (("tiny", gen.tiny_pair()), ("tiny-shared", gen.tiny_shared_pair()))}


def round_planes(target):
    """Every complete block of committed rows of the full layers' planes, in the values of its codes."""
    c = target.cfg
    for l, plane in target.planes.items():
        if c.layer_type[l] != gen.FULL:
            continue
        nkv, hd = c.kv_heads[l], c.head_dim
        rows = plane.reshape(-1, 2 * nkv, hd)
        for b in range(target.n // BLOCK):
            for h in range(2 * nkv):
                x = rows[BLOCK * b:BLOCK * (b + 1), h]
                codes, scale = quantise(x)
                x[:] = codes.astype(np.float32) * scale


def oracle_pair(pc, W):
    op = oracle.Pair(pc, W)
    forward = op.target.forward

    def rounded(tokens, head_rows=None):
        round_planes(op.target)
        return forward(tokens, head_rows)

    op.target.forward = rounded
    # a position's result depends on how its pass was cut (a pass sees its own rows unrounded): prompts in the engine's passes
    prefill = op.prefill
    op.prefill = lambda tokens, sampler, chunk=16: prefill(tokens, sampler, chunk=16)
    return op


def engine(pc, W):
    from dflash_speculative_decode_gb300 import Engine, config_from_pair
    eng = Engine(config_from_pair(pc, kv8=1))
    eng.load(W)
    return eng


@pytest.mark.parametrize("name,prompt,temperature", [("tiny", 5, None), ("tiny", 100, None), ("tiny", 63, 0.8), ("tiny-shared", 100, None),
                                                     ("tiny-shared", 37, 0.8)])
def test_lockstep_with_rounded_planes(weights, name, prompt, temperature):
    from gpu_harness import lockstep
    pc, W = weights[name]
    res, _ = lockstep(pc, W, gen.prompt(pc.target.vocab, prompt), 60, p=0.3, temperature=temperature, eng=engine(pc, W), op=oracle_pair(pc, W))
    assert res.passes > 10


def test_snapshot_restores_the_planes(weights):
    """A pinned prefix, requests A, B, A: the second A repeats the first, and lockstep holds on the restored prefix."""
    from dflash_speculative_decode_gb300 import DflError, spec_decode
    from gpu_harness import lockstep
    pc, W = weights["tiny"]
    eng, op = engine(pc, W), oracle_pair(pc, W)
    prefix = gen.prompt(pc.target.vocab, 80, request=5)
    eng.dfl_prefill(prefix)
    op.prefill(prefix, oracle.Sampler())
    snap, snap_o = eng.dfl_snapshot(), op.snapshot()
    got = []
    for request in (1, 2, 1):
        eng.dfl_restore(snap)
        got.append(spec_decode(eng, gen.prompt(pc.target.vocab, 9, request=request), 40).tokens)
    assert got[0] == got[2] and got[0] != got[1]
    eng.dfl_restore(snap)
    op.restore(snap_o)
    lockstep(pc, W, gen.prompt(pc.target.vocab, 9, request=1), 40, eng=eng, op=op)
    with pytest.raises(DflError):
        eng.dfl_debug_read("k3", (16,), np.float32)


def test_graphs_and_single_launches_agree(weights):
    from dflash_speculative_decode_gb300 import DFL_OPT_GRAPHS, spec_decode
    pc, W = weights["tiny-shared"]
    prompt = gen.prompt(pc.target.vocab, 70)
    tokens = []
    for graphs in (1, 0):
        eng = engine(pc, W)
        eng.dfl_set_option(DFL_OPT_GRAPHS, graphs)
        tokens.append(spec_decode(eng, prompt, 50).tokens)
    assert tokens[0] == tokens[1]
