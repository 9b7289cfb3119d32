"""An engine with its full layers' planes in 8 bits: what it reports, counts and stores."""
import numpy as np
import pytest

import gen

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def weights():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from dflash_speculative_decode_gb300 import build
    build.build()
    return {name: (pc, gen.generate(pc)) for name, pc in (("tiny", gen.tiny_pair()), ("tiny-shared", gen.tiny_shared_pair()))}


def engine(pc, W, kv8=1):
    from dflash_speculative_decode_gb300 import Engine, config_from_pair
    eng = Engine(config_from_pair(pc, kv8=kv8))
    eng.load(W)
    return eng


def owner_heads(pc):
    """Key/value heads of the planes held in 8 bits."""
    t = pc.target
    return sum(t.kv_heads[l] for l in range(t.n_layers) if t.layer_type[l] == gen.FULL and t.kv_owner[l] == l)


@pytest.mark.parametrize("name", ["tiny", "tiny-shared"])
@pytest.mark.parametrize("bad", [1 << 20, -1])
def test_a_plane_out_of_order_is_reported(weights, name, bad):
    """A snapshot whose sealed counts are out of range: the next pass raises instead of returning tokens, and so do all calls until a
    sound snapshot is restored. The counts are found as the words that go from 1 to 2 when the next stage seals the second block."""
    from dflash_speculative_decode_gb300 import DflError
    from dflash_speculative_decode_gb300._abi import DFL_E_STATE
    pc, W = weights[name]
    eng = engine(pc, W)
    rows = [int(t) for t in gen.prompt(pc.target.vocab, 8, request=2)]
    eng.dfl_prefill(gen.prompt(pc.target.vocab, 64))
    before = eng.dfl_snapshot()
    eng.dfl_verify_block(rows)
    eng.dfl_commit_verify_rows(0)
    snap = eng.dfl_snapshot()
    words = [x[:x.numel() // 4 * 4].cpu().numpy().view(np.int32) for x in (before, snap)]
    at = np.nonzero((words[0] == 1) & (words[1] == 2))[0]
    assert len(at) == owner_heads(pc)
    want = eng.dfl_verify_block(rows)
    eng.dfl_commit_verify_rows(0)
    spoilt = words[1].copy()
    spoilt[at] = bad
    broken = snap.clone()
    broken[:4 * len(spoilt)] = eng.torch.from_numpy(spoilt.view(np.uint8)).to(broken.device)
    for call in (lambda: eng.dfl_verify_block(rows), lambda: eng.dfl_prefill(rows)):
        eng.dfl_restore(broken)
        with pytest.raises(DflError) as e:
            call()
        assert e.value.code == DFL_E_STATE
        for again in (lambda: eng.dfl_verify_block(rows), lambda: eng.dfl_prefill(rows), lambda: eng.dfl_snapshot()):
            with pytest.raises(DflError) as e:
                again()
            assert e.value.code == DFL_E_STATE
        eng.dfl_restore(snap)
        got = eng.dfl_verify_block(rows)
        eng.dfl_commit_verify_rows(0)
        assert list(got[0]) == list(want[0]) and got[1] == want[1]


def test_snapshots_hold_what_is_held(weights):
    """What a snapshot takes for planes in 8 bits goes by the positions held, not by those that the engine could hold, and is below what
    fp32 planes take; one taken at any position restores into a used context."""
    from dataclasses import replace
    pc, W = weights["tiny"]
    t, prompt = pc.target, gen.prompt(pc.target.vocab, 150)
    rows = [int(x) for x in gen.prompt(t.vocab, 8, request=2)]
    engines = [(engine(p, W), engine(p, W, kv8=0)) for p in (pc, replace(pc, max_ctx=4096))]
    full = [l for l in range(t.n_layers) if t.layer_type[l] == gen.FULL]
    heads = sum(t.kv_heads[l] for l in full)
    for n in (0, 1, 32, 33, 100, 150):
        planes = []
        for pair in engines:
            if n:
                for eng in pair:
                    eng.dfl_prefill(prompt[eng.dfl_positions_held():n])
            planes.append(pair[0].dfl_snapshot_bytes() - pair[1].dfl_snapshot_bytes() + 2 * heads * t.head_dim * 4 * n)
        # keys and values: codes of the blocks that positions lie in, a scale each, 48 rows in fp32, the sealed counts
        blocks = -(-n // 32)
        assert planes == [2 * heads * (blocks * (32 * t.head_dim + 4) + 48 * t.head_dim * 4) + 4 * heads] * 2, n
        eng = engines[1][0]
        snap = eng.dfl_snapshot()
        want = eng.dfl_verify_block(rows)
        eng.dfl_commit_verify_rows(8)
        eng.dfl_prefill(gen.prompt(t.vocab, 70, request=9))
        eng.dfl_restore(snap)
        assert eng.dfl_positions_held() == n
        got = eng.dfl_verify_block(rows)
        eng.dfl_commit_verify_rows(0)
        assert list(got[0]) == list(want[0]) and got[1] == want[1]


@pytest.fixture(scope="module")
def wide():
    """A small target with the E4B pair's head layout: 12 query heads of 256 over 2 key/value heads in full layers, 1 in sliding ones."""
    from dataclasses import replace
    pc = gen.tiny_pair()
    pc = replace(pc, target=replace(pc.target, name="wide", n_heads=12, head_dim=256), max_ctx=512)
    return pc, gen.generate(pc)


@pytest.mark.parametrize("prompt,temperature", [(290, None), (95, 0.8)])
def test_lockstep_in_the_e4b_pairs_head_layout(wide, prompt, temperature):
    """Three groups of 16 rows a key/value head, up to eleven sealed blocks, against the oracle with planes rounded to the same codes."""
    from gpu_harness import lockstep
    from test_gpu_kv8_planes import oracle_pair
    pc, W = wide
    res, _ = lockstep(pc, W, gen.prompt(pc.target.vocab, prompt), 60, p=0.3, temperature=temperature, eng=engine(pc, W), op=oracle_pair(pc, W))
    assert res.passes > 10


def test_recovery_of_planes_in_8_bits(weights):
    """A prefill whose passes give up over held positions (a test option; no fault): the restored context is as one that never failed."""
    from dflash_speculative_decode_gb300 import DFL_OPT_KEEP_LOGITS, DflError
    from dflash_speculative_decode_gb300._abi import DFL_E_STATE, DFL_E_TIMEOUT, DFL_OPT_TEST_STALL
    pc, W = weights["tiny"]
    prompt, more = gen.prompt(pc.target.vocab, 90, request=31), gen.prompt(pc.target.vocab, 40, request=32)
    rows = [int(t) for t in gen.prompt(pc.target.vocab, 8, request=33)]
    a, b = engine(pc, W), engine(pc, W)
    for eng in (a, b):
        eng.dfl_set_option(DFL_OPT_KEEP_LOGITS, 1)
        eng.dfl_prefill(prompt)
    snap = a.dfl_snapshot()
    a.dfl_set_option(DFL_OPT_TEST_STALL, 1)
    with pytest.raises(DflError) as e:
        a.dfl_prefill(more)
    assert e.value.code == DFL_E_TIMEOUT and a.dfl_positions_held() == 90
    a.dfl_set_option(DFL_OPT_TEST_STALL, 0)
    with pytest.raises(DflError) as e:
        a.dfl_verify_block(rows)
    assert e.value.code == DFL_E_STATE
    a.dfl_restore(snap)
    got, want = a.dfl_verify_block(rows), b.dfl_verify_block(rows)
    np.testing.assert_array_equal(a.dfl_read_logits(0, 8), b.dfl_read_logits(0, 8))
    assert list(got[0]) == list(want[0]) and got[1] == want[1]
