"""CPU: what the dfl_kv8 calls refuse before anything reaches a device, and the plain model that the GPU tests use."""
import ctypes

import numpy as np
import pytest

from dflash_speculative_decode_gb300 import _abi
from kv8_plain import BLOCK, Head, quantise

A = 1 << 20          # an aligned address that nothing reads


def cache(**change):
    f = dict(n_seq=2, n_kv=2, head_dim=64, n_blocks=8, k=A, v=A, k_scale=A, v_scale=A, k_tail=A, v_tail=A, table=A, sealed=A, score=A, err=A)
    f.update(change)
    return _abi.dfl_kv8(**f)


def calls(c, L):
    """Every call with arguments that it takes, by name."""
    r = ctypes.byref(c)
    return {
        "init": lambda **k: L.dfl_kv8_init(r, None),
        "append": lambda **k: L.dfl_kv8_append(r, k.get("len", A), None, k.get("rows", 4), k.get("k", A), k.get("v", A), k.get("ld", 128), None),
        "stage": lambda **k: L.dfl_kv8_stage(r, k.get("len", A), None, k.get("rows", 4), k.get("k", A), k.get("v", A), k.get("ld", 128), None),
        "attn": lambda **k: L.dfl_kv8_attn(r, k.get("q", A), k.get("ldq", 256), k.get("n_q", 4), k.get("rows", 4), k.get("len", A), None,
                                           k.get("window", 0), 1, k.get("scale", 0.125), k.get("score", 0), k.get("out", A), k.get("ldo", 256),
                                           k.get("scratch", A), k.get("bytes", 1 << 40), None),
        "evict": lambda **k: L.dfl_kv8_evict(r, k.get("len", A), k.get("keep", 4), k.get("sink", 1), k.get("recent", 1), k.get("table", 2 * A),
                                             k.get("score", 3 * A), k.get("sealed", 4 * A), k.get("len_out", 5 * A), None),
        "read": lambda **k: L.dfl_kv8_read(r, k.get("len", A), None, k.get("rows", 4), k.get("k", A), k.get("v", A), None),
    }


@pytest.mark.parametrize("change,code", [
    (dict(n_seq=0), -1), (dict(n_seq=65536), -1), (dict(n_kv=0), -1), (dict(n_kv=1025), -1), (dict(n_blocks=0), -1), (dict(n_blocks=(1 << 20) + 1), -1),
    (dict(head_dim=96), -4), (dict(head_dim=512), -4), (dict(head_dim=0), -4), (dict(k=None), -1), (dict(v=A + 8), -1), (dict(k_scale=None), -1),
    (dict(v_scale=A + 4), -1), (dict(k_tail=None), -1), (dict(v_tail=A + 4), -1), (dict(table=None), -1), (dict(sealed=None), -1), (dict(err=None), -1),
    (dict(score=A + 4), -1)])
def test_a_bad_cache_is_refused_by_every_call(change, code):
    L = _abi.lib()
    for name, call in calls(cache(**change), L).items():
        assert call() == code, name
    assert L.dfl_kv8_status(ctypes.byref(cache(**change)), None) == code


@pytest.mark.parametrize("name,args,code", [
    ("append", dict(len=None), -1), ("append", dict(rows=0), -1), ("append", dict(rows=-1), -1), ("append", dict(rows=257), -3), ("append", dict(k=None), -1),
    ("append", dict(v=A + 4), -1), ("append", dict(ld=124), -1), ("append", dict(ld=130), -1), ("append", dict(ld=-128), -1),
    ("stage", dict(len=None), -1), ("stage", dict(rows=17), -4), ("stage", dict(rows=0), -1), ("stage", dict(v=None), -1),
    ("attn", dict(q=None), -1), ("attn", dict(q=A + 4), -1), ("attn", dict(ldq=252), -1), ("attn", dict(ldo=255), -1), ("attn", dict(out=None), -1),
    ("attn", dict(n_q=3), -1), ("attn", dict(n_q=0), -1), ("attn", dict(n_q=34, ldq=4096, ldo=4096), -4), ("attn", dict(rows=0), -1), ("attn", dict(rows=17), -4),
    ("attn", dict(window=-1), -1), ("attn", dict(len=None), -1), ("attn", dict(scale=float("inf")), -1), ("attn", dict(scale=float("nan")), -1),
    ("attn", dict(scratch=None), -1), ("attn", dict(scratch=A + 16), -1), ("attn", dict(bytes=0), -1),
    ("evict", dict(len=None), -1), ("evict", dict(keep=-1), -1), ("evict", dict(sink=-1), -1), ("evict", dict(recent=-1), -1), ("evict", dict(sink=3, recent=2), -1),
    ("evict", dict(sink=1 << 30, recent=1 << 30, keep=(1 << 31) - 1), -1), ("evict", dict(table=None), -1), ("evict", dict(score=None), -1),
    ("evict", dict(sealed=None), -1), ("evict", dict(len_out=None), -1), ("evict", dict(table=A), -1), ("evict", dict(score=A), -1),
    ("evict", dict(sealed=A), -1), ("evict", dict(len_out=A), -1),
    ("read", dict(len=None), -1), ("read", dict(rows=0), -1), ("read", dict(k=None), -1), ("read", dict(v=A + 4), -1)])
def test_bad_arguments_are_refused(name, args, code):
    if name == "evict" and args.get("keep") == (1 << 31) - 1:
        args = dict(args, keep=(1 << 31) - 2)
        args["sink"] = args["recent"] = 1 << 30      # their sum passes 31 bits
    assert calls(cache(), _abi.lib())[name](**args) == code


def test_scores_need_a_cache_that_keeps_them():
    L = _abi.lib()
    c = cache(score=None)
    assert calls(c, L)["attn"](score=1) == -1
    assert calls(c, L)["evict"]() == -1
    assert L.dfl_kv8_attn_scratch_bytes(ctypes.byref(cache()), 4, 8, 0, 1) > 0


@pytest.mark.parametrize("n_q,rows,window", [(3, 1, 0), (0, 1, 0), (4, 0, 0), (4, 17, 0), (34, 1, 0), (4, 1, -1)])
def test_scratch_of_shapes_it_does_not_take(n_q, rows, window):
    assert _abi.lib().dfl_kv8_attn_scratch_bytes(ctypes.byref(cache()), n_q, rows, window, 0) == -1


def test_constants():
    import os
    import re

    from dflash_speculative_decode_gb300 import kv8
    src = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "dfl.h")).read()
    got = dict(re.findall(r"#define (DFL_KV8_[A-Z]+) (\d+)", src))
    assert (int(got["DFL_KV8_BLOCK"]), int(got["DFL_KV8_TAIL"])) == (kv8.BLOCK, kv8.TAIL)


def test_the_binding_refuses_tensors_off_the_gpu():
    torch = pytest.importorskip("torch")
    from dflash_speculative_decode_gb300 import DflError, Kv8Cache
    z = torch.zeros
    ok = dict(k=z(1, 1, 2, 1, 32, 64, dtype=torch.uint8), v=z(1, 1, 2, 64, 32, dtype=torch.uint8), k_scale=z(1, 1, 2), v_scale=z(1, 1, 2),
              k_tail=z(1, 1, 48, 64), v_tail=z(1, 1, 64, 48), table=z(1, 1, 2, dtype=torch.int32), sealed=z(1, 1, dtype=torch.int32), score=z(1, 1, 2))
    with pytest.raises(DflError):
        Kv8Cache(**ok)
    for name, t in (("k", z(1, 1, 2, 32, 64, dtype=torch.uint8)), ("v", z(1, 1, 2, 32, 64, dtype=torch.uint8)), ("table", z(1, 1, 2)), ("sealed", z(1, 2, dtype=torch.int32)),
                    ("k_tail", z(1, 1, 64, 48)), ("score", z(1, 1, 3))):
        with pytest.raises(DflError, match=name):
            Kv8Cache(**dict(ok, **{name: t}))


# ---- the plain model ------------------------------------------------------------------------------------
def test_plain_codes():
    x = np.zeros((32, 64), np.float32)
    x[0, :5] = [127.0, 0.5, 1.5, -2.5, -126.5]
    c, s = quantise(x)
    assert s == 1 and list(c[0, :5]) == [127, 0, 2, -2, -126]
    x[1, 1] = np.inf
    assert np.isnan(quantise(x)[1]) and not quantise(x)[0].any()
    assert quantise(np.zeros((32, 64)))[1] == 0


def test_plain_head_seals_and_cuts():
    rng = np.random.default_rng(0)
    h = Head(8)
    rows = rng.standard_normal((100, 64)).astype(np.float32)
    h.write(0, rows[:70], rows[:70], True)
    assert len(h.blocks) == 2 and len(h.tail_k) == 6
    h.write(70, rows[:16], rows[:16], False)
    h.write(86, rows[:16], rows[:16], False)         # all 16 committed: nothing complete yet (22 rows)
    assert len(h.blocks) == 2 and len(h.tail_k) == 38
    h.write(102, rows[:3], rows[:3], False)          # 38 rows committed: one block sealed
    assert len(h.blocks) == 3 and len(h.tail_k) == 9
    h.write(40, rows[:1], rows[:1], False)
    assert len(h.blocks) == 1 and len(h.tail_k) == 9
    k, _ = h.rows(41)
    assert k.shape == (41, 64) and np.abs(k[:40] - rows[:40]).max() <= np.abs(rows).max() / 254 * 1.001
    assert (BLOCK, h.evict(0, 0, 0)) == (32, ([], 1))


# ---- planes in 8 bits (dfl_config.kv8) --------------------------------------------------------------------
def test_planes_in_8_bits_take_a_quarter_of_the_state():
    import gen
    L, sz = _abi.lib(), _abi.dfl_sizes()
    got = []
    for kv8 in (0, 1):
        cfg = _abi.config_from_pair(gen.e4b_pair(max_ctx=1 << 17), kv8=kv8)
        assert L.dfl_required_bytes(ctypes.byref(cfg), ctypes.byref(sz)) == 0
        got.append(sz.state_bytes)
    full = sum(1 for l in range(24) if gen.e4b_target().layer_type[l] == gen.FULL)
    plane = full * 2 * 2 * 256 * (1 << 17)                 # values of the full owners' planes
    assert 0.99 * 3 * plane < got[0] - got[1] < 3 * plane


def test_planes_in_8_bits_that_are_refused():
    import gen
    L, sz = _abi.lib(), _abi.dfl_sizes()
    cfg = _abi.config_from_pair(gen.tiny_pair(), prefill_rows=128, kv8=1)
    assert L.dfl_required_bytes(ctypes.byref(cfg), ctypes.byref(sz)) == _abi.DFL_E_INVALID_ARG
    for kv8 in (2, -1):
        cfg = _abi.config_from_pair(gen.tiny_pair(), kv8=kv8)
        assert L.dfl_required_bytes(ctypes.byref(cfg), ctypes.byref(sz)) == _abi.DFL_E_INVALID_ARG
    cfg = _abi.config_from_pair(gen.tiny_pair(), kv8=1)
    cfg.n_heads = 64                                       # 32 query heads a key/value head of the full layer
    assert L.dfl_required_bytes(ctypes.byref(cfg), ctypes.byref(sz)) == _abi.DFL_E_INVALID_ARG


def test_evictions_outputs_overlap_nothing():
    """c is 2 x 2 heads of 8 blocks: 128 bytes of table and of scores, 16 of sealed counts; len and len_out 8."""
    L = _abi.lib()
    evict = calls(cache(table=10 * A, score=11 * A, sealed=12 * A, err=13 * A), L)["evict"]
    for args in (dict(table=10 * A + 64), dict(table=10 * A - 64), dict(score=11 * A + 124), dict(sealed=12 * A + 12), dict(len_out=A + 4), dict(len_out=A - 4),
                 dict(table=11 * A), dict(score=10 * A + 4), dict(sealed=A), dict(len_out=13 * A), dict(score=2 * A + 124), dict(sealed=2 * A + 64),
                 dict(len_out=4 * A + 8)):
        assert evict(**args) == -1, args
