"""CPU: what the dfl_paged calls refuse before anything reaches a device, and the plain model that the GPU tests use."""
import ctypes

import numpy as np
import pytest

from dflash_speculative_decode_gb300 import _abi
from paged_plain import Plan, attend

A = 1 << 20          # aligned addresses that nothing reads, far enough apart
B = [A * (i + 2) for i in range(12)]


def cache(**change):
    f = dict(n_seq=2, n_kv=2, head_dim=64, page=32, n_pages=8, max_pages=4, type=0, k=B[0], v=B[1], table=B[2], held=B[3], ring=B[4], queue=B[5], err=B[6])
    f.update(change)
    return _abi.dfl_paged(**f)


def calls(c, L):
    """Every call with arguments that it takes, by name."""
    r = ctypes.byref(c)
    return {
        "init": lambda **k: L.dfl_paged_init(r, None),
        "plan": lambda **k: L.dfl_paged_plan(r, k.get("len", A), k.get("cnt", A), k.get("cu", B[7]), k.get("slots", B[8]), k.get("rows", 4), None),
        "append": lambda **k: L.dfl_paged_append(r, k.get("slots", A), k.get("rows", 4), k.get("k", A), k.get("ldk", 128), k.get("v", A), k.get("ldv", 128), None),
        "prompt": lambda **k: L.dfl_paged_prompt(r, k.get("q", A), k.get("ldq", 256), k.get("n_q", 4), k.get("k", A), k.get("ldk", 128), k.get("v", A),
                                                 k.get("ldv", 128), k.get("cu", A), k.get("rows", 4), k.get("window", 0), k.get("scale", 0.125),
                                                 k.get("out", B[9]), k.get("ldo", 256), None),
        "attn": lambda **k: L.dfl_paged_attn(r, k.get("q", A), k.get("ldq", 256), k.get("n_q", 4), k.get("total", 4), k.get("cu", A), k.get("len", A),
                                             k.get("rows", 4), k.get("window", 0), 1, k.get("scale", 0.125), k.get("out", B[9]), k.get("ldo", 256),
                                             k.get("scratch", A), k.get("bytes", 1 << 40), None),
    }


@pytest.mark.parametrize("change,code", [
    (dict(n_seq=0), -1), (dict(n_seq=4097), -1), (dict(n_kv=0), -1), (dict(n_kv=1025), -1), (dict(n_pages=0), -1), (dict(max_pages=0), -1),
    (dict(n_pages=1 << 26, page=32), -1), (dict(max_pages=1 << 25, page=64), -1), (dict(n_pages=(1 << 25) + 1, page=32), -1),
    (dict(max_pages=(1 << 24) + 1, page=64), -1), (dict(head_dim=96), -4), (dict(head_dim=512), -4), (dict(page=0), -4),
    (dict(page=48), -4), (dict(page=256), -4), (dict(type=2), -4), (dict(type=-1), -4), (dict(k=None), -1), (dict(v=A + 8), -1), (dict(table=None), -1),
    (dict(held=A + 2), -1), (dict(ring=None), -1), (dict(queue=None), -1), (dict(err=None), -1)])
def test_a_bad_cache_is_refused_by_every_call(change, code):
    L = _abi.lib()
    for name, call in calls(cache(**change), L).items():
        assert call() == code, name
    assert L.dfl_paged_status(ctypes.byref(cache(**change)), None) == code
    for name, call in calls(cache(**change), L).items():
        assert call(rows=0, total=0) == code, name


@pytest.mark.parametrize("name,args,code", [
    ("plan", dict(len=None), -1), ("plan", dict(cnt=None), -1), ("plan", dict(cu=None), -1), ("plan", dict(slots=None), -1), ("plan", dict(rows=-1), -1),
    ("plan", dict(len=A + 2), -1), ("plan", dict(cu=A + 1), -1),
    ("append", dict(slots=None), -1), ("append", dict(slots=A + 2), -1), ("append", dict(rows=-1), -1), ("append", dict(k=None), -1), ("append", dict(v=A + 8), -1),
    ("plan", dict(rows=(1 << 30) + 1), -4), ("append", dict(rows=(1 << 30) + 1), -4), ("prompt", dict(rows=(1 << 30) + 1), -4), ("attn", dict(total=(1 << 30) + 1), -4),
    ("append", dict(ldk=(1 << 22) + 8), -4), ("prompt", dict(ldo=(1 << 22) + 8), -4), ("attn", dict(ldq=(1 << 22) + 8), -4),
    ("append", dict(ldk=120), -1), ("append", dict(ldv=132), -1), ("append", dict(ldk=-128), -1),
    ("prompt", dict(q=None), -1), ("prompt", dict(q=A + 2), -1), ("prompt", dict(ldq=248), -1), ("prompt", dict(ldq=260), -1), ("prompt", dict(k=None), -1),
    ("prompt", dict(ldk=0), -1), ("prompt", dict(v=A + 8), -1), ("prompt", dict(cu=None), -1), ("prompt", dict(rows=-1), -1), ("prompt", dict(window=-1), -1),
    ("prompt", dict(scale=0.0), -1), ("prompt", dict(scale=-1.0), -1), ("prompt", dict(scale=float("nan")), -1), ("prompt", dict(scale=float("inf")), -1),
    ("prompt", dict(out=None), -1), ("prompt", dict(ldo=128), -1), ("prompt", dict(n_q=3), -1), ("prompt", dict(n_q=0), -1),
    ("prompt", dict(n_q=34, ldq=4096, ldo=4096), -4),
    ("attn", dict(q=None), -1), ("attn", dict(ldq=255), -1), ("attn", dict(n_q=3), -1), ("attn", dict(n_q=34, ldq=4096, ldo=4096), -4), ("attn", dict(total=-1), -1),
    ("attn", dict(cu=None), -1), ("attn", dict(len=None), -1), ("attn", dict(len=A + 2), -1), ("attn", dict(rows=0), -1), ("attn", dict(rows=17), -4),
    ("attn", dict(window=-1), -1), ("attn", dict(scale=0.0), -1), ("attn", dict(out=None), -1), ("attn", dict(ldo=255), -1), ("attn", dict(scratch=None), -1),
    ("attn", dict(scratch=A + 16), -1), ("attn", dict(bytes=0), -1)])
def test_bad_arguments_are_refused(name, args, code):
    assert calls(cache(), _abi.lib())[name](**args) == code


@pytest.mark.parametrize("name,args", [
    ("plan", dict(cu=A)), ("plan", dict(slots=A + 4)), ("plan", dict(cu=B[7], slots=B[7] + 8)), ("plan", dict(len=B[3])), ("plan", dict(cnt=B[2] + 28)),
    ("plan", dict(cu=B[4] + 28)), ("plan", dict(slots=B[5] + 12)), ("plan", dict(slots=B[2] - 12)),
    ("append", dict(k=B[0] + 64)), ("append", dict(v=B[1] - 16)), ("append", dict(k=B[1])),
    ("prompt", dict(out=A)), ("prompt", dict(q=B[9])), ("prompt", dict(k=B[9] + 1536)), ("prompt", dict(v=B[9] - 768)), ("prompt", dict(q=B[9] + 16, ldq=512, ldo=512)),
    ("prompt", dict(q=B[9] + 512 + 16, ldq=512, ldo=512)), ("prompt", dict(k=B[9] + 512, ldk=520, ldo=512)),
    ("attn", dict(q=B[9])), ("attn", dict(out=A + 1024)), ("attn", dict(out=B[0] + 64)), ("attn", dict(out=B[1] - 1024)), ("attn", dict(q=B[9] - 16, ldq=512, ldo=512))])
def test_outputs_that_lie_in_something_else_are_refused(name, args):
    assert calls(cache(), _abi.lib())[name](**args) == -1


def test_calls_of_no_rows_do_nothing():
    c = calls(cache(), _abi.lib())
    assert c["append"](rows=0, slots=None, k=None, v=None) == 0
    assert c["prompt"](rows=0, q=None, k=None, v=None, out=None) == 0
    assert c["attn"](total=0, q=None, out=None) == 0


@pytest.mark.parametrize("n_q,rows", [(3, 1), (0, 1), (4, 0), (4, 17), (34, 1)])
def test_scratch_of_shapes_it_does_not_take(n_q, rows):
    assert _abi.lib().dfl_paged_attn_scratch_bytes(ctypes.byref(cache()), n_q, rows) == -1


def test_constants():
    import os
    import re
    src = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "dfl.h")).read()
    assert re.search(r"DFL_BF16 = 0, DFL_F16 = 1", src) and (_abi.DFL_BF16, _abi.DFL_F16) == (0, 1)
    assert ctypes.sizeof(_abi.dfl_paged) == 88


def test_the_plain_plan():
    p = Plan(2, 4, 3, 16)
    cu, slots, short = p.step([0, 0], [17, 16], 40)
    assert cu.tolist() == [0, 17, 33] and not short and p.held == [2, 1]
    assert slots[:17].tolist() == list(range(17)) and slots[17:33].tolist() == list(range(32, 48)) and (slots[33:] == -1).all()
    cu, slots, short = p.step([0, 16], [0, 33], 40)              # the first ends, the second is longer than three pages
    assert short and p.held == [0, 1] and (slots == -1).all() and p.ring == [3, 0, 1]
    cu, slots, short = p.step([0, 16], [0, 32], 32)              # its pages come from those given back
    assert not short and p.table[1] == [2, 3, 0] and p.ring == [1]


def test_the_plain_attention():
    rng = np.random.default_rng(0)
    q, k, v = rng.standard_normal((2, 4, 8)), rng.standard_normal((5, 2, 8)), rng.standard_normal((5, 2, 8))
    out, tol = attend(q, k, v, 3, 0, True, 0.3, 8)
    a = 0.3 * k[:4, 1] @ q[0, 2]
    w = np.exp(a) / np.exp(a).sum()
    np.testing.assert_allclose(out[0, 2], w @ v[:4, 1], rtol=1e-12)
    np.testing.assert_array_equal(attend(q, k, v, 3, 1, True, 0.3, 8)[0][1, 3], v[4, 1])
    np.testing.assert_allclose(attend(q, k, v, 3, 1, False, 0.3, 8)[0], attend(q, k[2:], v[2:], 1, 0, False, 0.3, 8)[0])
    assert (tol > 0).all() and (tol < 0.1).all()
