"""Cases for the key/value cache in 8 bits: appending rows, attention over it, eviction by accumulated
attention weight, and a decode step of them together.

The cache (per sequence and key/value head): blocks of 32 tokens as uint8 codes with one fp32 scale for
a block's keys and one for its values (value = (code - 128) * scale, scale = amax / 127 rounded to
fp32, codes rounded to nearest even); the rows behind the last sealed block in an fp32 tail of 48 rows;
a table from logical to stored blocks; a score per logical block.

  k, v            uint8 [seq][kv][blocks][head_dim/64][32][64] and [seq][kv][blocks][head_dim][32]
  k_scale,v_scale fp32  [seq][kv][blocks]
  k_tail, v_tail  fp32  [seq][kv][48][head_dim] and [seq][kv][head_dim][48]
  table           int32 [seq][kv][blocks]  the stored block of each logical block (a permutation)
  sealed          int32 [seq][kv]          logical blocks held as codes
  score           fp32  [seq][kv][blocks]
"""
import math

import torch

own = False

BLOCK, TAIL = 32, 48
# query heads, key/value heads, head dimension: the tiny pair's layers, the E4B pair's sliding and full
# layers, the 27B-class target, the draft
HEADS = ((4, 1, 64), (4, 2, 64), (12, 1, 256), (12, 2, 256), (32, 16, 128), (32, 8, 128))
MOST_BYTES = 8 * 16 * 2 * 128 * 16384      # codes that the largest listed case reads
MOST_PAIRS = 8 * 8 * 32 * 128 * 16384      # rows x query heads x head dimension x keys of that case
DEVICE = "cuda"


def _attn(name, seqs, heads, rows, held, **more):
    case = dict(name=name, op="attn", seqs=seqs, n_q=heads[0], n_kv=heads[1], head_dim=heads[2], rows=rows, held=held, window=0,
                causal=True, score=False, ragged=False)
    case.update(more)
    return case


def listed():
    e4b_s, e4b_f, b27, draft = HEADS[2], HEADS[3], HEADS[4], HEADS[5]
    return [
        # a prompt's rows become the draft's context after a pinned prefix of 512 tokens
        dict(name="append prompt", op="append", seqs=1, n_kv=8, head_dim=128, rows=1024, held=512, ragged=False),
        # prompts of several requests, of different lengths, behind contexts that end inside a block
        dict(name="append ragged", op="append", seqs=16, n_kv=2, head_dim=256, rows=777, held=1000, ragged=True),
        # one token of one sequence on the tiny pair: a call's latency
        _attn("attn tiny token", 1, HEADS[1], 1, 200),
        # plain decode, a full layer of the E4B pair at a long context
        _attn("attn token long", 1, e4b_f, 1, 16384),
        # a verify of a draft block over the same layer, scores kept
        _attn("attn verify long", 1, e4b_f, 8, 16384, score=True),
        # a verify of the most rows on a sliding layer
        _attn("attn verify sliding", 4, e4b_s, 16, 4096, window=512),
        # the draft's own block over its context: every row sees the window and the whole block
        _attn("attn draft block", 1, draft, 8, 4096, window=1024, causal=False),
        # plain decode of many sequences of different lengths
        _attn("attn tokens batch", 64, draft, 1, 8191, ragged=True),
        # verifies of several long sequences of the 27B-class target
        _attn("attn verify batch", 8, b27, 8, 16384),
        # a step of a few sequences: the rows are staged, then attend, and the weights are added up
        dict(_attn("step", 4, draft, 8, 2000, score=True, ragged=True), op="step"),
        # one sequence of 16384 tokens thinned to half
        dict(name="evict half", op="evict", seqs=1, n_kv=2, head_dim=256, held=16384, keep=256, sink=4, recent=16),
        # several sequences of 131072 tokens thinned to an eighth
        dict(name="evict long", op="evict", seqs=8, n_kv=8, head_dim=64, held=131072, keep=512, sink=8, recent=64),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "attn", "attn", "attn", "step", "evict"])
    n_q, n_kv, hd = rng.choice(HEADS)
    if op == "append":
        seqs = _log(rng, 1, 16)
        rows = _log(rng, 1, min(8192, 24_000_000 // (seqs * n_kv * hd)))
        held = _log(rng, 1, 2048)
        return dict(op=op, seqs=seqs, n_kv=n_kv, head_dim=hd, rows=rows, held=held // BLOCK * BLOCK if rng.random() < 0.4 else held,
                    ragged=seqs > 1 and rng.random() < 0.6)
    if op == "evict":
        held = _log(rng, 64, 131072)
        blocks = held // BLOCK
        sink, recent = rng.randrange(0, 9), rng.randrange(0, 65)
        return dict(op=op, seqs=_log(rng, 1, 8), n_kv=rng.choice((1, 2, 8)), head_dim=64, held=held, keep=max(sink + recent, _log(rng, 1, blocks)), sink=sink,
                    recent=recent)
    seqs, rows = _log(rng, 1, 64), rng.randrange(1, 17)
    most = min(MOST_BYTES // (seqs * n_kv * 2 * hd), MOST_PAIRS // (seqs * rows * n_q * hd), 65536)
    case = _attn("", seqs, (n_q, n_kv, hd), rows, _log(rng, 1, most), window=rng.choice((0, 0, _log(rng, 1, 2048))),
                 causal=rng.random() < 0.7, score=rng.random() < 0.4, ragged=seqs > 1 and rng.random() < 0.6)
    del case["name"]
    case["op"] = op
    return case


# ---- sizes that a case stands for, the same for every seed ---------------------------------------------
def _lengths(case):
    """Tokens held by each sequence: all `held`, or spread evenly from `held` down to a quarter of it."""
    n = case["seqs"]
    return [case["held"] - (case["held"] * 3 * i // (4 * (n - 1)) if case["ragged"] and n > 1 else 0) for i in range(n)]


def _counts(case):
    """Rows of each sequence: all `rows`, or `rows`, then fewer, and none for the last but one of more than two."""
    n = case["seqs"]
    if not case["ragged"] or n == 1:
        return [case["rows"]] * n
    c = [max(1, case["rows"] - case["rows"] * i // n) for i in range(n)]
    if n > 2:
        c[n - 2] = 0
    return c


def _visible(case, length, count):
    """Keys that some row of a sequence sees."""
    if not count:
        return 0
    w = case["window"]
    first = 0 if not w else max(0, length - w + (1 if case["causal"] else 0))
    return length - first + count


def work(case):
    kv = case["n_kv"] * case["head_dim"] * 2
    if case["op"] == "append":
        n = sum(_counts(case))
        return {"bytes": n * kv * (4 + 1 + 4), "flops": n * kv * 6}
    if case["op"] == "evict":
        heads, blocks = case["seqs"] * case["n_kv"], case["held"] // BLOCK
        return {"bytes": heads * blocks * (8 + 8), "flops": heads * blocks * 8}
    b = f = 0
    for length, count in zip(_lengths(case), _counts(case)):
        keys, q = _visible(case, length, count), count * case["n_q"] * case["head_dim"]
        b += keys * kv + q * 8 + (count * kv * 8 if case["op"] == "step" else 0)
        f += 4 * keys * q
    return {"bytes": max(b, 1), "flops": max(f, 1)}


# ---- inputs ----------------------------------------------------------------------------------------
def _quantise(x):
    """Codes and scales of blocks x [.., 32, head_dim]. Quotients and their rounding in 64 bits: a value next to the border of two codes
    takes the code that the definition gives it."""
    amax = x.abs().amax((-1, -2))
    amax = torch.where(torch.isfinite(amax), amax, torch.full_like(amax, float("nan")))
    scale = (amax.double() / 127).float()
    safe = torch.where(scale > 0, scale, torch.ones_like(scale)).double()
    code = torch.round(x.double() / safe[..., None, None]).clamp(-127, 127)
    return torch.where(torch.isfinite(code), code + 128, torch.full_like(code, 128)).to(torch.uint8), scale


def _store_k(c):      # [.., 32, head_dim] -> [.., head_dim/64, 32, 64]
    return c.unflatten(-1, (-1, 64)).transpose(-3, -2).contiguous()


def _store_v(c):      # [.., 32, head_dim] -> [.., head_dim, 32]
    return c.transpose(-2, -1).contiguous()


def prepare(case, seed):
    g = torch.Generator(device=DEVICE).manual_seed(seed)
    S, kv, hd = case["seqs"], case["n_kv"], case["head_dim"]
    rand = lambda *shape: torch.randn(shape, generator=g, device=DEVICE)  # noqa: E731
    order = torch.randperm(S, generator=g, device=DEVICE)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=DEVICE)  # noqa: E731
    s = {"case": case}
    if case["op"] == "evict":
        blocks = case["held"] // BLOCK
        cap = blocks + 4
        s["len"] = i32([case["held"]] * S)
        s["k"] = torch.empty(S, kv, cap, hd // 64, 32, 64, dtype=torch.uint8, device=DEVICE)   # eviction reads no codes
        s["v"] = torch.empty(S, kv, cap, hd, 32, dtype=torch.uint8, device=DEVICE)
        s["k_scale"], s["v_scale"] = (torch.ones(S, kv, cap, device=DEVICE) for _ in range(2))
        s["k_tail"], s["v_tail"] = torch.zeros(S, kv, TAIL, hd, device=DEVICE), torch.zeros(S, kv, hd, TAIL, device=DEVICE)
        # weights add up to a few heavy blocks and many light ones, some of them never looked at (equal scores)
        score = torch.exp(2.5 * rand(S, kv, cap))
        s["score"] = torch.where(rand(S, kv, cap) > 1.2, torch.zeros_like(score), score)
        s["sealed"] = torch.full((S, kv), blocks, dtype=torch.int32, device=DEVICE)
        s["table"] = torch.argsort(rand(S, kv, cap), dim=-1).to(torch.int32)
        s["to"] = {"table": torch.empty_like(s["table"]), "score": torch.empty_like(s["score"]), "sealed": torch.empty_like(s["sealed"]),
                   "len": torch.empty_like(s["len"])}
        return s
    held, rows = _lengths(case), _counts(case)
    cap = max(held) // BLOCK + (case["rows"] + 2 * BLOCK - 1) // BLOCK + 2
    s["len"], s["n"] = i32(held)[order], i32(rows)[order]
    s["after"] = s["len"] + s["n"]
    s["sealed"] = (s["len"] // BLOCK)[:, None].expand(S, kv).contiguous()
    s["table"] = torch.argsort(rand(S, kv, cap), dim=-1).to(torch.int32)
    s["score"] = rand(S, kv, cap).abs()
    s["k"] = torch.empty(S, kv, cap, hd // 64, 32, 64, dtype=torch.uint8, device=DEVICE)
    s["v"] = torch.empty(S, kv, cap, hd, 32, dtype=torch.uint8, device=DEVICE)
    s["k_scale"], s["v_scale"] = (torch.empty(S, kv, cap, device=DEVICE) for _ in range(2))
    # keys have channels that stand out, as rotated keys do; rows differ in size
    gain_k, gain_v = torch.exp(0.5 * rand(kv, 1, hd)), torch.exp(0.2 * rand(kv, 1, hd))
    sized = lambda x: x * torch.exp(0.2 * rand(*x.shape[:-1], 1))  # noqa: E731
    for i in range(S):
        place, head = s["table"][i].long(), torch.arange(kv, device=DEVICE)[:, None]
        for gain, codes, scale, store in ((gain_k, "k", "k_scale", _store_k), (gain_v, "v", "v_scale", _store_v)):
            c, f = _quantise(sized(rand(kv, cap * BLOCK, hd) * gain).unflatten(1, (cap, BLOCK)))
            s[codes][i][head, place], s[scale][i][head, place] = store(c), f
    s["k_tail"] = (sized(rand(S, kv, TAIL, hd)) * gain_k)
    s["v_tail"] = (sized(rand(S, kv, TAIL, hd)) * gain_v).transpose(-2, -1).contiguous()
    if case["op"] in ("append", "step"):
        s["new_k"], s["new_v"] = (sized(rand(S, case["rows"], kv, hd)) * gain[:, 0] for gain in (gain_k, gain_v))
    if case["op"] == "append":
        s["read"] = [torch.zeros(S, case["rows"], kv, hd, device=DEVICE) for _ in range(2)]
    else:
        s["q"] = 1.5 * rand(S, case["rows"], case["n_q"], hd)
        s["out"] = torch.zeros_like(s["q"])
    return s


# ---- the operators in their plain form ----------------------------------------------------------------
def _arange(n):
    return torch.arange(n, device=DEVICE)


def _plain_write(s, commit):
    """The rows of s["new_k"], s["new_v"] go behind the s["len"] tokens held. Blocks of committed tokens that are complete are sealed (with
    `commit` the new rows are committed too), the others stay in the tail. Where more is sealed than is held, the cache is cut back: the
    rows of the block that the cut goes through come back from their codes."""
    z = torch.minimum(s["sealed"], (s["len"] // BLOCK)[:, None]).long()            # [S, kv]
    have = s["len"][:, None] - BLOCK * z                                           # rows of the tail in use
    new = s["new_k"].shape[1]
    cap = -(-(TAIL + new) // BLOCK)
    r = _arange(cap * BLOCK)
    total = have + s["n"][:, None]
    full = (total if commit else have) // BLOCK                                    # blocks to seal
    b = _arange(cap)
    seal = b < full[..., None]                                                     # [S, kv, cap]
    last = s["table"].shape[2] - 1
    place = torch.gather(s["table"].long(), 2, (z[..., None] + b).clamp(max=last))
    keep = seal & (z[..., None] + b <= last)
    seq, head = _arange(z.shape[0])[:, None, None], _arange(z.shape[1])[None, :, None]
    for codes, scale, tail, fresh, store in (("k", "k_scale", s["k_tail"], s["new_k"], _store_k), ("v", "v_scale", s["v_tail"].transpose(-2, -1), s["new_v"], _store_v)):
        hd = fresh.shape[-1]
        wide = lambda i: i[..., None].expand(*i.shape, hd)  # noqa: E731
        old = s[codes][seq, head, place[..., :1]].float() - 128
        old = (old.transpose(-3, -2).flatten(-2) if codes == "k" else old.transpose(-2, -1)) * s[scale][seq, head, place[..., :1]][..., None, None]
        old = torch.where((s["sealed"] > s["len"][:, None] // BLOCK)[..., None, None], torch.nn.functional.pad(old[:, :, 0], (0, 0, 0, TAIL - BLOCK)), tail)
        from_tail = torch.gather(old, 2, wide(r.clamp(max=TAIL - 1).expand(*z.shape, -1)))
        from_new = torch.gather(fresh.transpose(1, 2), 2, wide((r - have[..., None]).clamp(0, new - 1)))
        x = torch.where((r < have[..., None])[..., None], from_tail, from_new)     # [S, kv, cap * 32, hd]
        c, f = _quantise(x.unflatten(2, (cap, BLOCK)))
        where = [i.expand(place.shape)[keep] for i in (seq, head, place)]
        s[codes][tuple(where)], s[scale][tuple(where)] = store(c)[keep], f[keep]
        t = _arange(TAIL)
        left = torch.gather(x, 2, wide((t + BLOCK * full[..., None]).clamp(max=cap * BLOCK - 1)))
        tail.copy_(torch.where((t < (total - BLOCK * full)[..., None])[..., None], left, tail))
    s["sealed"].copy_(z + full)
    begun = _arange(last + 1) * BLOCK                                              # blocks whose first token is among the new rows
    lo, hi = s["len"][:, None, None], (s["len"] + s["n"])[:, None, None]
    s["score"].masked_fill_((begun >= lo) & (begun < hi), 0.0)


def _plain_values(s, blocks):
    """Keys and values [S, kv, blocks * 32, head_dim] of the first logical blocks."""
    got = []
    for codes, scale in (("k", "k_scale"), ("v", "v_scale")):
        c = s[codes]
        place = s["table"][:, :, :blocks].long()
        at = (_arange(c.shape[0])[:, None, None], _arange(c.shape[1])[None, :, None], place)
        x = c[at].float() - 128
        x = x.transpose(-3, -2).flatten(-2) if codes == "k" else x.transpose(-2, -1)
        got.append((x * s[scale][at][..., None, None]).flatten(2, 3))
    return got


def _plain_read(s, first, count, rows):
    """Rows first .. first + count of each sequence into s["read"]."""
    blocks = s["table"].shape[2]
    pos = (first[:, None] + _arange(rows)).long()                                  # [S, rows]
    z = s["sealed"].long()[..., None] * BLOCK
    for held, tail, out in zip(_plain_values(s, blocks), (s["k_tail"], s["v_tail"].transpose(-2, -1)), s["read"]):
        hd = held.shape[-1]
        p = pos[:, None, :].expand(-1, held.shape[1], -1)
        wide = lambda i: i[..., None].expand(*i.shape, hd)  # noqa: E731
        x = torch.where((p < z)[..., None], torch.gather(held, 2, wide(p.clamp(max=blocks * BLOCK - 1))),
                        torch.gather(tail, 2, wide((p - z).clamp(0, TAIL - 1))))
        valid = (_arange(rows) < count[:, None])[:, :, None, None]
        out.copy_(torch.where(valid, x.transpose(1, 2), out))
    return s["read"]


def _plain_attn(s):
    case, q = s["case"], s["q"]
    S, M, n_q, hd = q.shape
    kv, group = case["n_kv"], n_q // case["n_kv"]
    blocks = max(_lengths(case)) // BLOCK
    k, v = _plain_values(s, blocks)
    k, v = torch.cat([k, s["k_tail"]], 2), torch.cat([v, s["v_tail"].transpose(-2, -1)], 2)
    z = s["sealed"].long()[..., None] * BLOCK                                      # [S, kv, 1]
    coded = _arange(blocks * BLOCK).expand(S, kv, -1)
    pos = torch.cat([coded, z + _arange(TAIL)], 2)                                 # [S, kv, keys]
    end = s["after"].long()[:, None, None]
    held = torch.cat([coded < z, (z + _arange(TAIL)) < end], 2)
    k, v = torch.where(held[..., None], k, 0.0), torch.where(held[..., None], v, 0.0)
    m = _arange(M)
    own_pos = (s["len"].long()[:, None] + m)[:, None, :, None]                     # [S, 1, M, 1]
    key = pos[:, :, None, :]
    start = s["len"].long()[:, None, None, None]
    sees = held[:, :, None, :] & ((key <= own_pos) if case["causal"] else (key < end[..., None]))
    if case["window"]:
        sees = sees & ((key > own_pos - case["window"]) if case["causal"] else (key >= start - case["window"]))
    live = m < s["n"][:, None]                                                     # [S, M]
    rows = q.view(S, M, kv, group, hd).permute(0, 2, 1, 3, 4).reshape(S, kv, M * group, hd)
    a = (rows @ k.transpose(-2, -1) * hd ** -0.5).view(S, kv, M, group, -1)
    a = a.masked_fill(~sees[:, :, :, None, :], float("-inf"))
    top = a.amax(-1, keepdim=True)
    e = torch.exp(a - torch.where(torch.isfinite(top), top, 0.0))
    total = e.sum(-1, keepdim=True)
    p = e / torch.where(total > 0, total, 1.0)
    o = (p.view(S, kv, M * group, -1) @ v).view(S, kv, M, group, hd).permute(0, 2, 1, 3, 4).reshape(S, M, n_q, hd)
    s["out"].copy_(torch.where(live[:, :, None, None], o, s["out"]))
    if case["score"]:
        w = p[:, :, 0].sum(2) * live[:, :1, None]                                  # [S, kv, keys]: row 0's heads
        got = torch.zeros(S, kv, s["score"].shape[2] + 2, device=w.device)
        got[:, :, :blocks] = w[:, :, :blocks * BLOCK].unflatten(2, (blocks, BLOCK)).sum(3)
        at = s["sealed"].long()
        got.scatter_add_(2, at[..., None], w[:, :, blocks * BLOCK:blocks * BLOCK + BLOCK].sum(2, keepdim=True))
        got.scatter_add_(2, at[..., None] + 1, w[:, :, blocks * BLOCK + BLOCK:].sum(2, keepdim=True))
        s["score"].add_(got[:, :, :-2])
    return s["out"]


def _plain_evict(s):
    case, to = s["case"], s["to"]
    cap = s["table"].shape[2]
    n = s["sealed"].long()[..., None]                                              # [S, kv, 1]
    i = _arange(cap).expand(*s["table"].shape)
    keep = torch.minimum(n, torch.full_like(n, case["keep"]))
    key = torch.where(torch.isnan(s["score"]), float("-inf"), s["score"])
    # 2: outside the choice (first and last blocks), 1: chosen by score, 0: not held
    safe = (i < case["sink"]) | (i >= n - case["recent"])
    rank1 = torch.argsort(key, dim=-1, descending=True, stable=True)
    level = torch.where(i >= n, 0, torch.where(safe, 2, 1))
    rank2 = torch.argsort(torch.gather(level, 2, rank1), dim=-1, descending=True, stable=True)
    rank = torch.gather(rank1, 2, rank2)
    kept = torch.zeros_like(level).scatter_(2, rank, (i < keep).long()).bool()
    new = torch.argsort(torch.where(kept, 0, torch.where(i < n, 1, 2)), dim=-1, stable=True)
    to["table"].copy_(torch.gather(s["table"], 2, new))
    tail = (i >= keep) & (i < keep + 2) & (i + n - keep < cap)
    moved = torch.gather(s["score"], 2, torch.where(tail, (i + n - keep).clamp(max=cap - 1), new))
    to["score"].copy_(torch.where((i < keep) | tail, moved, 0.0))
    to["sealed"].copy_(keep[..., 0])
    to["len"].copy_(s["len"] - BLOCK * (n - keep)[:, 0, 0])
    return to


# ---- the operators by the framework ---------------------------------------------------------------------
def _cache(s):
    """The handle that a program keeps: made at a state's first pass."""
    if "cache" not in s:
        from dflash_speculative_decode_gb300 import Kv8Cache
        s["cache"] = Kv8Cache(**{name: s[name] for name in ("k", "v", "k_scale", "v_scale", "k_tail", "v_tail", "table", "sealed", "score")})
    return s["cache"]


def run(s):
    case = s["case"]
    if case["op"] == "append":
        if own:
            c = _cache(s)
            c.append(s["new_k"], s["new_v"], s["len"], s["n"])
            c.read(s["after"], case["rows"], first=s["len"], out=s["read"])
        else:
            _plain_write(s, commit=True)
            _plain_read(s, s["len"], s["n"], case["rows"])
        return s["read"], s["k_tail"], s["v_tail"], s["sealed"]
    if case["op"] == "evict":
        if own:
            return _cache(s).evict(s["len"], case["keep"], sink=case["sink"], recent=case["recent"], out=s["to"])
        return _plain_evict(s)
    if case["op"] == "step":
        if own:
            _cache(s).stage(s["new_k"], s["new_v"], s["len"], s["n"])
        else:
            _plain_write(s, commit=False)
    if own:
        _cache(s).attn(s["q"], s["len"], s["n"], window=case["window"], causal=case["causal"], score=case["score"], out=s["out"])
    else:
        _plain_attn(s)
    got = {"out": s["out"]}
    if case["score"]:
        got["score"] = s["score"]
    if case["op"] == "step":
        got.update(k_tail=s["k_tail"], v_tail=s["v_tail"])
    return got


# ---- the definition in 64 bits, one sequence and head at a time --------------------------------------------
def _exact_rows(s, i, h):
    """The rows that sequence i, head h holds before the call, keys and values, in 64 bits, and how many are sealed."""
    z, held = int(s["sealed"][i, h]), int(s["len"][i])
    got = []
    for codes, scale, tail in (("k", "k_scale", s["k_tail"][i, h]), ("v", "v_scale", s["v_tail"][i, h].T)):
        at = s["table"][i, h, :z].long()
        c = s[codes][i, h].index_select(0, at).double().sub_(128.0)
        c = torch.cat(list(c.unbind(1)), -1) if codes == "k" else torch.movedim(c, 1, 2)
        c = c * s[scale][i, h].index_select(0, at).double().reshape(-1, 1, 1)
        got.append(torch.cat([c.reshape(z * BLOCK, s["case"]["head_dim"]), tail[:held - z * BLOCK].double()]))
    return got, z


def _exact_append(s):
    case = s["case"]
    read = [x.double().clone() for x in s["read"]]
    tails = [s["k_tail"].double().clone(), s["v_tail"].double().clone()]
    for i in range(case["seqs"]):
        n, held = int(s["n"][i]), int(s["len"][i])
        for h in range(case["n_kv"]):
            z = int(s["sealed"][i, h])
            part = held - z * BLOCK
            for j, (tail, new) in enumerate(((s["k_tail"][i, h], s["new_k"]), (s["v_tail"][i, h].T, s["new_v"]))):
                x = torch.cat([tail[:part], new[i, :n, h]]).double()
                full = x.shape[0] // BLOCK
                for blk in x[:full * BLOCK].reshape(full, BLOCK, case["head_dim"]).split(4096):
                    step = (blk.abs().flatten(1).max(1).values / 127).float().double()[:, None, None]   # the scale as it is held
                    blk.copy_(torch.where(step > 0, torch.round(blk / torch.where(step > 0, step, 1.0)).clip(-127, 127) * step, 0.0))
                read[j][i, :n, h] = x[part:]
                rest = x[full * BLOCK:]
                if j:
                    tails[1][i, h, :, :len(rest)] = rest.T
                else:
                    tails[0][i, h, :len(rest)] = rest
    return read, tails[0], tails[1], None


def _exact_attn(s):
    case = s["case"]
    out, score = s["out"].double().clone(), s["score"].double().clone()
    tails = [s["k_tail"].double().clone(), s["v_tail"].double().clone()]
    group, hd = case["n_q"] // case["n_kv"], case["head_dim"]
    for i in range(case["seqs"]):
        n, held = int(s["n"][i]), int(s["len"][i])
        if case["op"] == "step":
            at = (torch.arange(held, held + n) // BLOCK)[torch.arange(held, held + n) % BLOCK == 0].tolist()
            score[i][:, at] = 0.0
        if not n:
            continue
        for h in range(case["n_kv"]):
            (k, v), z = _exact_rows(s, i, h)
            part = held - z * BLOCK
            if case["op"] == "step":
                nk, nv = s["new_k"][i, :n, h].double(), s["new_v"][i, :n, h].double()
                tails[0][i, h, part:part + n], tails[1][i, h, :, part:part + n] = nk, nv.T
            else:
                nk, nv = s["k_tail"][i, h, part:part + n].double(), s["v_tail"][i, h, :, part:part + n].T.double()
            k, v = torch.cat([k, nk]), torch.cat([v, nv])
            key = torch.arange(held + n, device=k.device)
            for m in range(n):
                lo, hi = 0, held + (m + 1 if case["causal"] else n)
                if case["window"]:
                    lo = max(0, held + m - case["window"] + 1 if case["causal"] else held - case["window"])
                a = s["q"][i, m, h * group:(h + 1) * group].double() @ k[lo:hi].T / math.sqrt(hd)
                p = torch.softmax(a, -1)
                out[i, m, h * group:(h + 1) * group] = p @ v[lo:hi]
                if m == 0 and case["score"]:
                    score[i, h].index_add_(0, key[lo:hi] // BLOCK, p.sum(0))
    got = {"out": out}
    if case["score"]:
        got["score"] = score
    if case["op"] == "step":
        got.update(k_tail=tails[0], v_tail=tails[1])
    return got


def _exact_evict(s):
    case, blocks = s["case"], s["case"]["held"] // BLOCK
    score = torch.zeros_like(s["score"], dtype=torch.float64)
    old = s["score"].double().cpu()
    for i in range(case["seqs"]):
        for h in range(case["n_kv"]):
            w = old[i, h].tolist()
            keep = min(blocks, case["keep"])
            safe = {b for b in range(blocks) if b < case["sink"] or b >= blocks - case["recent"]}
            best = sorted(range(blocks), key=lambda b: (b not in safe, -w[b], b))[:keep]
            row = [w[b] for b in sorted(best)] + w[blocks:blocks + 2]
            score[i, h, :len(row)] = torch.tensor(row, dtype=torch.float64)
    return {"table": None, "score": score, "sealed": None, "len": None}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "append":
        return _exact_append(s)
    return _exact_evict(s) if case["op"] == "evict" else _exact_attn(s)
