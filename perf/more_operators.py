"""Cases for a paged key/value cache in 16 bits and the attention beside it: block tables and slot maps planned
from request lengths, rows into pages, attention over whole packed prompts, and attention of one token or a
verify's rows over the pages.

The cache is a pool of pages that all sequences share. A page holds `page` tokens of every key/value head:

  k, v    bf16 or fp16 [n_pages][n_kv][page][head_dim]
  table   int32 [n_seq][max_pages]  the page of each `page` tokens of a sequence; entries behind `held` mean nothing
  held    int32 [n_seq]             pages that a sequence has
  free    int32 [n_pages]           a ring of the pages that no sequence has
  queue   int32 [4]                 where the ring begins, how many pages it holds, and two words of the library's (0)

Rows of a call are packed: sequence s has rows cu[s] .. cu[s+1] - 1 of [rows][heads][head_dim], at positions
len[s], len[s] + 1, ...; rows behind the last sequence's are not touched.
"""
import math

import torch

own = False

# query heads, key/value heads, head dimension: the tiny pair's layers, the E4B pair's sliding and full
# layers, the 27B-class target, the draft
HEADS = ((4, 1, 64), (4, 2, 64), (12, 1, 256), (12, 2, 256), (32, 16, 128), (32, 8, 128))
PAGES = (16, 32, 64, 128)
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
MOST_SCORES = 32 * 16384 * 16384           # heads x rows x keys of the largest prompt, masked places among them
MOST_BYTES = 8 * 16 * 2 * 2 * 128 * 16384  # keys and values of the largest attention over pages
MOST_PAIRS = 8 * 8 * 32 * 128 * 16384      # its rows x query heads x head dimension x keys
DEVICE = "cuda"


def _plan(name, seqs, held, rows, every, page):
    return dict(name=name, op="plan", seqs=seqs, held=held, rows=rows, every=every, page=page)


def _append(name, seqs, heads, rows, held, page, ragged, dtype="bf16"):
    return dict(name=name, op="append", seqs=seqs, n_kv=heads[1], head_dim=heads[2], rows=rows, held=held, page=page, ragged=ragged, dtype=dtype)


def _prompt(name, seqs, heads, rows, window=0, ragged=False, dtype="bf16"):
    return dict(name=name, op="prompt", seqs=seqs, n_q=heads[0], n_kv=heads[1], head_dim=heads[2], rows=rows, window=window, ragged=ragged, dtype=dtype)


def _attn(name, seqs, heads, rows, held, page, window=0, causal=True, ragged=False, dtype="bf16"):
    return dict(name=name, op="attn", seqs=seqs, n_q=heads[0], n_kv=heads[1], head_dim=heads[2], rows=rows, held=held, page=page, window=window, causal=causal,
                ragged=ragged, dtype=dtype)


def listed():
    tiny, e4b_s, e4b_f, b27, draft = HEADS[1:]
    return [
        # a decode step of a full batch: one row a sequence, every eighth place gets a new request or loses one that has ended
        _plan("plan decode step", 64, 8191, 300, 8, 32),
        # a batch of prompts comes in as another goes out
        _plan("plan prompts", 512, 1, 2048, 1, 64),
        # the step's new tokens of a batch into their pages
        _append("append tokens", 64, draft, 1, 8191, 32, True),
        # several requests' prompts into their pages
        _append("append prompts", 16, b27, 1501, 0, 64, True),
        # one short prompt on the tiny pair: a call's latency
        _prompt("prompt tiny", 1, tiny, 32),
        # prompts of several requests, of different lengths, one after another in one call
        _prompt("prompt packed", 16, draft, 2047, ragged=True, dtype="fp16"),
        # the prompt of a sliding layer of the E4B pair
        _prompt("prompt sliding", 2, e4b_s, 4096, window=512),
        # one long prompt of the 27B-class target
        _prompt("prompt long", 1, b27, 16384),
        # one token of one sequence on the tiny pair: a call's latency
        _attn("attn tiny token", 1, tiny, 1, 200, 16),
        # plain decode, a full layer of the E4B pair at a long context
        _attn("attn token long", 1, e4b_f, 1, 16384, 64),
        # plain decode of many sequences of different lengths
        _attn("attn tokens batch", 64, draft, 1, 8191, 32, ragged=True, dtype="fp16"),
        # verifies of several long sequences of the 27B-class target
        _attn("attn verify batch", 8, b27, 8, 16384, 64),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))


def draw(rng):
    op = rng.choice(["plan", "append", "prompt", "prompt", "attn", "attn"])
    heads, page, dtype = rng.choice(HEADS), rng.choice(PAGES), rng.choice(("bf16", "fp16"))
    seqs = _log(rng, 1, 64)
    if op == "plan":
        seqs = _log(rng, 1, 1024)
        case = _plan("", seqs, _log(rng, 1, min(16384, (1 << 21) // seqs)), _log(rng, 1, min(16384, (1 << 20) // seqs)), rng.choice((1, 2, 8)), page)
    elif op == "append":
        rows = _log(rng, 1, min(8192, 48_000_000 // (seqs * heads[1] * heads[2])))
        held = _log(rng, 1, 8192) if rng.random() < 0.6 else 0
        while seqs * (held + rows) * heads[1] * heads[2] > 600_000_000:
            held //= 2
        case = _append("", seqs, heads, rows, held, page, seqs > 1 and rng.random() < 0.6, dtype)
    elif op == "prompt":
        rows = _log(rng, 1, min(16384, math.isqrt(MOST_SCORES // (seqs * heads[0]))))
        case = _prompt("", seqs, heads, rows, rng.choice((0, 0, _log(rng, 1, 2048))), seqs > 1 and rng.random() < 0.6, dtype)
    else:
        rows = rng.choice((1, 1, rng.randrange(1, 17)))
        most = min(MOST_BYTES // (seqs * heads[1] * 4 * heads[2]), MOST_PAIRS // (seqs * rows * heads[0] * heads[2]), 65536)
        case = _attn("", seqs, heads, rows, _log(rng, 1, most), page, rng.choice((0, 0, _log(rng, 1, 2048))), rng.random() < 0.7,
                     seqs > 1 and rng.random() < 0.6, dtype)
    del case["name"]
    return case


# ---- sizes that a case stands for, the same for every seed ---------------------------------------------
def _spread(most, n, ragged):
    """Lengths: all `most`, or spread evenly from `most` down to a quarter of it."""
    return [most - (most * 3 * i // (4 * (n - 1)) if ragged and n > 1 else 0) for i in range(n)]


def _counts(case):
    """Rows of each sequence. Ragged: spread (prompts, appended ones), or `rows`, then fewer; and none for the last but one of more than two."""
    n, rows = case["seqs"], case["rows"]
    c = _spread(rows, n, case["ragged"])
    if case["op"] == "attn" and case["ragged"]:
        c = [max(1, rows - rows * i // n) for i in range(n)]
    if case["ragged"] and n > 2:
        c[n - 2] = 0
    return c


def _turns(case):
    """Lengths and rows of the two steps between which a plan case goes to and fro: places 0, every, 2 * every, .. hold a prompt in one of
    them and nothing in the other, the others decode."""
    got = []
    lens, prompts = _spread(case["held"], case["seqs"], True), _spread(case["rows"], case["seqs"], True)
    for turn in range(2):
        length, n = [], []
        for i in range(case["seqs"]):
            goes = i % case["every"] == 0
            length.append(0 if goes else lens[i] + turn)
            n.append((prompts[i] if i // case["every"] % 2 == turn else 0) if goes else 1)
        got.append((length, n))
    return got


def _pages(tokens, page):
    return -(-tokens // page)


def _visible(case, length, count):
    """Keys that some row of a sequence sees."""
    if not count:
        return 0
    w = case["window"]
    return length - (0 if not w else max(0, length - w + (1 if case["causal"] else 0))) + count


def work(case):
    if case["op"] == "plan":
        turns = _turns(case)
        rows = max(sum(n) for _, n in turns)
        moved = sum(_pages(case["rows"], case["page"]) for _ in range(0, case["seqs"], case["every"])) * 5 // 8
        return {"bytes": case["seqs"] * 5 * 4 + rows * 4 + moved * 8, "flops": rows}
    if case["op"] == "append":
        kv = case["n_kv"] * case["head_dim"] * 2 * 2
        return {"bytes": sum(_counts(case)) * (2 * kv + 4), "flops": 1}
    b = f = 0
    if case["op"] == "prompt":
        for n in _counts(case):
            w = min(case["window"] or n, n)
            pairs = n * (n + 1) // 2 - (n - w) * (n - w + 1) // 2
            f += 4 * pairs * case["n_q"] * case["head_dim"]
            b += n * (case["n_q"] + case["n_kv"]) * case["head_dim"] * 2 * 2
        return {"bytes": b, "flops": f}
    for length, n in zip(_spread(case["held"], case["seqs"], case["ragged"]), _counts(case)):
        keys, q = _visible(case, length, n), n * case["n_q"] * case["head_dim"]
        b += keys * case["n_kv"] * case["head_dim"] * 2 * 2 + q * 2 * 2 + _pages(keys, case["page"]) * 4
        f += 4 * keys * q
    return {"bytes": b, "flops": f}


# ---- inputs ----------------------------------------------------------------------------------------
def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEVICE)


def _cu(n):
    """Where each sequence's rows begin, and where the last one's end."""
    return torch.nn.functional.pad(torch.cumsum(n, 0, dtype=torch.int32), (1, 0))


def prepare(case, seed):
    g = torch.Generator(device=DEVICE).manual_seed(seed)
    rand = lambda *shape: torch.randn(shape, generator=g, device=DEVICE)  # noqa: E731
    S = case["seqs"]
    s = {"case": case, "turn": 0}
    order = torch.randperm(S, generator=g, device=DEVICE)
    if case["op"] == "plan":
        P, turns = case["page"], _turns(case)
        s["turns"] = [(_i32(a)[order], _i32(b)[order]) for a, b in turns]
        most = max(_pages(a + b, P) for length, n in turns for a, b in zip(length, n)) + 2
        has = _pages(s["turns"][0][0], P)                       # each decoding sequence's pages
        n_pages = max(sum(_pages(a + b, P) for a, b in zip(length, n)) for length, n in turns) * 9 // 8 + S
        perm = torch.randperm(n_pages, generator=g, device=DEVICE).to(torch.int32)
        first = _cu(has)
        i = torch.arange(most, device=DEVICE)
        s["table"] = torch.where(i < has[:, None], perm[(first[:-1, None] + i).clamp(max=n_pages - 1)], 0).contiguous()
        s["held"] = has.to(torch.int32)
        used = first[-1]
        s["free"] = torch.roll(perm, 7)                         # the ring begins anywhere and runs over its end
        s["queue"] = torch.stack([(used + 7) % n_pages, n_pages - used, used * 0, used * 0]).to(torch.int32)
        rows = max(sum(n) for _, n in turns) + 3
        s["cu"], s["slots"] = torch.zeros(S + 1, dtype=torch.int32, device=DEVICE), torch.zeros(rows, dtype=torch.int32, device=DEVICE)
        s["k"], s["v"] = (torch.zeros(n_pages, 1, P, 64, dtype=torch.bfloat16, device=DEVICE) for _ in range(2))   # planning reads no pages
        return s
    kv, hd, dtype = case["n_kv"], case["head_dim"], TYPES[case["dtype"]]
    rows = _counts(case)
    held = _spread(case["held"], S, case["ragged"]) if case["op"] != "prompt" else [0] * S
    s["len"], s["n"] = _i32(held)[order], _i32(rows)[order]
    s["cu"] = _cu(s["n"])
    total = sum(rows) + 3                                       # a buffer with room behind the last row
    # keys have channels that stand out, as rotated keys do; rows differ in size
    gain_k, gain_v = torch.exp(0.5 * rand(kv, 1, hd)), torch.exp(0.2 * rand(kv, 1, hd))
    sized = lambda x: x * torch.exp(0.2 * rand(*x.shape[:-1], 1))  # noqa: E731
    P = case.get("page", 64)
    pages = [_pages(a + b, P) for a, b in zip(held, rows)]
    n_pages, most = sum(pages) + 3, max(max(pages), 1)
    perm = torch.randperm(n_pages, generator=g, device=DEVICE).to(torch.int32)
    has = _i32(pages)[order]
    first, i = _cu(has), torch.arange(most, device=DEVICE)
    s["table"] = torch.where(i < has[:, None], perm[(first[:-1, None] + i).clamp(max=n_pages - 1)], 0).contiguous()
    s["held"] = has
    s["free"], s["queue"] = torch.roll(perm, 3), _i32([0, 3, 0, 0])
    if case["op"] == "attn":
        s["k"], s["v"] = (torch.empty(n_pages, kv, P, hd, dtype=dtype, device=DEVICE) for _ in range(2))
        for gain, x in ((gain_k, s["k"]), (gain_v, s["v"])):
            for part in x.split(max(1, (1 << 26) // (kv * P * hd))):
                part.copy_(sized(rand(*part.shape)) * gain)
    else:
        s["k"], s["v"] = (torch.zeros(n_pages, kv, P, hd, dtype=dtype, device=DEVICE) for _ in range(2))
        s["new_k"], s["new_v"] = ((sized(rand(total, kv, hd)) * gain[:, 0]).to(dtype) for gain in (gain_k, gain_v))
    if case["op"] == "append":
        r = torch.arange(total, device=DEVICE)
        seq = torch.searchsorted(s["cu"][1:].contiguous(), r.to(torch.int32), right=True).clamp(max=S - 1)
        pos = s["len"][seq] + r - s["cu"][seq]
        slots = s["table"][seq, (pos // P).clamp(max=most - 1)] * P + pos % P
        s["slots"] = torch.where(r < s["cu"][-1], slots, -1).to(torch.int32)
    else:
        s["q"] = (1.5 * rand(total, case["n_q"], hd)).to(dtype)
        s["out"] = torch.zeros_like(s["q"])
    return s


# ---- the operators in their plain form ----------------------------------------------------------------
def _plain_plan(s, length, n):
    """A sequence needs the pages of its len + n tokens: it gives back what it has beyond them, and takes what it lacks from the front of
    the ring, in the order of the sequences, after all that is given back has gone to the ring's end. A sequence that is too long, or whose
    pages are not there, keeps what it has, and its rows get no slots."""
    P, (S, most), N, cap = s["case"]["page"], s["table"].shape, s["free"].numel(), s["slots"].numel()
    length, n, held = length.long(), n.long(), s["held"].long()
    first, count = s["queue"][0].long(), s["queue"][1].long()
    good = (length >= 0) & (n >= 0)
    n = torch.where(good, n, 0)
    end = torch.cumsum(n, 0)
    fine = good & (length + n <= most * P) & (end <= cap)
    want = torch.where(fine, (length + n + P - 1) // P, held)
    give, take = (held - want).clamp(min=0), (want - held).clamp(min=0)
    give_end, take_end = torch.cumsum(give, 0), torch.cumsum(take, 0)
    have = count + give_end[-1]
    got = fine & ((take == 0) | (take_end <= have))
    i = torch.arange(most, device=DEVICE)
    back = (i >= want[:, None]) & (i < held[:, None])
    at = (first + count + (give_end - give)[:, None] + i - want[:, None]) % N
    ring = torch.cat([s["free"], s["free"][:1]])                # one entry more, for what is not given back
    ring.scatter_(0, torch.where(back, at, N).flatten(), s["table"].flatten())
    s["free"].copy_(ring[:N])
    new = (got[:, None] & (i >= held[:, None]) & (i < want[:, None]))
    at = (first + (take_end - take)[:, None] + i - held[:, None]) % N
    s["table"].copy_(torch.where(new, s["free"][at], s["table"]))
    used = torch.where(got & (take > 0), take_end, 0).amax()
    s["queue"].copy_(torch.stack([(first + used) % N, have - used, used * 0, used * 0]))
    s["held"].copy_(torch.where(got, want, held))
    s["cu"][1:].copy_(end.clamp(max=cap))
    r = torch.arange(cap, device=DEVICE)
    seq = torch.searchsorted(end, r, right=True).clamp(max=S - 1)
    pos = length[seq] + r - (end - n)[seq]
    slot = s["table"][seq, (pos // P).clamp(0, most - 1)] * P + pos % P
    s["slots"].copy_(torch.where(got[seq] & (r < end[-1]), slot, -1))
    return {x: s[x] for x in ("table", "held", "free", "queue", "cu", "slots")}


def _plain_append(s):
    P = s["case"]["page"]
    ok = s["slots"] >= 0
    at = torch.where(ok, s["slots"], 0).long()
    for x, new in ((s["k"], s["new_k"]), (s["v"], s["new_v"])):
        # rows without a slot write the first row's own value where that goes
        to = torch.where(ok, at, at[0])
        rows = torch.where(ok[:, None, None], new, new[0])
        x[to // P, :, to % P] = rows
    return s["k"], s["v"]


def _softmax(a, sees):
    """Weights over the last axis, in place, and their sums; a row that sees nothing gets zeros."""
    a.masked_fill_(~sees, float("-inf"))
    top = a.amax(-1, keepdim=True)
    a.sub_(torch.where(top == float("-inf"), 0.0, top)).exp_()
    total = a.sum(-1, keepdim=True)
    return a, torch.where(total > 0, total, 1.0)


def _padded(s, x, most):
    """Packed rows [rows][heads][hd] as fp32 [seq][heads][most][hd], zeros behind each sequence's."""
    m = torch.arange(most, device=DEVICE)
    at = (s["cu"][:-1, None] + m).clamp(max=x.shape[0] - 1).long()
    live = m < s["n"][:, None]
    return torch.where(live[..., None, None], x[at].float(), 0.0).transpose(1, 2)


def _unpadded(s, o):
    """fp32 [seq][heads][most][hd] into the rows of s["out"]."""
    out, most = s["out"], o.shape[2]
    r = torch.arange(out.shape[0], device=DEVICE)
    seq = torch.searchsorted(s["cu"][1:].contiguous(), r.to(torch.int32), right=True).clamp(max=o.shape[0] - 1)
    rows = o[seq, :, (r - s["cu"][seq]).clamp(0, most - 1)]
    out.copy_(torch.where((r < s["cu"][-1])[:, None, None], rows.to(out.dtype), out))
    return out


def _plain_prompt(s):
    case, most = s["case"], max(_counts(s["case"]))
    q, k, v = (_padded(s, s[x], most) for x in ("q", "new_k", "new_v"))
    S, kv, group = q.shape[0], case["n_kv"], case["n_q"] // case["n_kv"]
    i = torch.arange(most, device=DEVICE)
    sees = i <= i[:, None]
    if case["window"]:
        sees = sees & (i > i[:, None] - case["window"])
    a = torch.matmul(q.reshape(S, kv, group, most, -1) * case["head_dim"] ** -0.5, k[:, :, None].transpose(-2, -1))
    p, total = _softmax(a, sees)
    o = torch.matmul(p, v[:, :, None]) / total
    return _unpadded(s, o.reshape(S, case["n_q"], most, -1))


def _plain_attn(s):
    case, P, kv, hd = s["case"], s["case"]["page"], s["case"]["n_kv"], s["case"]["head_dim"]
    S, M, group, keys = case["seqs"], case["rows"], case["n_q"] // case["n_kv"], s["table"].shape[1] * P
    held = torch.arange(keys, device=DEVICE) < (s["len"] + s["n"])[:, None]                  # [S, keys]
    place = s["table"].long()
    k, v = (torch.where(held[:, None, :, None], s[x][place].transpose(1, 2).reshape(S, kv, keys, hd).float(), 0.0) for x in ("k", "v"))
    q = _padded(s, s["q"], M).reshape(S, kv, group, M, hd) * hd ** -0.5
    key, m = torch.arange(keys, device=DEVICE), torch.arange(M, device=DEVICE)
    length = s["len"][:, None, None].long()
    pos = length + m[:, None]
    sees = held[:, None] & ((key <= pos) if case["causal"] else (key >= 0))                  # [S, M, keys]
    if case["window"]:
        sees = sees & (key > pos - case["window"] if case["causal"] else key >= length - case["window"])
    a = torch.matmul(q.reshape(S, kv, group * M, hd), k.transpose(-2, -1)).view(S, kv, group, M, keys)
    p, total = _softmax(a, sees[:, None, None])
    o = torch.matmul(p.view(S, kv, group * M, keys), v) / total.view(S, kv, group * M, 1)
    return _unpadded(s, o.view(S, case["n_q"], M, hd))


# ---- the operators by the framework ---------------------------------------------------------------------
def _cache(s):
    """The handle that a program keeps: made at a state's first pass."""
    if "cache" not in s:
        from dflash_speculative_decode_gb300 import PagedCache
        s["cache"] = PagedCache(s["k"], s["v"], s["table"], s["held"], s["free"], s["queue"])
    return s["cache"]


def run(s):
    case = s["case"]
    if case["op"] == "plan":
        length, n = s["turns"][s["turn"]]
        s["turn"] = 1 - s["turn"]
        if own:
            _cache(s).plan(length, n, out=(s["cu"], s["slots"]))
            return {x: s[x] for x in ("table", "held", "free", "queue", "cu", "slots")}
        return _plain_plan(s, length, n)
    if case["op"] == "append":
        if own:
            _cache(s).append(s["new_k"], s["new_v"], s["slots"])
            return s["k"], s["v"]
        return _plain_append(s)
    if case["op"] == "prompt":
        return _cache(s).prompt(s["q"], s["new_k"], s["new_v"], s["cu"], window=case["window"], out=s["out"]) if own else _plain_prompt(s)
    if own:
        return _cache(s).attn(s["q"], s["cu"], s["len"], case["rows"], window=case["window"], causal=case["causal"], out=s["out"])
    return _plain_attn(s)


# ---- the definition in 64 bits, one sequence and head at a time --------------------------------------------
def _exact_rows(case, q, k, v, first, causal):
    """Attention of rows q [rows][group][hd], the first of them at position `first`, over k, v [keys][hd], in 64 bits, some rows at a time."""
    out = torch.empty_like(q)
    keys, w = k.shape[0], case["window"]
    for a in range(0, q.shape[0], 512):
        b = min(a + 512, q.shape[0])
        lo, hi = 0, (first + b if causal else keys)
        if w:
            lo = max(0, first + a - w + 1 if causal else first - w)
        scores = torch.einsum("mgd,kd->mgk", q[a:b], k[lo:hi]) / math.sqrt(q.shape[2])
        pos = torch.arange(first + a, first + b, device=q.device)[:, None, None]
        at = torch.arange(lo, hi, device=q.device)
        if causal:
            scores = scores.masked_fill(at > pos, -math.inf)
            if w:
                scores = scores.masked_fill(at <= pos - w, -math.inf)
        out[a:b] = torch.einsum("mgk,kd->mgd", torch.softmax(scores, -1), v[lo:hi])
    return out


def exact(case, seed):
    if case["op"] == "plan":                                    # whole numbers alone
        return None
    s = prepare(case, seed)
    cu, length = s["cu"].tolist(), s["len"].tolist()
    P = case.get("page", 0)
    if case["op"] == "append":
        k, v, table = s["k"].double(), s["v"].double(), s["table"].tolist()
        for i in range(case["seqs"]):
            r = cu[i]
            while r < cu[i + 1]:                                # the rows that go into one page
                pos = length[i] + r - cu[i]
                m = min(P - pos % P, cu[i + 1] - r)
                for x, new in ((k, s["new_k"]), (v, s["new_v"])):
                    x[table[i][pos // P], :, pos % P:pos % P + m] = new[r:r + m].double().transpose(0, 1)
                r += m
        return k, v
    out, group = s["out"].double().clone(), case["n_q"] // case["n_kv"]
    for i in range(case["seqs"]):
        a, b = cu[i], cu[i + 1]
        if a == b:
            continue
        end = length[i] + b - a
        for h in range(case["n_kv"]):
            if case["op"] == "prompt":
                k, v = s["new_k"][a:b, h].double(), s["new_v"][a:b, h].double()
            else:
                place = s["table"][i, :_pages(end, P)].long()
                k, v = (x[place, h].reshape(-1, case["head_dim"])[:end].double() for x in (s["k"], s["v"]))
            heads = slice(h * group, (h + 1) * group)
            out[a:b, heads] = _exact_rows(case, s["q"][a:b, heads].double(), k, v, length[i], case.get("causal", True))
    return out
