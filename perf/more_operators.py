"""The attention of a decode step, between the projections of a token and its output projection, with plain forms.

Each case is one pass through one operator on synthetic inputs:

  norm_rope  root mean square norm of each query and key head, then rotary positions:
             y = turn(position * frequency) (w * x / sqrt(mean(x^2) + eps))
  store      keys and values of new tokens into a paged cache of 4-bit codes, and what the cache holds of them
  attention  softmax attention of each sequence's new tokens over its cache: token j is seen from position i if
             j <= i and, with a window, j < sinks or j > i - window

A group of the cache (32, 64 or 128 channels of a head of a token) is held as 4-bit codes q with b = half(min),
s = half((max - b) * (1/15)), q = rint((x - b) * (1/s)) within 0..15 (each step in fp32) and stands for half(s q + b).

``run`` computes them in elementary torch operations, or, where ``own`` is true, by the library's entry points.
"""
import math
import random

import torch

own = False

BF16, F32, F16 = torch.bfloat16, torch.float32, torch.float16
_TYPES = {"bf16": BF16, "f32": F32}
_EPS = 1e-6


# --------------------------------------------------------------------------- cases
def _norm(name, tokens, heads, kv_heads, dim, rot, interleaved, first, x, y):
    return {"name": name, "op": "norm_rope", "tokens": tokens, "heads": heads, "kv_heads": kv_heads, "dim": dim, "rot": rot,
            "interleaved": interleaved, "first": first, "x": x, "y": y}


def _cached(op, name, sequences, new, ragged, context, kv_heads, dim, group, page, x, y, **more):
    return {"name": name, "op": op, "sequences": sequences, "new": new, "ragged": ragged, "context": context,
            "kv_heads": kv_heads, "dim": dim, "group": group, "page": page, "x": x, "y": y, **more}


def listed():
    return [
        # queries and keys of one token far into its context, the smallest call of a step
        _norm("norm_rope_token", 1, 32, 8, 128, 128, False, 900000, "bf16", "bf16"),
        # heads of an odd size, half of which turns, in a small batch of fp32 projections
        _norm("norm_rope_odd", 333, 14, 2, 80, 40, True, 5000, "f32", "bf16"),
        # queries and keys of a prompt
        _norm("norm_rope_prompt", 8192, 32, 8, 128, 128, False, 0, "bf16", "bf16"),
        # the new token of each sequence of a batch
        _cached("store", "store_step", 64, 1, False, 8192, 8, 128, 128, 64, "bf16", "bf16"),
        # prompts of several lengths, some of them continued inside a page
        _cached("store", "store_prompts", 5, 3000, True, 4000, 8, 128, 64, 16, "bf16", "bf16"),
        # one token of one short sequence: latency
        _cached("attention", "attention_token", 1, 1, False, 1500, 8, 128, 128, 64, "bf16", "bf16", heads=32, window=0, sinks=0),
        # one token of one sequence that fills a long cache
        _cached("attention", "attention_long", 1, 1, False, 131072, 8, 128, 128, 64, "bf16", "bf16", heads=32, window=0, sinks=0),
        # one token each of a batch of sequences of different lengths
        _cached("attention", "attention_batch", 64, 1, False, 8000, 8, 128, 128, 64, "bf16", "bf16", heads=32, window=0, sinks=0),
        # a batch far beyond its window, whose pages between the first tokens and the window have been freed
        _cached("attention", "attention_sinks", 96, 1, False, 30000, 4, 64, 32, 16, "bf16", "bf16", heads=32, window=1024, sinks=4),
        # drafted tokens in fp32, seven query heads to a key head, heads of an odd size, one slot of the batch empty
        _cached("attention", "attention_drafts", 7, 5, False, 3001, 2, 80, 32, 32, "f32", "f32", heads=14, window=0, sinks=0),
        # a prompt
        _cached("attention", "attention_prompt", 1, 8192, False, 8192, 8, 128, 128, 64, "bf16", "bf16", heads=32, window=0, sinks=0),
        # pieces of prompts of several lengths under a window
        _cached("attention", "attention_pieces", 3, 1100, True, 20000, 8, 128, 64, 64, "bf16", "bf16", heads=32, window=4096, sinks=4),
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def _padded(dim):
    return next(d for d in (64, 96, 128, 192, 256) if d >= dim)


def draw(rng):
    op = rng.choice(["norm_rope", "store", "attention", "attention", "attention"])
    x, y = rng.choice(["bf16", "bf16", "f32"]), rng.choice(["bf16", "bf16", "f32"])
    dim = rng.choice([64, 80, 96, 128, 128, 128, 192, 256])
    if op == "norm_rope":
        while True:
            tokens, heads, kv_heads = _log(rng, 1, 8192), _log(rng, 1, 64), rng.choice([1, 2, 4, 5, 8])
            if tokens * (heads + kv_heads) * dim <= 8192 * 40 * 128:
                break
        return {"op": op, "tokens": tokens, "heads": heads, "kv_heads": kv_heads, "dim": dim,
                "rot": dim if rng.random() < 0.6 else 2 * rng.randint(1, dim // 2), "interleaved": rng.random() < 0.4,
                "first": _log(rng, 1, 1000000), "x": x, "y": y}
    c = {"op": op, "kv_heads": rng.choice([1, 2, 4, 5, 8]), "dim": dim,
         "group": rng.choice([g for g in (32, 64, 128) if _padded(dim) % g == 0]), "page": rng.choice([16, 32, 64, 128]),
         "ragged": rng.random() < 0.5, "x": x, "y": y}
    if op == "store":
        while True:
            c["sequences"] = _log(rng, 1, 96)
            c["new"] = 1 if rng.random() < 0.4 else _log(rng, 1, 8192)
            if c["sequences"] * c["new"] * c["kv_heads"] * dim <= 8192 * 8 * 128:
                break
        c["context"] = c["new"] + rng.randint(0, 2000)
        return c
    c["heads"] = c["kv_heads"] * rng.choice([1, 2, 3, 4, 4, 7, 8, 16])
    kind = rng.choice(["token", "token", "drafts", "prompt"])
    c["window"] = 0 if rng.random() < 0.6 else _log(rng, 1, 8192)
    c["sinks"] = rng.choice([0, 1, 4, 4, 20]) if c["window"] else 0
    while True:
        c["sequences"] = _log(rng, 1, 96 if kind != "prompt" else 8)
        c["new"] = 1 if kind == "token" else rng.randint(2, 8) if kind == "drafts" else _log(rng, 9, 8192)
        c["context"] = max(c["new"], _log(rng, 1, 131072))
        cells = c["sequences"] * c["context"] * c["kv_heads"] * dim
        pairs = c["sequences"] * c["new"] * c["heads"] * c["context"]
        if cells <= 64 * 4500 * 8 * 128 and pairs * dim <= 8192 * 8192 * 32 * 128 // 2 and pairs <= 1 << 30:
            return c


def _lengths(case):
    """(tokens in the cache, new ones among them) of each sequence: lists that belong to the case."""
    r = random.Random(str(sorted((k, v) for k, v in case.items() if k != "name")))
    b, new, context = case["sequences"], case["new"], case["context"]
    count = [max(1, int(new * r.uniform(0.2, 1))) if case["ragged"] and b > 1 else new for _ in range(b)]
    length = [max(n, int(context * r.uniform(0.25, 1))) if b > 1 else context for n in count]
    length[0] = context
    if case["op"] == "attention" and 1 < b < 16 and not case["ragged"]:
        length[-1] = 0  # a slot of the batch that no sequence has taken
    return length, count


# --------------------------------------------------------------------------- the cache's layout
# A page holds for each key head: key codes, key records, value codes, value records (d: padded head size).
#   key codes      [token][4 g][d/32 k] words of 8 nibbles e: channel 32 k + 8 g + e
#   key records    [token][group] pairs of halves s, b
#   value codes    [token / 8][16 c][d/16 n] words of 8 nibbles e: channel 16 n + c of token 8 (token / 8) + e
#   value records  [token / 8][group] 8 halves s, 8 halves b of tokens 0 4 1 5 2 6 3 7
_ORDER = [0, 4, 1, 5, 2, 6, 3, 7]
_PLACE = [0, 2, 4, 6, 1, 3, 5, 7]  # of token e among them


def _sections(case):
    d, page = _padded(case["dim"]), case["page"]
    codes, records = page * d // 2, page * (d // case["group"]) * 4
    return codes, records, 2 * (codes + records)


def _quantize(x, case):
    """Codes [..., d] (uint8) and records s, b [..., groups] (fp16) of x [..., dim], padded channels being 0."""
    d, group = _padded(case["dim"]), case["group"]
    x = x.float()
    pad = [d - case["dim"]]
    real = torch.arange(d, device=x.device).view(-1, group) < case["dim"]
    x = torch.nn.functional.pad(x, (0, pad[0])).unflatten(-1, (-1, group))
    low = torch.where(real, x, math.inf).amin(-1)
    high = torch.where(real, x, -math.inf).amax(-1)
    some = real.any(-1)
    low, high = torch.where(some, low, 0.0), torch.where(some, high, 0.0)
    b = low.to(F16)
    fifteenth = torch.tensor(1 / 15, dtype=F32, device=x.device)
    s = ((high - b.float()) * fifteenth).clamp_min(0).to(F16)
    inverse = torch.where(s > 0, (1.0 / s.double()).float(), 0.0)
    q = torch.round((x - b.float()[..., None]) * inverse[..., None]).clamp(0, 15)
    q = torch.where(real, q, 0.0)
    return q.to(torch.uint8).flatten(-2), s, b


def _value(q, s, b, case):
    """What codes [..., d] with records [..., groups] stand for."""
    q = q.float().unflatten(-1, (-1, case["group"]))
    return (s.float()[..., None] * q + b.float()[..., None]).to(F16).float().flatten(-2)[..., : case["dim"]]


def _pack_pages(k, v, case):
    """Bytes [pages, page bytes] of quantized k and v (codes [pages, page, heads, d], records [pages, page, heads, groups])."""
    d, page = _padded(case["dim"]), case["page"]
    (kq, ks, kb), (vq, vs, vb) = ([t.transpose(1, 2) for t in x] for x in (k, v))  # [pages, heads, page, ...]
    n, h = kq.shape[:2]

    def words(nibbles):  # [..., 8] in order -> bytes
        return (nibbles[..., 0::2] | (nibbles[..., 1::2] << 4)).reshape(n, h, -1)

    kw = words(kq.unflatten(-1, (d // 32, 4, 8)).transpose(-3, -2))
    kr = torch.stack((ks, kb), -1).contiguous().view(torch.uint8).reshape(n, h, -1)
    vw = words(vq.unflatten(2, (page // 8, 8)).unflatten(-1, (d // 16, 16)).permute(0, 1, 2, 5, 4, 3))
    vr = torch.stack((vs, vb), -1).unflatten(2, (page // 8, 8))[:, :, :, _ORDER].permute(0, 1, 2, 4, 5, 3).contiguous()
    return torch.cat((kw, kr, vw, vr.view(torch.uint8).reshape(n, h, -1)), -1).reshape(n, -1)


def _unpack_pages(pages, case):
    """The values of pages [..., page bytes]: k, v [..., heads, page, dim] in fp32."""
    d, page, groups = _padded(case["dim"]), case["page"], _padded(case["dim"]) // case["group"]
    codes, records, _ = _sections(case)
    lead = pages.shape[:-1]
    part = pages.view(*lead, case["kv_heads"], -1).split([codes, records, codes, records], -1)

    def nibbles(w):
        return torch.stack((w & 15, w >> 4), -1).flatten(-2)

    def halves(r):
        return r.contiguous().view(F16)

    kq = nibbles(part[0]).unflatten(-1, (page, 4, d // 32, 8)).transpose(-3, -2).flatten(-3)
    kr = halves(part[1]).unflatten(-1, (page, groups, 2))
    vq = nibbles(part[2]).unflatten(-1, (page // 8, 16, d // 16, 8)).transpose(-1, -3).flatten(-2).flatten(-3, -2)
    vr = halves(part[3]).unflatten(-1, (page // 8, groups, 2, 8))[..., _PLACE].movedim(-1, -3).flatten(-4, -3)
    return _value(kq, kr[..., 0], kr[..., 1], case), _value(vq, vr[..., 0], vr[..., 1], case)


# --------------------------------------------------------------------------- inputs
def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(1 + int(seed))


def _key_values(g, case, *shape):
    """Keys with the few large channels that keys have, and values."""
    h, d = case["kv_heads"], case["dim"]
    k = torch.empty(*shape, h, d, device="cuda").normal_(generator=g)
    v = torch.empty(*shape, h, d, device="cuda").normal_(generator=g)
    at = torch.arange(h * d, device="cuda").view(h, d)
    return k + torch.where(at % 37 == 5, 4.0, 0.0), v


def _first_page(case, length, count):
    """Pages of the first tokens, and the first page behind them that a new token sees."""
    if not case["window"]:
        return 0, 0
    sink_pages = -(-min(case["sinks"], length) // case["page"])
    return sink_pages, max(sink_pages, max(0, length - count - case["window"] + 1) // case["page"])


def prepare(case, seed):
    g, s = _generator(seed), {"case": case}
    xt, yt = _TYPES[case["x"]], _TYPES[case["y"]]
    if case["op"] == "norm_rope":
        t, d, half = case["tokens"], case["dim"], case["rot"] // 2
        # one row of a fused projection: queries, keys and values of a token
        row = torch.empty(t, case["heads"] + 2 * case["kv_heads"], d, device="cuda").normal_(0, 3, generator=g).to(xt)
        s["q"], s["k"] = row[:, : case["heads"]], row[:, case["heads"] : case["heads"] + case["kv_heads"]]
        s["qw"], s["kw"] = ((1 + 0.2 * torch.randn(d, device="cuda", generator=g)).to(BF16) for _ in range(2))
        s["pos"] = torch.arange(case["first"], case["first"] + t, dtype=torch.int32, device="cuda")
        s["freq"] = 500000.0 ** (-torch.arange(half, dtype=torch.float64, device="cuda") / half)
        s["q_out"] = torch.empty(t, case["heads"], d, dtype=yt, device="cuda")
        s["k_out"] = torch.empty(t, case["kv_heads"], d, dtype=yt, device="cuda")
        return s
    page, store = case["page"], case["op"] == "store"
    length, count = _lengths(case)
    width = max(-(-max(length) // page), 1)
    # pages that hold a token which a new one sees (all that are written, for a store); the others have been freed
    held = []
    for b, (n, c) in enumerate(zip(length, count)):
        sinks, first = (0, (n - c) // page) if store else _first_page(case, n, c)
        held += [b * width + p for p in range(-(-n // page)) if p < sinks or p >= first]
    pages = max(1, len(held))
    table = torch.full((case["sequences"] * width,), -1, dtype=torch.int32, device="cuda")
    where = torch.randperm(pages, device="cuda", generator=g).to(torch.int32)
    if held:
        table[torch.tensor(held, device="cuda")] = where[: len(held)]
    s["table"] = table.view(-1, width)
    s["lens"] = torch.tensor(length, dtype=torch.int32, device="cuda")
    ends = torch.tensor([0] + count, dtype=torch.int32).cumsum(0).to(torch.int32)
    s["new_ptr"] = ends.cuda() if case["ragged"] else None
    total = int(ends[-1])
    s["pool"] = torch.empty(pages, _sections(case)[2] * case["kv_heads"], dtype=torch.uint8, device="cuda")
    if store:
        s["pool"].random_(0, 256, generator=g)  # what pages held before
        s["k"], s["v"] = (t.to(xt) for t in _key_values(g, case, total))
        s["k_out"], s["v_out"] = (torch.empty(total, case["kv_heads"], case["dim"], dtype=yt, device="cuda") for _ in range(2))
    else:
        step = max(1, (1 << 26) // (page * case["kv_heads"] * case["dim"]))
        for p in range(0, pages, step):
            n = min(step, pages - p)
            k, v = _key_values(g, case, n, page)
            s["pool"][p : p + n] = _pack_pages(_quantize(k, case), _quantize(v, case), case)
        # queries that single some keys out
        s["q"] = torch.empty(total, case["heads"], case["dim"], device="cuda").normal_(0, 2, generator=g).to(xt)
        s["out"] = torch.empty(total, case["heads"], case["dim"], dtype=yt, device="cuda")
    if own:  # the program keeps the cache's description
        import spmspv_graph_traversal_amd as dbs

        s["cache"] = dbs.dbs_kv4_cache(pages, case["kv_heads"], case["dim"], case["group"], page, pool=s["pool"])
    return s


# --------------------------------------------------------------------------- one pass
def run(state):
    return _own(state) if own else _plain(state)


def _own(s):
    import spmspv_graph_traversal_amd as dbs

    case = s["case"]
    if case["op"] == "norm_rope":
        dbs.dbs_norm_rope(s["q"], s["k"], s["qw"], s["kw"], s["pos"], s["freq"], s["q_out"], s["k_out"], eps=_EPS,
                          layout=dbs.DBS_ROPE_INTERLEAVED if case["interleaved"] else dbs.DBS_ROPE_HALF)
        return s["q_out"], s["k_out"]
    if case["op"] == "store":
        dbs.dbs_kv4_store(s["cache"], s["table"], s["lens"], s["k"], s["v"], new_ptr=s["new_ptr"], k_out=s["k_out"], v_out=s["v_out"])
        return {"pool": s["pool"], "k": s["k_out"], "v": s["v_out"]}
    dbs.dbs_kv4_attention(s["cache"], s["table"], s["lens"], s["q"], s["out"], new_ptr=s["new_ptr"], window=case["window"], sinks=case["sinks"])
    return s["out"]


def _plain(s):
    return {"norm_rope": _plain_norm_rope, "store": _plain_store, "attention": _plain_attention}[s["case"]["op"]](s)


def _plain_norm_rope(s):
    case, rot = s["case"], s["case"]["rot"]
    angle = s["pos"].double()[:, None] * s["freq"]  # far positions turn many times: the angle needs 64 bits
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]

    def one(x, w):
        x = x.float()
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + _EPS) * w.float()
        a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if case["interleaved"] else (x[..., : rot // 2], x[..., rot // 2 : rot])
        u, v = a * cos - b * sin, a * sin + b * cos
        turned = torch.stack((u, v), -1).flatten(-2) if case["interleaved"] else torch.cat((u, v), -1)
        return torch.cat((turned, x[..., rot:]), -1).to(_TYPES[case["y"]])

    return one(s["q"], s["qw"]), one(s["k"], s["kw"])


def _rows(s, total):
    """Sequence and position of each new token."""
    b, device = s["lens"].numel(), s["lens"].device
    if s["new_ptr"] is None:
        first = torch.arange(b + 1, device=device) * (total // b)
    else:
        first = s["new_ptr"].long()
    row = torch.arange(total, device=device)
    of = torch.searchsorted(first[1:].contiguous(), row, right=True)
    return of, s["lens"].long()[of] - first[of + 1] + row, row - first[of]


def _plain_store(s):
    case, page, h = s["case"], s["case"]["page"], s["case"]["kv_heads"]
    d, groups = _padded(case["dim"]), _padded(case["dim"]) // case["group"]
    codes, records, size = _sections(case)
    of, pos, _ = _rows(s, s["k"].shape[0])
    base = s["table"][of, pos // page].long()[:, None] * (size * h) + torch.arange(h, device=pos.device) * size  # bytes, [tokens, heads]
    t = (pos % page)[:, None]
    (kq, ks, kb), (vq, vs, vb) = _quantize(s["k"], case), _quantize(s["v"], case)
    pool = s["pool"].view(-1)
    words, halves = pool.view(torch.int32), pool.view(F16)
    device = pos.device
    # keys: whole words and records
    w = kq.long().unflatten(-1, (d // 32, 4, 8)).transpose(-3, -2).flatten(-3, -2)
    w = (w << (4 * torch.arange(8, device=device))).sum(-1)
    w = torch.where(w >= 1 << 31, w - (1 << 32), w).to(torch.int32)
    words[((base + t * (d // 2)) // 4)[..., None] + torch.arange(d // 8, device=device)] = w
    at = (base + codes + t * (groups * 4))[..., None] // 2 + 2 * torch.arange(groups, device=device)
    halves[at], halves[at + 1] = ks, kb
    # values: one nibble of a word that eight tokens share
    e = (t % 8)[..., None]
    channel = torch.arange(d, device=device)
    at = ((base + codes + records + t // 8 * (d * 4)) // 4)[..., None] + channel % 16 * (d // 16) + channel // 16
    bits = torch.zeros(words.numel(), dtype=torch.int64, device=device).index_add_(0, at.flatten(), (vq.long() << (4 * e)).flatten())
    mask = torch.zeros_like(bits).index_add_(0, at.flatten(), (15 << (4 * e)).expand_as(at).flatten())
    both = (words.long() & ~mask) | bits
    both &= 0xFFFFFFFF
    words.copy_(torch.where(both >= 1 << 31, both - (1 << 32), both).to(torch.int32))
    place = torch.tensor(_PLACE, device=device)[t % 8]
    at = (base + 2 * codes + records + t // 8 * (groups * 32))[..., None] // 2 + 16 * torch.arange(groups, device=device) + place[..., None]
    halves[at], halves[at + 8] = vs, vb
    s["k_out"].copy_(_value(kq, ks, kb, case))
    s["v_out"].copy_(_value(vq, vs, vb, case))
    return {"pool": s["pool"], "k": s["k_out"], "v": s["v_out"]}


def _plain_attention(s):
    case, page, hk, dim = s["case"], s["case"]["page"], s["case"]["kv_heads"], s["case"]["dim"]
    window, sinks, rep = case["window"], case["sinks"], case["heads"] // case["kv_heads"]
    total, device = s["q"].shape[0], s["q"].device
    length, count = _lengths(case)
    of, pos, nth = _rows(s, total)
    # the pages that a sequence's new tokens see, as one list each
    spans = [_first_page(case, n, c) + (-(-n // page),) for n, c in zip(length, count)]
    lead, tail = max(x[0] for x in spans), max(1, max(x[2] - x[1] for x in spans))
    first = torch.tensor([x[1] for x in spans], device=device)[:, None]
    last = torch.tensor([x[2] for x in spans], device=device)[:, None]
    logical = torch.cat((torch.arange(lead, device=device).expand(len(spans), -1), first + torch.arange(tail, device=device)), 1)
    mine = torch.cat((logical[:, :lead] < first, logical[:, lead:] < last), 1)
    mine &= logical < last
    physical = torch.where(mine, s["table"].gather(1, logical.clamp_max(s["table"].shape[1] - 1)), 0).clamp_min(0)
    k, v = _unpack_pages(s["pool"][physical], case)  # [sequences, pages, heads, page, dim]
    k, v = (x.transpose(1, 2).flatten(2, 3).flatten(0, 1) for x in (k, v))  # [sequences * heads, tokens, dim]
    at = (logical[..., None] * page + torch.arange(page, device=device)).masked_fill(~mine[..., None], 1 << 40).flatten(1)
    # queries, padded to as many in each sequence
    most, b = max(count), len(spans)
    q = torch.zeros(b, most, hk, rep, dim, device=device)
    q[of, nth] = s["q"].float().view(total, hk, rep, dim)
    p = torch.full((b, most), -1, dtype=torch.int64, device=device)
    p[of, nth] = pos
    sees = at[:, None] <= p[..., None]
    if window:
        sees &= (at[:, None] < sinks) | (at[:, None] > p[..., None] - window)
    score = q.permute(0, 2, 1, 3, 4).reshape(b * hk, most * rep, dim) @ k.transpose(1, 2).contiguous()
    score = score.mul_(1 / math.sqrt(dim)).view(b, hk, most, rep, -1)
    score.masked_fill_(~sees[:, None, :, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    e = score.sub_(torch.where(top > -math.inf, top, 0.0)).exp_()
    o = (e.view(b * hk, most * rep, -1) @ v).view(b, hk, most, rep, dim)
    o = o / e.sum(-1, keepdim=True).clamp_min(1e-30)  # a row that sees a token has a sum of at least 1
    return o.permute(0, 2, 1, 3, 4)[of, nth].reshape(total, case["heads"], dim).to(_TYPES[case["y"]])


# --------------------------------------------------------------------------- what a pass cannot do without
def _seen(first, count, window, sinks):
    """Pairs of a query at position first + i, i < count, and a token that it sees; tokens that any of them sees."""
    if first < 0:
        first, count = 0, max(0, first + count)
    if not count:
        return 0, 0
    end = first + count
    if not window:
        return count * (first + 1 + end) // 2, end
    pairs = sum(min(p + 1, window) + min(sinks, max(0, p + 1 - window)) for p in range(first, end))
    low = max(0, first - window + 1)
    return pairs, end - low + min(sinks, low)


def work(case):
    size = {"bf16": 2, "f32": 4}
    if case["op"] == "norm_rope":
        n = case["tokens"] * (case["heads"] + case["kv_heads"]) * case["dim"]
        return {"bytes": n * (size[case["x"]] + size[case["y"]]), "flops": 7 * n}
    length, count = _lengths(case)
    token = case["kv_heads"] * _sections(case)[2] // case["page"]
    if case["op"] == "store":
        n = sum(count) * case["kv_heads"] * case["dim"]
        return {"bytes": 2 * n * (size[case["x"]] + size[case["y"]]) + sum(count) * token, "flops": 12 * n}
    seen = [_seen(n - c, c, case["window"], case["sinks"]) for n, c in zip(length, count)]
    rows = sum(count) * case["heads"] * case["dim"]
    return {"bytes": sum(x[1] for x in seen) * token + rows * (size[case["x"]] + size[case["y"]]),
            "flops": 4 * sum(x[0] for x in seen) * case["heads"] * case["dim"]}


# --------------------------------------------------------------------------- the definition in 64 bits
def _exact_token(pool, case, pages, tokens, head, values):
    """Keys (or values) of one head at slot `tokens` of `pages`, read word by word from the layout, in 64 bits."""
    d, dim, group, page = _padded(case["dim"]), case["dim"], case["group"], case["page"]
    codes, records, size = _sections(case)
    base = pages.long() * pool.shape[1] + head * size
    flat, c = pool.view(-1), torch.arange(dim, device=pool.device)
    t = tokens.long()
    if values:
        word = (t // 8 * d)[:, None] + c % 16 * (d // 16) + c // 16
        nibble = (t % 8)[:, None].expand_as(word)
        at = base[:, None] + codes + records + 4 * word + nibble // 2
        place = t % 4 * 2 + t % 8 // 4
        rec = (base + 2 * codes + records + t // 8 * (d // group * 32) + 2 * place)[:, None] + c // group * 32
        step = 16
    else:
        word = (t * (d // 8))[:, None] + c % 32 // 8 * (d // 32) + c // 32
        nibble = (c % 8).expand_as(word)
        at = base[:, None] + 4 * word + nibble // 2
        rec = (base + codes + t * (d // group * 4))[:, None] + c // group * 4
        step = 2
    q = (flat[at].long() // torch.where(nibble % 2 == 0, 1, 16)) % 16
    halves = flat.view(F16)
    s, b = halves[rec // 2].double(), halves[(rec + step) // 2].double()
    return (s * q + b).to(F16).double()


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm_rope":
        rot, results = case["rot"], []
        turn = torch.polar(torch.ones(1, dtype=torch.float64, device="cuda"), s["pos"].double()[:, None] * s["freq"])[:, None]
        first = slice(0, rot, 2) if case["interleaved"] else slice(0, rot // 2)
        second = slice(1, rot, 2) if case["interleaved"] else slice(rot // 2, rot)
        for x, w in ((s["q"], s["qw"]), (s["k"], s["kw"])):
            x = x.double()
            x = w.double() * x * (x.square().sum(-1, keepdim=True) / case["dim"] + _EPS).rsqrt()
            out = x.clone()
            z = torch.complex(x[..., first].contiguous(), x[..., second].contiguous()) * turn
            out[..., first], out[..., second] = z.real, z.imag
            results.append(out)
        return tuple(results)
    if case["op"] == "store":
        results = []
        for x in (s["k"], s["v"]):
            x, out = x.double(), torch.empty(x.shape, dtype=torch.float64, device="cuda")
            for low in range(0, case["dim"], case["group"]):
                part = x[..., low : low + case["group"]]
                b = part.amin(-1, keepdim=True).to(F16)
                # the records and the scaled distances are defined by their steps in fp32
                scale = ((part.amax(-1, keepdim=True).float() - b.float()) * torch.tensor(1 / 15, device="cuda")).clamp_min(0).to(F16).double()
                steps = (part.float() - b.float()) * (1 / scale).float()
                q = torch.where(scale > 0, steps.double().round().clamp(0, 15), 0.0)
                out[..., low : low + case["group"]] = (scale * q + b.double()).to(F16).double()
            results.append(out)
        return {"pool": None, "k": results[0], "v": results[1]}
    length, count = _lengths(case)
    out = torch.zeros(sum(count), case["heads"], case["dim"], dtype=torch.float64, device="cuda")
    window, rep, row = case["window"], case["heads"] // case["kv_heads"], 0
    for b, (n, c) in enumerate(zip(length, count)):
        at = torch.arange(n, device="cuda")
        if window:
            at = at[(at < case["sinks"]) | (at > n - c - window)]
        pages = s["table"][b][at // case["page"]]
        for h in range(case["kv_heads"] if n else 0):
            k = _exact_token(s["pool"], case, pages, at % case["page"], h, False)
            v = _exact_token(s["pool"], case, pages, at % case["page"], h, True)
            for low in range(0, c, 2048):
                p = torch.arange(n - c + low, n - c + min(c, low + 2048), device="cuda")
                hidden = at > p[:, None]
                if window:
                    hidden |= (at >= case["sinks"]) & (at <= p[:, None] - window)
                rows = slice(row + low, row + low + p.numel())
                for i in range(h * rep, (h + 1) * rep):
                    score = s["q"][rows, i].double() @ k.t() / math.sqrt(case["dim"])
                    out[rows, i] = torch.softmax(score.masked_fill(hidden, -math.inf), -1).nan_to_num(0.0) @ v
        row += c
    return out
