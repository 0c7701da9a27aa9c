"""The operators of a decode step that stand around the sparse layers, with their plain forms.

Each case is one pass through one operator on synthetic inputs:

  product   y_t = W x_t with W_ij = s_ig (q_ij - z_ig): 4-bit codes q, one scale s and zero point z per
            row and group of columns (without zero points z = 8)
  masked    the same where token t wants only the rows of its bit mask; the other entries are -inf
  gated     act(G x_t) * (U x_t), both matrices in 4 bits
  logits    penalties for repeated tokens, sparse biases and a bit mask on rows of logits
  rope      rotary positions on the heads of projected tokens

``run`` computes them in elementary torch operations, or, where ``own`` is true, by the library's entry
points on the handle and output buffers that ``prepare`` made.
"""
import math

import torch

own = False

BF16, F32 = torch.bfloat16, torch.float32
_TYPES = {"bf16": BF16, "f32": F32}


# --------------------------------------------------------------------------- cases
def _q4(op, name, m, n, tokens, group, zeros, x, y, scales="bf16", **more):
    return {"name": name, "op": op, "m": m, "n": n, "tokens": tokens, "group": group, "zeros": zeros, "x": x, "y": y,
            "scales": scales, **more}


def listed():
    return [
        # an attention projection of one token, the smallest call of a decode step
        _q4("product", "token_square", 4096, 4096, 1, 128, False, "bf16", "f32"),
        # the down projection of one token, fed by another layer's fp32 output
        _q4("product", "token_down_f32", 4096, 11008, 1, 64, True, "f32", "f32", "f32"),
        # five drafted tokens through a layer of odd sizes (last tile, last group and last code byte all cut)
        _q4("product", "drafts_odd", 1001, 2047, 5, 32, True, "bf16", "f32"),
        # the up projection of a batch of sequences
        _q4("product", "batch_up", 11008, 4096, 64, 128, True, "bf16", "bf16"),
        # the head of one token while a grammar leaves a few hundred tokens
        _q4("masked", "head_grammar_token", 65536, 4096, 1, 128, True, "bf16", "f32", allowed=256),
        # the head of a batch whose masks leave most of the vocabulary; the last sequence's mask is empty
        _q4("masked", "head_grammar_batch", 50021, 2048, 13, 64, False, "bf16", "f32", allowed=40000),
        # gate and up projection of one token, the output being the next sparse layer's activation
        _q4("gated", "gated_token", 11008, 4096, 1, 128, False, "bf16", "bf16", act="silu"),
        # the same for a small batch in fp32, odd sizes
        _q4("gated", "gated_batch_odd", 5461, 2001, 24, 64, True, "f32", "f32", act="gelu"),
        # the logits of one sequence
        {"name": "logits_token", "op": "logits", "rows": 1, "vocab": 65536, "history": 1500, "biases": 40, "allowed": 0, "x": "f32", "y": "f32"},
        # the logits of a batch under grammars, a long history each
        {"name": "logits_batch", "op": "logits", "rows": 96, "vocab": 131072, "history": 4000, "biases": 100, "allowed": 50000, "x": "f32", "y": "f32"},
        # queries and keys of one token far into its context
        {"name": "rope_token", "op": "rope", "tokens": 1, "heads": 40, "dim": 128, "rot": 128, "interleaved": True, "inverse": False, "first": 900000, "x": "f32", "y": "bf16"},
        # queries and keys of a prompt
        {"name": "rope_prompt", "op": "rope", "tokens": 8192, "heads": 40, "dim": 128, "rot": 128, "interleaved": False, "inverse": False, "first": 0, "x": "bf16", "y": "bf16"},
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["product", "product", "masked", "gated", "logits", "rope"])
    x, y = rng.choice(["bf16", "f32"]), rng.choice(["bf16", "f32"])
    if op in ("product", "masked", "gated"):
        most = 1 << (26 if op == "gated" else 27)
        while True:
            m, n = _log(rng, 256, 65536), _log(rng, 256, 16384)
            if rng.random() < 0.5:  # layers are usually multiples of 64; the others are cut anywhere
                m, n = max(1, m // 64) * 64, max(1, n // 64) * 64
            if m * n <= most:
                break
        tokens = 1 if rng.random() < 0.4 else _log(rng, 1, 64)
        c = {"op": op, "m": m, "n": n, "tokens": tokens, "group": rng.choice([32, 64, 128]), "zeros": rng.random() < 0.5,
             "x": x, "y": y, "scales": rng.choice(["bf16", "bf16", "f32"])}
        if op == "masked":
            c["allowed"], c["y"] = _log(rng, 1, m), "f32"
        if op == "gated":
            c["act"] = rng.choice(["silu", "gelu", "relu"])
        return c
    if op == "logits":
        while True:
            rows, vocab = _log(rng, 1, 96), _log(rng, 1000, 160000)
            if rows * vocab <= 96 * 131072:
                break
        return {"op": op, "rows": rows, "vocab": vocab, "history": _log(rng, 1, 16000 if rows < 8 else 4000), "biases": _log(rng, 1, 300),
                "allowed": rng.choice([0, _log(rng, 1, vocab)]), "x": x, "y": y}
    while True:
        tokens, heads, dim = _log(rng, 1, 8192), _log(rng, 1, 64), rng.choice([64, 80, 96, 128, 192, 256])
        if tokens * heads * dim <= 8192 * 40 * 128:
            break
    return {"op": op, "tokens": tokens, "heads": heads, "dim": dim, "rot": dim if rng.random() < 0.5 else 2 * rng.randint(1, dim // 2),
            "interleaved": rng.random() < 0.5, "inverse": rng.random() < 0.25, "first": _log(rng, 1, 1000000), "x": x, "y": y}


# --------------------------------------------------------------------------- inputs
def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(1 + int(seed))


def _weights(g, m, n, group, zeros, scales):
    """Codes as rounding to nearest makes them of normal weights, two to a byte (even column low), scales of a
    group's width and zero points near the middle."""
    nb = (n + 1) // 2
    pair = [torch.empty(m, nb, device="cuda").normal_(8, 2.4, generator=g).round_().clamp_(0, 15).to(torch.uint8) for _ in range(2)]
    if n & 1:
        pair[1][:, -1] = 0
    groups = (n + group - 1) // group
    s = (0.004 + 0.008 * torch.rand(m, groups, device="cuda", generator=g)).to(_TYPES[scales])
    z = torch.empty(m, groups, device="cuda").normal_(8, 1.2, generator=g).round_().clamp_(0, 15).to(torch.uint8) if zeros else None
    return pair[0] | (pair[1] << 4), s, z


def _mask(g, rows, vocab, allowed, empty_last):
    """int32 words whose bit v % 32 of word v // 32 allows v: half of the allowed ones in a run, the others anywhere."""
    words = (vocab + 31) // 32
    ids = torch.arange(words * 32, device="cuda")
    start = torch.randint(0, max(1, vocab - allowed // 2), (rows, 1), device="cuda", generator=g)
    bits = (ids >= start) & (ids < start + allowed // 2)
    bits |= torch.rand(rows, words * 32, device="cuda", generator=g) * vocab < (allowed - allowed // 2)
    bits &= ids < vocab
    if empty_last and rows > 1:
        bits[-1] = False
    weight = torch.ones(32, dtype=torch.int64, device="cuda") << torch.arange(32, device="cuda")
    return (bits.view(rows, words, 32) * weight).sum(-1).to(torch.int32)


def prepare(case, seed):
    g, s = _generator(seed), {"case": case}
    xt, yt = _TYPES[case["x"]], _TYPES[case["y"]]
    if case["op"] in ("product", "masked", "gated"):
        m, n, t = case["m"], case["n"], case["tokens"]
        x = torch.empty(t, n, device="cuda").normal_(generator=g)
        x[:, torch.randint(0, n, (max(1, n // 500),), device="cuda", generator=g)] *= 20  # the few large channels
        s["x"] = x.to(xt)
        s["w"] = [_weights(g, m, n, case["group"], case["zeros"], case["scales"]) for _ in range(2 if case["op"] == "gated" else 1)]
        if case["op"] == "masked":
            s["mask"] = _mask(g, t, m, case["allowed"], True)
        if own:  # the program keeps the laid out weights and an output buffer
            import spmspv_graph_traversal_amd as dbs

            s["handles"] = [dbs.dbs_q4_build(m, n, case["group"], *w) for w in s["w"]]
            s["out"] = torch.empty(t, m, dtype=yt, device="cuda")
    elif case["op"] == "logits":
        b, v = case["rows"], case["vocab"]
        s["logits"] = torch.empty(b, v, device="cuda").normal_(0, 3, generator=g).to(xt)

        def lists(length, least):
            sizes = torch.randint(least, 2 * length - least + 1, (b,), device="cuda", generator=g)
            ptr = torch.zeros(b + 1, dtype=torch.int32, device="cuda")
            ptr[1:] = sizes.cumsum(0)
            return ptr, int(ptr[-1])

        s["hist_ptr"], total = lists(case["history"], min(1, case["history"]))
        # text repeats itself: frequent ids are low ones
        s["hist"] = (v ** torch.rand(total, device="cuda", generator=g)).long().clamp_(0, v - 1).to(torch.int32)
        s["hist_new"] = ((s["hist_ptr"][1:] - s["hist_ptr"][:-1]) * 0.6).to(torch.int32)  # the prompt is the first 60 %
        s["repetition"] = 1 + 0.3 * torch.rand(b, device="cuda", generator=g)
        s["frequency"] = 0.5 * torch.rand(b, device="cuda", generator=g)
        s["presence"] = 0.5 * torch.rand(b, device="cuda", generator=g)
        s["bias_ptr"], total = lists(case["biases"], 1)
        s["bias_idx"] = torch.randint(0, v, (total,), device="cuda", generator=g).to(torch.int32)
        s["bias_val"] = torch.empty(total, device="cuda").normal_(0, 2, generator=g)
        s["mask"] = _mask(g, b, v, case["allowed"], True) if case["allowed"] else None
        if own:
            s["out"] = torch.empty(b, v, dtype=yt, device="cuda")
    else:
        t, h, d = case["tokens"], case["heads"], case["dim"]
        s["x"] = torch.empty(t, h, d, device="cuda").normal_(generator=g).to(xt)
        s["pos"] = torch.arange(case["first"], case["first"] + t, dtype=torch.int32, device="cuda")
        half = case["rot"] // 2
        s["freq"] = 500000.0 ** (-torch.arange(half, dtype=torch.float64, device="cuda") / half)
        if own:
            s["out"] = torch.empty(t, h, d, dtype=yt, device="cuda")
    return s


# --------------------------------------------------------------------------- one pass
def run(state):
    return _own(state) if own else _plain(state)


def _own(s):
    import spmspv_graph_traversal_amd as dbs

    case, out = s["case"], s["out"]
    op = case["op"]
    if op == "product":
        dbs.dbs_q4_product(s["handles"][0], s["x"], out)
    elif op == "masked":
        dbs.dbs_q4_product_masked(s["handles"][0], s["x"], s["mask"], out)
    elif op == "gated":
        act = {"silu": dbs.DBS_ACT_SILU, "gelu": dbs.DBS_ACT_GELU_TANH, "relu": dbs.DBS_ACT_RELU}[case["act"]]
        dbs.dbs_q4_gated(s["handles"][0], s["handles"][1], s["x"], act, out)
    elif op == "logits":
        dbs.dbs_logits_adjust(s["logits"], out, hist_ptr=s["hist_ptr"], hist=s["hist"], hist_new=s["hist_new"],
                              repetition=s["repetition"], frequency=s["frequency"], presence=s["presence"],
                              bias_ptr=s["bias_ptr"], bias_idx=s["bias_idx"], bias_val=s["bias_val"], mask=s["mask"])
    else:
        dbs.dbs_rope(s["x"], s["pos"], s["freq"], out, layout=dbs.DBS_ROPE_INTERLEAVED if case["interleaved"] else dbs.DBS_ROPE_HALF,
                     inverse=case["inverse"])
    return out


def _dequantized(case, codes, scales, zeros):
    m, n, group = case["m"], case["n"], case["group"]
    q = torch.stack((codes & 15, codes >> 4), -1).view(m, -1)[:, :n].float()
    of = torch.arange(n, device=codes.device) // group
    z = 8.0 if zeros is None else zeros.float()[:, of]
    return (q - z) * scales.float()[:, of]


def _allowed(mask, vocab):
    v = torch.arange(vocab, device=mask.device)
    return (mask[:, v // 32] >> (v % 32)) & 1 != 0


def _plain(s):
    case = s["case"]
    yt = _TYPES[case["y"]]
    if case["op"] in ("product", "masked", "gated"):
        x = s["x"].float()
        y = x @ _dequantized(case, *s["w"][0]).t()
        if case["op"] == "masked":
            y = torch.where(_allowed(s["mask"], case["m"]), y, -math.inf)
        if case["op"] == "gated":
            up = x @ _dequantized(case, *s["w"][1]).t()
            if case["act"] == "silu":
                a = y / (1 + torch.exp(-y))
            elif case["act"] == "gelu":
                a = 0.5 * y * (1 + torch.tanh(math.sqrt(2 / math.pi) * (y + 0.044715 * y * y * y)))
            else:
                a = torch.where(y > 0, y, 0.0)
            y = a * up
        return y.to(yt)
    if case["op"] == "logits":
        b, v = case["rows"], case["vocab"]
        l = s["logits"].float()

        def row_of(ptr, total):
            return torch.repeat_interleave(torch.arange(b, device=ptr.device), (ptr[1:] - ptr[:-1]).long(), output_size=total)

        row = row_of(s["hist_ptr"], s["hist"].numel())
        at = row * v + s["hist"]
        new = torch.arange(at.numel(), device=at.device) - s["hist_ptr"][row] >= s["hist_new"][row]
        seen = torch.zeros(b * v, dtype=torch.int32, device=at.device).index_add_(0, at, torch.ones_like(at, dtype=torch.int32)).view(b, v) > 0
        count = torch.zeros(b * v, dtype=torch.int32, device=at.device).index_add_(0, at, new.int()).view(b, v)
        r = s["repetition"][:, None]
        l = torch.where(seen, torch.where(l > 0, l / r, l * r), l)
        l = l - s["frequency"][:, None] * count - s["presence"][:, None] * (count > 0)
        at = row_of(s["bias_ptr"], s["bias_idx"].numel()) * v + s["bias_idx"]
        entry = torch.arange(1, at.numel() + 1, device=at.device)
        last = torch.zeros(b * v, dtype=torch.int64, device=at.device).scatter_reduce_(0, at, entry, "amax").view(b, v)
        l = l + torch.where(last > 0, s["bias_val"][(last - 1).clamp_min(0)], 0.0)
        if s["mask"] is not None:
            l = torch.where(_allowed(s["mask"], v), l, -math.inf)
        return l.to(yt)
    x, rot = s["x"].float(), case["rot"]
    angle = s["pos"].double()[:, None] * s["freq"]  # far positions turn many times: the angle needs 64 bits
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    if case["inverse"]:
        sin = -sin
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if case["interleaved"] else (x[..., : rot // 2], x[..., rot // 2 : rot])
    u, w = a * cos - b * sin, a * sin + b * cos
    turned = torch.stack((u, w), -1).flatten(-2) if case["interleaved"] else torch.cat((u, w), -1)
    return torch.cat((turned, x[..., rot:]), -1).to(yt)


# --------------------------------------------------------------------------- what a pass cannot do without
def work(case):
    size = {"bf16": 2, "f32": 4}
    if case["op"] in ("product", "masked", "gated"):
        m, n, t = case["m"], case["n"], case["tokens"]
        rows, mask = m, 0
        if case["op"] == "masked":  # rows that some token wants (the last of several wants none)
            wanting = t - 1 if t > 1 else 1
            rows, mask = m * (1 - (1 - min(1.0, case["allowed"] / m)) ** wanting), t * m / 8
        mats = 2 if case["op"] == "gated" else 1
        groups = (n + case["group"] - 1) // case["group"]
        per_row = n / 2 + groups * (size[case["scales"]] + (0.5 if case["zeros"] else 0))
        return {"bytes": mats * rows * per_row + mask + t * n * size[case["x"]] + t * m * size[case["y"]], "flops": 2 * mats * rows * n * t}
    if case["op"] == "logits":
        b, v = case["rows"], case["vocab"]
        read = b * (min(v, case["allowed"]) if case["allowed"] else v) * size[case["x"]]
        return {"bytes": read + b * v * size[case["y"]] + (b * v / 8 if case["allowed"] else 0) + b * (4 * case["history"] + 8 * case["biases"]),
                "flops": 4 * b * v}
    n = case["tokens"] * case["heads"] * case["dim"]
    return {"bytes": n * (size[case["x"]] + size[case["y"]]), "flops": 3 * n}


# --------------------------------------------------------------------------- the definition in 64 bits
def exact(case, seed):
    s = prepare({**case}, seed)
    if case["op"] in ("product", "masked", "gated"):
        m, n, group = case["m"], case["n"], case["group"]
        x = s["x"].to(torch.float64)
        results = []
        for codes, scales, zeros in s["w"]:
            total = torch.zeros(x.shape[0], m, dtype=torch.float64, device="cuda")
            for k in range(scales.shape[1]):  # group by group: s (sum q x - z sum x)
                low, high = k * group, min(n, (k + 1) * group)
                part = codes[:, low // 2 : (high + 1) // 2].to(torch.int64)
                dot = x[:, low:high:2] @ (part % 16).to(torch.float64).t().contiguous()
                odd = x[:, low + 1 : high : 2]
                dot += odd @ (part // 16).to(torch.float64)[:, : odd.shape[1]].t().contiguous()
                z = 8.0 if zeros is None else zeros[:, k].to(torch.float64)
                total += scales[:, k].to(torch.float64) * (dot - z * x[:, low:high].sum(1, keepdim=True))
            results.append(total)
        y = results[0]
        if case["op"] == "masked":
            words = s["mask"].to(torch.int64).repeat_interleave(32, 1)[:, :m]
            forbidden = (words // (1 << (torch.arange(m, device="cuda") % 32))) % 2 == 0
            y.masked_fill_(forbidden, -math.inf)
        if case["op"] == "gated":
            if case["act"] == "silu":
                y = y * torch.special.expit(y)
            elif case["act"] == "gelu":
                y = y * torch.special.expit(2 * math.sqrt(2 / math.pi) * (y + 0.044715 * y**3))
            else:
                y = y.clamp_min(0)
            y = y * results[1]
        return y
    if case["op"] == "logits":
        l = s["logits"].to(torch.float64)
        hp, bp = s["hist_ptr"].tolist(), s["bias_ptr"].tolist()
        new = s["hist_new"].tolist()
        for b in range(case["rows"]):
            h = s["hist"][hp[b] : hp[b + 1]].long()
            ids = h.unique()
            v, r = l[b, ids], s["repetition"][b].double()
            l[b, ids] = torch.where(v > 0, v / r, v * r)
            ids, counts = h[new[b] :].unique(return_counts=True)
            l[b, ids] -= s["frequency"][b].double() * counts + s["presence"][b].double()
            pairs = dict(zip(s["bias_idx"][bp[b] : bp[b + 1]].tolist(), s["bias_val"][bp[b] : bp[b + 1]].tolist()))
            l[b, torch.tensor(list(pairs), dtype=torch.long, device="cuda")] += torch.tensor(list(pairs.values()), dtype=torch.float64, device="cuda")
        if s["mask"] is not None:
            words = s["mask"].to(torch.int64).repeat_interleave(32, 1)[:, : case["vocab"]]
            l.masked_fill_((words // (1 << (torch.arange(case["vocab"], device="cuda") % 32))) % 2 == 0, -math.inf)
        return l
    rot = case["rot"]
    x = s["x"].to(torch.float64)
    turn = torch.polar(torch.ones(1, dtype=torch.float64, device="cuda"), s["pos"].to(torch.float64)[:, None] * s["freq"])[:, None]
    if case["inverse"]:
        turn = turn.conj()
    out = x.clone()
    first = slice(0, rot, 2) if case["interleaved"] else slice(0, rot // 2)
    second = slice(1, rot, 2) if case["interleaved"] else slice(rot // 2, rot)
    z = torch.complex(x[..., first].contiguous(), x[..., second].contiguous()) * turn
    out[..., first], out[..., second] = z.real, z.imag
    return out
