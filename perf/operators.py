"""Measured cases of the paged key/value cache operators: append with quantisation, read back, and attention
of new tokens over the cache.

A cache is a pool of pages; a page holds, for each key/value head, units of 16 tokens.  Keys and values are
stored as microscaled codes, E4M3 ("mxfp8") or E2M1 ("mxfp4"), with one E8M0 scale byte (2^(b - 127)) for each 32
consecutive elements of a token's head vector.  Within a unit the bytes stand in the order in which the attention
kernels read them:

  key codes    [piece][16 tokens][bytes of a piece]       pieces of 16 bytes of a token's codes (8 for mxfp4 at 64
                                                          elements);
  key scales   [16 tokens][elements / 32];
  value codes  [slot][4 quads][16 rows][tokens of a slot][elements / 16]
                                                          row r holds elements r * (elements / 16) .. of a token, quad
                                                          and slot the tokens: token = 4 quad + (tokens of a slot) * slot
                                                          + t, with slots of at most 16 bytes of 4 tokens;
  value scales [4 quads][elements / 32][4 tokens].
"""
import math
import random

import torch

own = False

DEV = "cuda"


# ------------------------------------------------------------------ the cases

def _case(name, op, **kw):
    c = {"name": name, "op": op, "q_heads": 32, "heads": 8, "dim": 128, "k_bits": 8, "v_bits": 8, "page": 64,
         "seqs": 1, "new_min": 1, "new_max": 1, "past_min": 0, "past_max": 0, "window": 0, "tree": False,
         "f32": False, "lengths": 1}
    c.update(kw)
    return c


def listed():
    return [
        # One decoded token after a short prompt: the call's latency is what counts.
        _case("decode_short", "attention", past_min=1036, past_max=1036),
        # Single-stream decode at the long end of a context, the 5120-wide model's 40 heads of 128.
        _case("decode_long", "attention", q_heads=40, past_min=131007, past_max=131007),
        # Served decode: 64 sequences of very different lengths, 4-bit keys with 8-bit values, small pages.
        _case("decode_batch", "attention", k_bits=4, page=16, seqs=64, past_min=1, past_max=8191, lengths=7),
        # Speculative verify: a tree of 7 drafted tokens and the token before them, everything in 4 bits.
        _case("verify_tree", "attention", q_heads=40, k_bits=4, v_bits=4, new_min=8, new_max=8, past_min=16377,
              past_max=16377, tree=True),
        # A 512-token prefill chunk in the middle of a prompt.
        _case("chunk_512", "attention", new_min=512, new_max=512, past_min=7680, past_max=7680),
        # The largest: a 2048-token chunk at the end of a 32768-token context.
        _case("chunk_2048", "attention", q_heads=40, new_min=2048, new_max=2048, past_min=30720, past_max=30720),
        # Mixed serving step with a sliding window: some sequences decode, some prefill, heads of 64.
        _case("ragged_window", "attention", q_heads=64, dim=64, seqs=7, new_min=1, new_max=301, past_min=0,
              past_max=5003, window=1024, page=32, lengths=3),
        # A chunk of a model with wide heads, 4-bit keys.
        _case("chunk_wide_heads", "attention", q_heads=24, heads=4, dim=256, k_bits=4, new_min=333, new_max=333,
              past_min=4099, past_max=4099, page=128),
        # The decode step's own write: one token of each of 64 sequences.
        _case("append_batch", "append", seqs=64, past_min=1, past_max=8191, page=16, lengths=7),
        # A prefill chunk written in 4 bits from the float32 outputs of the projection products.
        _case("append_chunk", "append", k_bits=4, v_bits=4, new_min=2048, new_max=2048, past_min=30719,
              past_max=30719, f32=True),
        # A stored prefix given back, to hand it to another program.
        _case("read_prefix", "read", new_min=65521, new_max=65521),
        # The newest tokens of several sequences, 4-bit keys, wide heads.
        _case("read_ragged", "read", heads=4, dim=256, k_bits=4, seqs=9, new_min=1, new_max=1500, past_min=0,
              past_max=3000, page=32, lengths=5),
    ]


def _between(rng, lo, hi):
    """A whole number of lo..hi, even over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))) - 0.5))))


def draw(rng):
    op = rng.choice(["attention"] * 5 + ["append"] * 2 + ["read"] * 2)
    q_heads, heads = rng.choice([(32, 8), (40, 8), (24, 4), (8, 8), (16, 1), (28, 4), (64, 8), (12, 2)])
    c = _case("", op, q_heads=q_heads, heads=heads, dim=rng.choice([64, 128, 128, 256]), k_bits=rng.choice([4, 8]),
              v_bits=rng.choice([4, 8]), page=rng.choice([16, 32, 64, 128, 256]), lengths=rng.randrange(1 << 30))
    del c["name"]
    if op == "attention":
        kind = rng.choice(["decode", "verify", "chunk", "chunk", "mixed"])
        top = {"decode": 1, "verify": _between(rng, 2, 40), "chunk": _between(rng, 65, 2048),
               "mixed": _between(rng, 16, 700)}[kind]
        c["new_max"], c["new_min"] = top, 1 if kind == "mixed" else max(1, int(top * rng.uniform(0.6, 1.0)))
        c["seqs"] = _between(rng, 1, 64 if kind == "decode" else 16 if kind == "verify" else 6)
        c["past_max"] = _between(rng, 1, 131007 if kind == "decode" and c["seqs"] < 4 else 30720)
        c["past_min"] = rng.choice([0, c["past_max"] // 2, c["past_max"]])
        c["tree"] = kind == "verify" and rng.random() < 0.5
        c["window"] = _between(rng, 100, 4096) if not c["tree"] and rng.random() < 0.3 else 0
        most = next(w for w in listed() if w["name"] == "chunk_2048")
        scores = lambda w: w["seqs"] * w["q_heads"] * w["new_max"] * (w["new_max"] + w["past_max"])
        while scores(c) > 0.9 * scores(most) or work(c)["flops"] > 0.9 * work(most)["flops"]:
            c["past_max"] = c["past_max"] * 2 // 3
            c["past_min"] = min(c["past_min"], c["past_max"])
        most = next(w for w in listed() if w["name"] == "decode_long")
        while c["seqs"] * c["heads"] * c["dim"] * (c["new_max"] + c["past_max"]) > 8 * 8 * 128 * 131072:
            c["past_max"] = c["past_max"] * 2 // 3
            c["past_min"] = min(c["past_min"], c["past_max"])
        return c
    c["f32"] = rng.random() < 0.4
    c["seqs"] = _between(rng, 1, 64)
    c["new_max"] = _between(rng, 1, max(1, (4096 if op == "append" else 65521) // c["seqs"]))
    c["new_min"] = rng.choice([1, c["new_max"]])
    c["past_max"] = _between(rng, 1, max(1, 65536 // c["seqs"]))
    c["past_min"] = rng.choice([0, c["past_max"]])
    return c


def _lengths(case):
    """(new tokens, tokens before them) of each sequence, from the case alone."""
    r = random.Random(case["lengths"])
    return [(r.randint(case["new_min"], case["new_max"]), r.randint(case["past_min"], case["past_max"]))
            for _ in range(case["seqs"])]


def _tokens(case):
    return sum(n for n, _ in _lengths(case))


def work(case):
    rows = [case["dim"] * bits // 8 + case["dim"] // 32 for bits in (case["k_bits"], case["v_bits"])]
    held = case["heads"] * sum(rows)                     # bytes of one token in the cache
    tokens = _tokens(case)
    if case["op"] != "attention":
        wide = 2 * case["heads"] * case["dim"] * tokens
        back = 2 * wide                                  # the values read back are bfloat16
        if case["op"] == "append":
            # the inputs, the cache written, the cache read back, the values that come back
            return {"bytes": (4 if case["f32"] else 2) * wide + 2 * held * tokens + back, "flops": 0}
        return {"bytes": held * tokens + back, "flops": 0}
    keys = pairs = 0
    for n, past in _lengths(case):
        first = max(0, past + 1 - case["window"]) if case["window"] else 0
        keys += past + n - first
        if case["window"]:
            pairs += sum(min(case["window"], past + i + 1) for i in range(n))
        elif case["tree"]:
            pairs += n * past + sum(bin(m).count("1") for m in _tree(case, n))
        else:
            pairs += n * past + n * (n + 1) // 2
    q = tokens * case["q_heads"] * case["dim"] * 2
    return {"bytes": keys * held + 2 * q + 4 * tokens * case["q_heads"],
            "flops": 4 * case["dim"] * case["q_heads"] * pairs}


def _tree(case, n):
    """The ancestors (and itself) of each of n drafted tokens, as bits: token 0 is the root, each other token
    hangs on an earlier one."""
    r = random.Random(case["lengths"] + n)
    masks = []
    for i in range(n):
        masks.append((masks[r.randrange(i)] if i else 0) | 1 << i)
    return masks


# ------------------------------------------------------- the inputs of a pass

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def prepare(case, seed):
    g = _gen(seed)
    lengths = _lengths(case)
    seqs, heads, dim, page = case["seqs"], case["heads"], case["dim"], case["page"]
    tokens = _tokens(case)
    context = max(n + p for n, p in lengths)
    width = -(-context // page)
    pages = sum(-(-(n + p) // page) for n, p in lengths) + 3
    # the pages of a pool in use lie in any order
    order = torch.randperm(pages, generator=g, device=DEV).tolist()
    table = torch.full((seqs, width), -1, dtype=torch.int32)
    for s, (n, p) in enumerate(lengths):
        for k in range(-(-(n + p) // page)):
            table[s, k] = order.pop()
        if case["window"]:       # pages that have left every window are given back
            table[s, :max(0, p + 1 - case["window"]) // page] = -1
    offsets = [0]
    for n, _ in lengths:
        offsets.append(offsets[-1] + n)
    state = {
        "case": dict(case), "tokens": tokens, "context": context, "max_new": max(n for n, _ in lengths),
        "table": table.to(DEV), "offsets": torch.tensor(offsets, dtype=torch.int32, device=DEV),
        "past": torch.tensor([p for _, p in lengths], dtype=torch.int32, device=DEV),
    }
    if case["op"] == "append":
        # keys and values are column ranges of one projection's output [tokens][(q_heads + 2 heads) * dim]
        cols = (case["q_heads"] + 2 * heads) * dim
        qkv = torch.randn(tokens, cols, generator=g, device=DEV)
        if not case["f32"]:
            qkv = qkv.to(torch.bfloat16)
        at = case["q_heads"] * dim
        state["k"] = qkv[:, at:at + heads * dim].view(tokens, heads, dim)
        state["v"] = qkv[:, at + heads * dim:].view(tokens, heads, dim)
        for side in ("k", "v"):
            codes, scales = _blank(case, side, pages)
            state[side + "_codes"], state[side + "_scales"] = codes, scales
    else:
        for side in ("k", "v"):
            x = torch.randn(pages, heads, page, dim, generator=g, device=DEV)
            if side == "k":      # a few large channels, as keys have them
                x.mul_(1 + 3 * (torch.rand(heads, 1, dim, generator=g, device=DEV) < 0.03))
            state[side + "_codes"], state[side + "_scales"] = _pack(side, case, *_quantize(x, case[side + "_bits"]))
            del x
    if case["op"] == "attention":
        state["q"] = (1.5 * torch.randn(tokens, case["q_heads"], dim, generator=g, device=DEV)).to(torch.bfloat16)
        state["scale"] = 1.0 / math.sqrt(dim)
        state["out"] = torch.empty_like(state["q"])
        state["lse"] = torch.empty(tokens, case["q_heads"], device=DEV)
        if case["tree"]:
            masks = [m for n, _ in lengths for m in _tree(case, n)]
            state["tree"] = torch.tensor([m - (1 << 64) if m >> 63 else m for m in masks], dtype=torch.int64, device=DEV)
    else:
        state["k_out"] = torch.empty(tokens, heads, dim, dtype=torch.bfloat16, device=DEV)
        state["v_out"] = torch.empty(tokens, heads, dim, dtype=torch.bfloat16, device=DEV)
    return state


def _blank(case, side, pages):
    tokens = pages * case["heads"] * case["page"]
    return (torch.zeros(tokens * case["dim"] * case[side + "_bits"] // 8, dtype=torch.uint8, device=DEV),
            torch.zeros(tokens * case["dim"] // 32, dtype=torch.uint8, device=DEV))


# ---------------------------------------------------------- one pass, measured

def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(state):
    import block_scaled_bit_nvfp4_amd as nv
    case = state["case"]
    if "cache" not in state:     # what a program makes once and keeps
        form = {8: nv.NVFP4_KV_MXFP8, 4: nv.NVFP4_KV_MXFP4}
        state["cache"] = nv.KvCache(state["k_codes"], state["k_scales"], state["v_codes"], state["v_scales"],
                                    form[case["k_bits"]], form[case["v_bits"]], case["page"], case["heads"],
                                    case["dim"])
        state["batch"] = nv.KvBatch(state["table"], state["offsets"], state["past"], state["tokens"],
                                    state["max_new"], state["context"])
        if case["op"] == "attention":
            need = nv.nvfp4_kv_attention_workspace_bytes(state["cache"], state["batch"], case["q_heads"])
            state["workspace"] = torch.empty(max(1, need), dtype=torch.uint8, device=DEV)
    if case["op"] == "attention":
        nv.nvfp4_kv_attention(state["cache"], state["batch"], state["q"], state["scale"], state["out"],
                              lse=state["lse"], window=case["window"], tree=state.get("tree"),
                              workspace=state["workspace"])
        return {"out": state["out"], "lse": state["lse"]}
    if case["op"] == "append":
        nv.nvfp4_kv_append(state["cache"], state["batch"], state["k"], state["v"])
    nv.nvfp4_kv_read(state["cache"], state["batch"], state["k_out"], state["v_out"])
    return {"k": state["k_out"], "v": state["v_out"]}


def _run_plain(state):
    case = state["case"]
    if case["op"] == "attention":
        return _attention_plain(state)
    token = torch.arange(state["tokens"], dtype=torch.int32, device=DEV)
    s = torch.searchsorted(state["offsets"], token, right=True) - 1
    pos = state["past"][s] + token - state["offsets"][s]
    slot = state["table"][s, (pos // case["page"]).long()].long() * case["page"] + pos % case["page"]
    if case["op"] == "append":
        planes = {}
        for side in ("k", "v"):
            codes, scales = _quantize(state[side].float(), case[side + "_bits"])
            at_codes, at_scales = _places(side, case, slot)
            planes[side] = (state[side + "_codes"].index_put_((at_codes,), _bytes(codes, case[side + "_bits"])),
                            state[side + "_scales"].index_put_((at_scales,), scales))
    else:
        planes = {side: (state[side + "_codes"], state[side + "_scales"]) for side in ("k", "v")}
    got = {}
    for side in ("k", "v"):
        at_codes, at_scales = _places(side, case, slot)
        codes, scales = planes[side][0][at_codes], planes[side][1][at_scales]
        got[side] = _values(_codes(codes, case[side + "_bits"]), scales, case[side + "_bits"]).to(torch.bfloat16)
    return got


# ------------------------------------------------------------- the plain forms

def _quantize(x, bits):
    """float32 [..., dim] -> codes uint8 [..., dim] (4-bit ones 0..15), scale bytes [..., dim / 32]."""
    blocks = x.unflatten(-1, (-1, 32))
    amax = blocks.abs().amax(-1, keepdim=True)
    part, exponent = torch.frexp(amax)                     # amax = part * 2^exponent, part in [1/2, 1)
    if bits == 8:
        e = torch.where(part <= 0.875, exponent - 9, exponent - 8)
    else:
        e = exponent - 3
    e = torch.where(amax > 0, e.clamp(-127, 127), -127)
    y = torch.ldexp(blocks, -e)
    if bits == 8:
        codes = y.to(torch.float8_e4m3fn).view(torch.uint8)
    else:
        a = y.abs()
        codes = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5))
        codes = codes | (torch.signbit(y).to(torch.uint8) << 3)
    return codes.flatten(-2), (e + 127).squeeze(-1).to(torch.uint8)


def _values(codes, scales, bits):
    """The float32 values of codes [..., dim] with scale bytes [..., dim / 32]."""
    if bits == 8:
        x = codes.view(torch.float8_e4m3fn).float()
    else:
        table = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6], device=codes.device)
        x = table[(codes & 7).long()] * (1 - 2 * (codes >> 3).float())
    power = torch.ldexp(torch.ones((), device=codes.device), scales.to(torch.int32) - 127)
    return (x.unflatten(-1, (-1, 32)) * power.unsqueeze(-1)).flatten(-2)


def _bytes(codes, bits):
    return codes if bits == 8 else codes[..., 0::2] | codes[..., 1::2] << 4


def _codes(data, bits):
    return data if bits == 8 else torch.stack((data & 15, data >> 4), -1).flatten(-2)


def _unit_shape(side, dim, bits):
    """The code bytes of a unit: their shape in memory, and the order of its axes that gives [16 tokens][bytes]."""
    row = dim * bits // 8
    if side == "k":
        piece = min(16, row // 4)
        return (row // piece, 16, piece), (1, 0, 2)        # [piece][token][byte]
    part = row // 16                                       # bytes of a token that a row holds
    per = min(16, 4 * part) // part                        # tokens of a slot
    return (4 // per, 4, 16, per, part), (1, 0, 3, 2, 4)   # [slot][quad][row][token][byte]


def _pack(side, case, codes, scales):
    """codes [pages][heads][page][dim], scales [pages][heads][page][dim / 32] -> the planes, flat."""
    bits, dim = case[side + "_bits"], case["dim"]
    data = _bytes(codes, bits)
    shape, order = _unit_shape(side, dim, bits)
    lead = data.shape[:2] + (case["page"] // 16,)
    data = data.reshape(*lead, *[shape[i] for i in order])
    back = [order.index(i) for i in range(len(order))]
    data = data.permute(0, 1, 2, *[3 + i for i in back]).contiguous().view(-1)
    if side == "v":
        scales = scales.reshape(*lead, 4, 4, dim // 32).transpose(-1, -2)
    return data, scales.contiguous().view(-1)


def _unpack(side, case, data, scales):
    """The planes' bytes of some pages [...][heads][page's bytes] -> float32 [...][heads][page][dim]."""
    bits, dim, page = case[side + "_bits"], case["dim"], case["page"]
    shape, order = _unit_shape(side, dim, bits)
    lead = data.shape[:-1]
    n = len(lead) + 1
    data = data.reshape(*lead, page // 16, *shape).permute(*range(n), *[n + i for i in order])
    data = data.reshape(*lead, page, dim * bits // 8)
    if side == "v":
        scales = scales.reshape(*lead, page // 16, 4, dim // 32, 4).transpose(-1, -2)
    return _values(_codes(data, bits), scales.reshape(*lead, page, dim // 32), bits)


def _places(side, case, slot):
    """For tokens at `slot` (page * tokens of a page + place): the plane indexes [tokens][heads][bytes] of their code
    bytes and of their scale bytes."""
    bits, dim, page, heads = case[side + "_bits"], case["dim"], case["page"], case["heads"]
    row, blocks = dim * bits // 8, dim // 32
    shape, order = _unit_shape(side, dim, bits)
    units = page // 16
    unit = ((slot // page)[:, None] * heads + torch.arange(heads, device=DEV)) * units + (slot % page // 16)[:, None]
    inner = torch.arange(16 * row, device=DEV).reshape(shape).permute(order).reshape(16, row)
    if side == "k":
        scale = torch.arange(16 * blocks, device=DEV).reshape(16, blocks)
    else:
        scale = torch.arange(16 * blocks, device=DEV).reshape(4, blocks, 4).transpose(1, 2).reshape(16, blocks)
    r = slot % 16
    return ((unit * 16 * row)[..., None] + inner[r][:, None, :], (unit * 16 * blocks)[..., None] + scale[r][:, None, :])


def _attention_plain(state):
    case = state["case"]
    heads, dim, page, seqs = case["heads"], case["dim"], case["page"], case["seqs"]
    group = case["q_heads"] // heads
    n_max = state["max_new"]
    table = state["table"]
    width = table.shape[1]
    span = width * page
    kv = []
    for side in ("k", "v"):
        data = state[side + "_codes"].view(-1, heads, page * dim * case[side + "_bits"] // 8)
        scales = state[side + "_scales"].view(-1, heads, page * dim // 32)
        at = table.clamp(min=0).long()
        x = _unpack(side, case, data[at], scales[at])                    # [seqs][width][heads][page][dim]
        kv.append(x.permute(0, 2, 1, 3, 4).reshape(seqs, heads, span, dim))
    k, v = kv
    offsets, past = state["offsets"].long(), state["past"].long()
    i = torch.arange(n_max, device=DEV)
    n = offsets[1:] - offsets[:-1]
    token = (offsets[:-1, None] + i).clamp(max=state["tokens"] - 1)      # [seqs][n_max]
    q = state["q"][token].float().view(seqs, n_max, heads, group, dim)
    q = q.permute(0, 2, 1, 3, 4).reshape(seqs, heads, n_max * group, dim)
    s = torch.matmul(q, k.transpose(-1, -2).contiguous()).mul_(state["scale"]).view(seqs, heads, n_max, group, span)
    j = torch.arange(span, device=DEV)
    pos = past[:, None] + i
    seen = j <= pos[..., None]                                           # [seqs][n_max][span]
    if case["tree"]:
        bit = (j - past[:, None]).clamp(0, 63)
        mine = state["tree"][token][..., None] >> bit[:, None, :] & 1
        new = (j >= past[:, None])[:, None, :]
        seen = torch.where(new, (mine == 1) & (j - past[:, None] < n[:, None])[:, None, :], seen)
    if case["window"]:
        seen = seen & (j > pos[..., None] - case["window"])
    s.masked_fill_(~seen[:, None, :, None, :], -math.inf)
    top = s.amax(-1, keepdim=True)
    s = s.sub_(top.clamp(min=torch.finfo(torch.float32).min)).exp_()
    total = s.sum(-1, keepdim=True)
    o = torch.matmul(s.view(seqs, heads, n_max * group, span), v).view(seqs, heads, n_max, group, dim)
    o = o / total.clamp(min=1e-38)
    lse = (top + total.log()).squeeze(-1)
    o = o.permute(0, 2, 1, 3, 4).reshape(seqs, n_max, case["q_heads"], dim)
    lse = lse.permute(0, 2, 1, 3).reshape(seqs, n_max, case["q_heads"])
    t = torch.arange(state["tokens"], device=DEV)
    at = torch.searchsorted(offsets, t, right=True) - 1
    return {"out": o[at, t - offsets[at]].to(torch.bfloat16), "lse": lse[at, t - offsets[at]]}


# ------------------------------------------------------------------ in 64 bits

def exact(case, seed):
    state = prepare(case, seed)
    if case["op"] == "attention":
        return _attention_exact(case, state)
    if case["op"] == "append":
        return {side: _rounded(state[side].double(), case[side + "_bits"]) for side in ("k", "v")}
    got = {}
    for side in ("k", "v"):
        parts = [_stored(case, state, side, s)[p:p + n] for s, (n, p) in enumerate(_lengths(case))]
        got[side] = torch.cat(parts)
    return got


def _grid(bits):
    """The non-negative values of a code's format, in order."""
    if bits == 4:
        return torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=DEV)
    small = [m * 2.0 ** -9 for m in range(8)]
    rest = [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8)]
    return torch.tensor((small + rest)[:127], dtype=torch.float64, device=DEV)


def _rounded(x, bits):
    """The nearest values to x [tokens][heads][dim] that its blocks of 32 can hold (halfway: the even code)."""
    grid = _grid(bits)
    x = x.reshape(*x.shape[:-1], -1, 32)
    amax = x.abs().amax(-1, keepdim=True)
    least = torch.full_like(amax, 2.0 ** -140)
    if bits == 4:
        e = torch.floor(torch.log2(torch.maximum(amax, least))) - 2
    else:
        e = torch.ceil(torch.log2(torch.maximum(amax, least) / 448))
    unit = torch.pow(2.0, e.clamp(-127, 127))
    a = (x.abs() / unit).clamp(max=float(grid[-1]))
    hi = torch.searchsorted(grid, a.contiguous()).clamp(max=grid.numel() - 1)
    lo = (hi - 1).clamp(min=0)
    up, down = grid[hi] - a, a - grid[lo]
    pick = torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    return (torch.sign(x) * grid[pick] * unit).flatten(-2)


def _stored(case, state, side, s):
    """The values of sequence s that the cache holds, float64 [tokens of its pages][heads][dim], code by code from
    the place of each byte."""
    bits, dim, page, heads = case[side + "_bits"], case["dim"], case["page"], case["heads"]
    table = state["table"][s].long().clamp(min=0)
    n, past = _lengths(case)[s]
    table = table[:-(-(n + past) // page)]
    row, blocks = dim * bits // 8, dim // 32
    r = torch.arange(16, device=DEV)[:, None]
    d = torch.arange(dim, device=DEV)[None, :]
    if side == "k":
        piece = min(16, row // 4)
        byte = d * bits // 8
        at = (byte // piece) * 16 * piece + r * piece + byte % piece
        scale = r * blocks + d // 32
    else:
        part = row // 16
        per = min(16, 4 * part) // part
        byte = d % (dim // 16) * bits // 8
        slot, t = r % 4 // per, r % per
        at = (((slot * 4 + r // 4) * 16 + d // (dim // 16)) * per + t) * part + byte
        scale = ((r // 4) * blocks + d // 32) * 4 + r % 4
    data = state[side + "_codes"].view(-1, heads, page // 16, 16 * row)[table][..., at]
    power = state[side + "_scales"].view(-1, heads, page // 16, 16 * blocks)[table][..., scale]
    if bits == 4:
        data = torch.where(d % 2 == 0, data % 16, data // 16)
    half = 1 << (bits - 1)
    grid = _grid(bits)
    x = grid[(data % half).long().clamp(max=grid.numel() - 1)] * torch.where(data >= half, -1.0, 1.0).double()
    x = x * torch.pow(2.0, power.double() - 127)               # [pages][heads][units][16][dim]
    return x.permute(0, 2, 3, 1, 4).reshape(-1, heads, dim)


def _attention_exact(case, state):
    group = case["q_heads"] // case["heads"]
    out = torch.zeros(state["q"].shape, dtype=torch.float64, device=DEV)
    lse = torch.full(out.shape[:2], -math.inf, dtype=torch.float64, device=DEV)
    at = 0
    for s, (n, past) in enumerate(_lengths(case)):
        first = max(0, past + 1 - case["window"]) if case["window"] else 0
        k, v = (_stored(case, state, side, s)[first:past + n] for side in ("k", "v"))
        key = torch.arange(first, past + n, device=DEV)[None, :]
        own_pos = torch.arange(past, past + n, device=DEV)[:, None]
        if case["tree"]:
            bits = torch.tensor([[m >> b & 1 for b in range(n)] for m in _tree(case, n)], device=DEV)
            hidden = torch.cat((torch.zeros(n, past, dtype=torch.bool, device=DEV), bits == 0), 1)
        else:
            hidden = key > own_pos
        if case["window"]:
            hidden = hidden | (own_pos - key >= case["window"])
        for h in range(case["q_heads"]):
            z = state["q"][at:at + n, h].double() @ k[:, h // group].T * state["scale"]
            z = z.masked_fill(hidden, -math.inf)
            lse[at:at + n, h] = torch.logsumexp(z, -1)
            out[at:at + n, h] = torch.softmax(z, -1) @ v[:, h // group]
        at += n
    return {"out": out, "lse": lse}
