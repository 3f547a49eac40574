"""Measured cases of what a long decode needs around its products and its attention: rotary positions of several
axes, the attention weight that each cached key has gathered, eviction from the cache by it, and the log probabilities
of tokens with their entropy and top alternatives.

The cache is the paged one of perf/operators.py: a pool of pages; a page holds, for each key/value head, units of 16
tokens.  Keys and values are microscaled codes, E4M3 (8 bits) or E2M1 (4 bits), with one E8M0 scale byte (2^(b - 127))
for each 32 consecutive elements of a token's head vector.  The bytes of a unit:

  key codes    [piece][16 tokens][bytes of a piece]       pieces of 16 bytes of a token's codes (8 for 4 bits at 64
                                                          elements);
  key scales   [16 tokens][elements / 32];
  value codes  [slot][4 quads][16 rows][tokens of a slot][elements / 16]
                                                          row r holds elements r * (elements / 16) .. of a token;
                                                          token = 4 quad + (tokens of a slot) * slot + t, slots of at
                                                          most 16 bytes of 4 tokens;
  value scales [4 quads][elements / 32][4 tokens].
"""
import math
import random

import torch

own = False

DEV = "cuda"


# ------------------------------------------------------------------ the cases

def _rope(name, **kw):
    c = {"name": name, "op": "rope", "tokens": 1, "q_heads": 32, "heads": 8, "dim": 128, "rotary": 128, "axes": 1,
         "mixed": False, "adjacent": False, "f32": True, "factor": 1.0, "far": 4096}
    return {**c, **kw}


def _logprobs(name, **kw):
    c = {"name": name, "op": "logprobs", "rows": 1, "vocab": 151936, "given": 1, "top": 20, "f32": True, "scale": 1.0,
         "masked": False}
    return {**c, **kw}


def _cached(name, op, **kw):
    c = {"name": name, "op": op, "q_heads": 32, "heads": 8, "dim": 128, "k_bits": 8, "v_bits": 8, "page": 64, "seqs": 1,
         "new_min": 1, "new_max": 1, "past_min": 0, "past_max": 0, "lengths": 1}
    c.update({"window": 0, "tree": False, "decay": 1.0} if op == "weights" else {"budget": 4096, "first": 4, "recent": 64})
    c.update(kw)
    return c


def listed():
    return [
        # The decode step of 64 served sequences: their q and k from the projection's float32 rows, far positions.
        _rope("rope_decode", tokens=64, far=1 << 20),
        # A 2048-token chunk of a prompt with video in it: time, height and width in sections of the head.
        _rope("rope_video", tokens=2048, q_heads=40, axes=3, far=32768),
        # The patches of a large image in its encoder: 16 heads of 72, height and width by turns, bfloat16.
        _rope("rope_patches", tokens=16383, q_heads=16, heads=16, dim=72, rotary=72, axes=2, mixed=True, f32=False,
              far=128),
        # One decoded token's answer: its log probability, the entropy, 20 alternatives.
        _logprobs("logprobs_step"),
        # 64 sampled sequences under a grammar's mask, bfloat16 logits of an odd vocabulary, a temperature.
        _logprobs("logprobs_masked", rows=64, vocab=32003, given=3, top=5, f32=False, scale=1.25, masked=True),
        # A 512-token prompt scored over the whole vocabulary.
        _logprobs("logprobs_prompt", rows=512),
        # A decode step's weights at the long end of a context.
        _cached("weights_decode", "weights", q_heads=40, past_min=131007, past_max=131007),
        # A decode step of 64 sequences of very different lengths, 4-bit keys, small pages, older weight fading.
        _cached("weights_batch", "weights", k_bits=4, page=16, seqs=64, past_min=1, past_max=8191, lengths=7, decay=0.9),
        # The last chunk of a prompt, by whose weights the prompt is cut down.
        _cached("weights_chunk", "weights", q_heads=40, new_min=2048, new_max=2048, past_min=30720, past_max=30720,
                decay=0.0),
        # A sequence at its budget loses a block's worth of tokens.
        _cached("evict_block", "evict", past_min=4607, past_max=4607),
        # A prompt cut down to an eighth after its prefill.
        _cached("evict_prompt", "evict", past_min=32768, past_max=32768, recent=256),
        # 64 sequences, those past the budget cut to it; 4-bit keys, 8-bit values.
        _cached("evict_batch", "evict", k_bits=4, page=16, seqs=64, past_min=1, past_max=8191, lengths=7, budget=2048),
    ]


def _between(rng, lo, hi):
    """A whole number of lo..hi, even over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))) - 0.5))))


def draw(rng):
    c = _draw(rng, rng.choice(["rope", "rope", "logprobs", "logprobs", "weights", "weights", "weights", "evict", "evict"]))
    del c["name"]
    return c


def _draw(rng, op):
    q_heads, heads = rng.choice([(32, 8), (40, 8), (8, 8), (16, 1), (28, 4), (64, 8), (12, 2)])
    if op == "rope":
        dim = rng.choice([64, 72, 80, 128, 128, 256])
        rotary = dim if rng.random() < 0.7 else max(8, dim // rng.choice([2, 4]) // 8 * 8)
        tokens = _between(rng, 1, 65536 * 1152 // ((q_heads + heads) * dim))
        return _rope("", tokens=tokens, q_heads=q_heads, heads=heads, dim=dim, rotary=rotary, axes=rng.choice([1, 2, 3]),
                     mixed=rng.random() < 0.5, adjacent=rng.random() < 0.4, f32=rng.random() < 0.5,
                     factor=rng.choice([1.0, 1.0, 1.1386]), far=_between(rng, 16, 1 << 20))
    if op == "logprobs":
        vocab = _between(rng, 1000, 262144)
        return _logprobs("", rows=_between(rng, 1, 512 * 151936 // vocab if vocab > 75000 else 1024), vocab=vocab,
                         given=rng.randint(1, 8), top=rng.choice([0, 1, 5, 20, rng.randint(2, 64)]),
                         f32=rng.random() < 0.6, scale=rng.choice([1.0, 1.0, 0.7, 1.4286]), masked=rng.random() < 0.4)
    c = _cached("", op, q_heads=q_heads, heads=heads, dim=rng.choice([64, 128, 128, 256]), k_bits=rng.choice([4, 8]),
                v_bits=rng.choice([4, 8]), page=rng.choice([16, 32, 64, 128, 256]), lengths=rng.randrange(1 << 30))
    if op == "evict":
        c["seqs"] = _between(rng, 1, 64)
        c["past_max"] = _between(rng, 16, 65536 // c["seqs"])
        c["past_min"] = rng.choice([1, c["past_max"] // 2 + 1, c["past_max"]])
        c["budget"] = max(2, int(c["past_max"] * rng.uniform(0.1, 0.95)))
        c["first"] = rng.randint(0, min(4, c["budget"] // 2))
        c["recent"] = min(c["budget"] - c["first"], _between(rng, 1, 256))
        return c
    kind = rng.choice(["decode", "verify", "chunk", "chunk", "mixed"])
    top = {"decode": 1, "verify": _between(rng, 2, 40), "chunk": _between(rng, 65, 2048), "mixed": _between(rng, 16, 700)}[kind]
    c["new_max"], c["new_min"] = top, 1 if kind == "mixed" else max(1, int(top * rng.uniform(0.6, 1.0)))
    c["seqs"] = _between(rng, 1, 64 if kind == "decode" else 16 if kind == "verify" else 6)
    c["past_max"] = _between(rng, 1, 131007 if kind == "decode" and c["seqs"] < 4 else 30720)
    c["past_min"] = rng.choice([0, c["past_max"] // 2, c["past_max"]])
    c["tree"] = kind == "verify" and rng.random() < 0.5
    c["window"] = _between(rng, 100, 4096) if not c["tree"] and rng.random() < 0.3 else 0
    c["decay"] = rng.choice([0.0, 1.0, 0.9])
    most = next(w for w in listed() if w["name"] == "weights_chunk")
    scores = lambda w: w["seqs"] * w["q_heads"] * w["new_max"] * (w["new_max"] + w["past_max"])
    held = lambda w: w["seqs"] * w["heads"] * w["dim"] * (w["new_max"] + w["past_max"])
    while (scores(c) > 0.9 * scores(most) or work(c)["flops"] > 0.9 * work(most)["flops"]
           or held(c) > 4 * 8 * 128 * 131072):
        c["past_max"] = c["past_max"] * 2 // 3
        c["past_min"] = min(c["past_min"], c["past_max"])
    return c


def _lengths(case):
    """(new tokens, tokens before them) of each sequence, from the case alone."""
    r = random.Random(case["lengths"])
    return [(r.randint(case["new_min"], case["new_max"]), r.randint(case["past_min"], case["past_max"]))
            for _ in range(case["seqs"])]


def _tree(case, n):
    """The ancestors (and itself) of each of n drafted tokens, as bits: token 0 is the root, each other token
    hangs on an earlier one."""
    r = random.Random(case["lengths"] + n)
    masks = []
    for i in range(n):
        masks.append((masks[r.randrange(i)] if i else 0) | 1 << i)
    return masks


def work(case):
    if case["op"] == "rope":
        values = case["tokens"] * case["dim"]
        size = 4 if case["f32"] else 2
        return {"bytes": values * (case["q_heads"] * (size + 2) + case["heads"] * 2 * size) + 4 * case["tokens"] * case["axes"],
                "flops": 3 * case["tokens"] * case["rotary"] * (case["q_heads"] + case["heads"])}
    if case["op"] == "logprobs":
        n = case["rows"]
        return {"bytes": n * case["vocab"] * (4 if case["f32"] else 2) + n * (8 * case["given"] + 8 * case["top"] + 8),
                "flops": 5 * n * case["vocab"]}
    k_row, v_row = [case["dim"] * case[b] // 8 + case["dim"] // 32 for b in ("k_bits", "v_bits")]
    if case["op"] == "evict":
        total = 0
        for _, past in _lengths(case):
            if past > case["budget"]:      # weights read and written, the kept tokens behind the first ones moved
                moved = case["budget"] - case["first"]
                total += case["heads"] * (4 * past + 8 * case["budget"] + 2 * moved * (k_row + v_row))
            else:
                total += case["heads"] * (8 * past + 4 * case["budget"])
        return {"bytes": total, "flops": 0}
    keys = held = pairs = rows = 0
    for n, past in _lengths(case):
        first = max(0, past + 1 - case["window"]) if case["window"] else 0
        keys += past + n - first
        held += past + n
        rows += n * case["q_heads"]
        if case["window"]:
            pairs += sum(min(case["window"], past + i + 1) for i in range(n))
        elif case["tree"]:
            pairs += n * past + sum(bin(m).count("1") for m in _tree(case, n))
        else:
            pairs += n * past + n * (n + 1) // 2
    return {"bytes": case["heads"] * (keys * k_row + held * (8 if case["decay"] else 4)) + rows * (2 * case["dim"] + 4),
            "flops": 2 * case["dim"] * case["q_heads"] * pairs}


# ------------------------------------------------------- the inputs of a pass

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def prepare(case, seed):
    g = _gen(seed)
    state = {"case": dict(case)}
    if case["op"] == "rope":
        _prepare_rope(case, state, g)
    elif case["op"] == "logprobs":
        _prepare_logprobs(case, state, g)
    else:
        _prepare_cached(case, state, g)
    return state


def _prepare_rope(case, state, g):
    tokens, dim, q_heads, heads, axes = (case[n] for n in ("tokens", "dim", "q_heads", "heads", "axes"))
    dtype = torch.float32 if case["f32"] else torch.bfloat16
    # q and k are column ranges of one projection's rows
    qkv = torch.randn(tokens, (q_heads + 2 * heads) * dim, generator=g, device=DEV).to(dtype)
    state["q"] = qkv[:, :q_heads * dim].view(tokens, q_heads, dim)
    state["k"] = qkv[:, q_heads * dim:(q_heads + heads) * dim].view(tokens, heads, dim)
    state["q_out"] = torch.empty(tokens, q_heads, dim, dtype=torch.bfloat16, device=DEV)
    state["k_out"] = torch.empty(tokens, heads, dim, dtype=dtype, device=DEV)
    state["positions"] = torch.randint(0, case["far"], (axes, tokens), generator=g, device=DEV, dtype=torch.int32)
    pairs = case["rotary"] // 2
    i = torch.arange(pairs, device=DEV, dtype=torch.float64)
    state["freqs"] = torch.pow(10000.0 if case["axes"] > 1 else 500000.0, -i / pairs)
    i = torch.arange(pairs, device=DEV)
    state["axis"] = (i % axes if case["mixed"] else i * axes // pairs).to(torch.uint8)


def _prepare_logprobs(case, state, g):
    n, vocab = case["rows"], case["vocab"]
    x = torch.randn(n, vocab, generator=g, device=DEV).mul_(2.0)
    # the few likely tokens of a row, from nearly certain to undecided
    likely = torch.randint(0, vocab, (n, 8), generator=g, device=DEV)
    x.scatter_add_(1, likely, 4 + 10 * torch.rand(n, 8, generator=g, device=DEV))
    if case["masked"]:
        x.masked_fill_(torch.rand(n, vocab, generator=g, device=DEV) < 0.6, -math.inf)
    state["logits"] = x if case["f32"] else x.to(torch.bfloat16)
    tokens = torch.randint(0, vocab, (n, case["given"]), generator=g, device=DEV, dtype=torch.int32)
    tokens[:, 0] = likely[:, 0]
    state["tokens"] = tokens
    state["logp"] = torch.empty(n, case["given"], device=DEV)
    state["lse"], state["entropy"] = torch.empty(n, device=DEV), torch.empty(n, device=DEV)
    state["top_logp"] = torch.empty(n, case["top"], device=DEV)
    state["top_index"] = torch.empty(n, case["top"], dtype=torch.int32, device=DEV)


def _prepare_cached(case, state, g):
    lengths = _lengths(case)
    if case["op"] == "evict":
        lengths = [(0, p) for _, p in lengths]
    seqs, heads, dim, page = case["seqs"], case["heads"], case["dim"], case["page"]
    tokens = sum(n for n, _ in lengths)
    context = max(n + p for n, p in lengths)
    width = -(-context // page)
    pages = sum(-(-(n + p) // page) for n, p in lengths) + 3
    # the pages of a pool in use lie in any order
    order = torch.randperm(pages, generator=g, device=DEV).tolist()
    table = torch.full((seqs, width), -1, dtype=torch.int32)
    for s, (n, p) in enumerate(lengths):
        for k in range(-(-(n + p) // page)):
            table[s, k] = order.pop()
    offsets = [0]
    for n, _ in lengths:
        offsets.append(offsets[-1] + n)
    state.update({
        "tokens": tokens, "context": context, "max_new": max(n for n, _ in lengths),
        "table": table.to(DEV), "offsets": torch.tensor(offsets, dtype=torch.int32, device=DEV),
        "past": torch.tensor([p for _, p in lengths], dtype=torch.int32, device=DEV),
    })
    for side in ("k", "v"):
        if side == "v" and case["op"] == "weights":      # the values are not read; they are there
            n = pages * heads * page * dim
            state["v_codes"] = torch.zeros(n * case["v_bits"] // 8, dtype=torch.uint8, device=DEV)
            state["v_scales"] = torch.zeros(n // 32, dtype=torch.uint8, device=DEV)
            continue
        x = torch.randn(pages, heads, page, dim, generator=g, device=DEV)
        if side == "k":      # a few large channels, as keys have them
            x.mul_(1 + 3 * (torch.rand(heads, 1, dim, generator=g, device=DEV) < 0.03))
        state[side + "_codes"], state[side + "_scales"] = _pack(side, case, *_quantize(x, case[side + "_bits"]))
        del x
    span = width * page
    # what the steps before have gathered: most keys a little, a few much
    held = torch.rand(seqs, heads, span, generator=g, device=DEV).pow_(8).mul_(16)
    past = state["past"][:, None, None]
    held.masked_fill_(torch.arange(span, device=DEV) >= past, 0.0)
    state["weights"] = held
    if case["op"] == "evict":
        state["weights_out"] = torch.zeros_like(held)
        state["left"] = torch.zeros(seqs, dtype=torch.int32, device=DEV)
        state["kept"] = torch.zeros(seqs, heads, case["budget"], dtype=torch.int32, device=DEV)
        return
    state["q"] = (1.5 * torch.randn(tokens, case["q_heads"], dim, generator=g, device=DEV)).to(torch.bfloat16)
    state["scale"] = 1.0 / math.sqrt(dim)
    if case["tree"]:
        masks = [m for n, _ in lengths for m in _tree(case, n)]
        state["tree"] = torch.tensor([m - (1 << 64) if m >> 63 else m for m in masks], dtype=torch.int64, device=DEV)
    # the attention's log-sum-exp, which the step has already
    lse = torch.empty(tokens, case["q_heads"], device=DEV)
    group = case["q_heads"] // heads
    at = 0
    for s, (n, p) in enumerate(lengths):
        hidden = _hidden(case, n, p)
        used = table[s, :-(-(n + p) // page)].to(DEV).long()
        data = state["k_codes"].view(-1, heads, page * dim * case["k_bits"] // 8)[used]
        k = _unpack("k", case, data, state["k_scales"].view(-1, heads, page * dim // 32)[used])
        k = k.permute(1, 0, 2, 3).reshape(heads, -1, dim)[:, :n + p]
        for h in range(heads):
            q = state["q"][at:at + n, h * group:(h + 1) * group].float()
            z = torch.matmul(q.reshape(n * group, dim), k[h].t().contiguous()).mul_(state["scale"]).view(n, group, n + p)
            z.masked_fill_(hidden[:, None, :], -math.inf)
            lse[at:at + n, h * group:(h + 1) * group] = torch.logsumexp(z, -1)
            del z
        at += n
    state["lse"] = lse


def _hidden(case, n, past):
    """[new tokens][keys]: the keys that a token does not see."""
    key = torch.arange(past + n, device=DEV)[None, :]
    pos = torch.arange(past, past + n, device=DEV)[:, None]
    if case["tree"]:
        bits = torch.tensor([[m >> b & 1 for b in range(n)] for m in _tree(case, n)], device=DEV)
        return torch.cat((torch.zeros(n, past, dtype=torch.bool, device=DEV), bits == 0), 1)
    hidden = key > pos
    return hidden | (pos - key >= case["window"]) if case["window"] else hidden


# ---------------------------------------------------------- one pass, measured

def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(state):
    import block_scaled_bit_nvfp4_amd as nv
    case = state["case"]
    op = case["op"]
    if op == "rope":
        nv.nvfp4_rope([(state["q"], state["q_out"]), (state["k"], state["k_out"])], state["positions"], state["freqs"],
                      axis=state["axis"], adjacent=case["adjacent"], factor=case["factor"])
        return {"q": state["q_out"], "k": state["k_out"]}
    if op == "logprobs":
        if "workspace" not in state:     # what a program makes once and keeps
            need = nv.nvfp4_logprobs_workspace_bytes(case["rows"], case["vocab"], case["top"])
            state["workspace"] = torch.empty(max(1, need), dtype=torch.uint8, device=DEV)
        top = case["top"] > 0
        nv.nvfp4_logprobs(state["logits"], tokens=state["tokens"], logp=state["logp"], lse=state["lse"],
                          entropy=state["entropy"], top_logp=state["top_logp"] if top else None,
                          top_index=state["top_index"] if top else None, scale=case["scale"],
                          workspace=state["workspace"])
        return {n: state[n] for n in ("logp", "lse", "entropy", "top_logp", "top_index")}
    if "cache" not in state:
        form = {8: nv.NVFP4_KV_MXFP8, 4: nv.NVFP4_KV_MXFP4}
        state["cache"] = nv.KvCache(state["k_codes"], state["k_scales"], state["v_codes"], state["v_scales"],
                                    form[case["k_bits"]], form[case["v_bits"]], case["page"], case["heads"],
                                    case["dim"])
        state["batch"] = nv.KvBatch(state["table"], state["offsets"], state["past"], state["tokens"],
                                    state["max_new"], state["context"])
    if op == "weights":
        nv.nvfp4_kv_weights(state["cache"], state["batch"], state["q"], state["scale"], state["lse"], state["weights"],
                            decay=case["decay"], window=case["window"], tree=state.get("tree"))
        return {"weights": state["weights"]}
    nv.nvfp4_kv_evict(state["cache"], state["batch"], state["weights"], case["budget"], state["kept"],
                      state["left"], weights_out=state["weights_out"], first=case["first"], recent=case["recent"])
    return _evicted(state)


def _evicted(state):
    # eviction moves the planes' bytes and computes none of them: they come back as they stand
    return {n: state[n] for n in ("kept", "left", "weights_out", "k_codes", "k_scales", "v_codes", "v_scales")}


def _run_plain(state):
    op = state["case"]["op"]
    if op == "rope":
        return _rope_plain(state)
    if op == "logprobs":
        return _logprobs_plain(state)
    return _weights_plain(state) if op == "weights" else _evict_plain(state)


# ------------------------------------------------------------- the plain forms

def _rope_plain(state):
    case = state["case"]
    # far positions times small frequencies: the angles need 64 bits
    angle = state["positions"][state["axis"].long()].double() * state["freqs"][:, None]      # [pairs][tokens]
    cos = (angle.cos() * case["factor"]).float().t()[:, None, :]
    sin = (angle.sin() * case["factor"]).float().t()[:, None, :]
    return {name: _turn(case, state[name].float(), cos, sin).to(state[name + "_out"].dtype) for name in ("q", "k")}


def _turn(case, x, cos, sin):
    part, rest = x[..., :case["rotary"]], x[..., case["rotary"]:]
    if case["adjacent"]:
        a, b = part[..., 0::2], part[..., 1::2]
        part = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = part.chunk(2, -1)
        part = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((part, rest), -1)


def _logprobs_plain(state):
    case = state["case"]
    x = state["logits"].float()
    z = x * case["scale"]
    top = z.amax(-1, keepdim=True)
    e = (z - top.clamp(min=torch.finfo(torch.float32).min)).exp()
    total = e.sum(-1, keepdim=True)
    lse = top + total.log()
    nats = torch.where(e > 0, e * (z - top), 0.0).sum(-1)
    entropy = total.squeeze(-1).log() - nats / total.squeeze(-1)
    order = torch.sort(x, dim=-1, descending=True, stable=True)
    k = case["top"]
    return {"logp": z.gather(1, state["tokens"].long()) - lse, "lse": lse.squeeze(-1), "entropy": entropy,
            "top_logp": order.values[:, :k] * case["scale"] - lse, "top_index": order.indices[:, :k].to(torch.int32)}


def _weights_plain(state):
    case = state["case"]
    heads, dim, page, seqs = case["heads"], case["dim"], case["page"], case["seqs"]
    group = case["q_heads"] // heads
    n_max, table = state["max_new"], state["table"]
    span = table.shape[1] * page
    at = table.clamp(min=0).long()
    data = state["k_codes"].view(-1, heads, page * dim * case["k_bits"] // 8)[at]
    k = _unpack("k", case, data, state["k_scales"].view(-1, heads, page * dim // 32)[at])   # [seqs][width][heads][page][dim]
    k = k.permute(0, 2, 1, 3, 4).reshape(seqs, heads, span, dim)
    offsets, past = state["offsets"].long(), state["past"].long()
    i = torch.arange(n_max, device=DEV)
    n = offsets[1:] - offsets[:-1]
    token = (offsets[:-1, None] + i).clamp(max=state["tokens"] - 1)      # [seqs][n_max]
    q = state["q"][token].float().view(seqs, n_max, heads, group, dim)
    q = q.permute(0, 2, 1, 3, 4).reshape(seqs, heads, n_max * group, dim)
    lse = state["lse"][token].view(seqs, n_max, heads, group).permute(0, 2, 1, 3)
    s = torch.matmul(q, k.transpose(-1, -2).contiguous()).mul_(state["scale"]).view(seqs, heads, n_max, group, span)
    s = s.sub_(lse[..., None]).exp_()
    j = torch.arange(span, device=DEV)
    pos = past[:, None] + i
    seen = (j <= pos[..., None]) & (i < n[:, None])[..., None]           # [seqs][n_max][span]
    if case["tree"]:
        bit = (j - past[:, None]).clamp(0, 63)
        mine = state["tree"][token][..., None] >> bit[:, None, :] & 1
        new = (j >= past[:, None])[:, None, :]
        drafted = (mine == 1) & (j - past[:, None] < n[:, None])[:, None, :] & (i < n[:, None])[..., None]
        seen = torch.where(new, drafted, seen)
    if case["window"]:
        seen = seen & (j > pos[..., None] - case["window"])
    s.masked_fill_(~seen[:, None, :, None, :], 0.0)
    gathered = s.sum((2, 3))
    w = state["weights"]
    old = torch.where(j < past[:, None, None], w * case["decay"], 0.0) if case["decay"] else torch.zeros_like(w)
    w.copy_(torch.where(j < (past + n)[:, None, None], old + gathered, w))
    return {"weights": w}


def _evict_plain(state):
    case = state["case"]
    heads, page, seqs, budget = case["heads"], case["page"], case["seqs"], case["budget"]
    w, past = state["weights"], state["past"].long()
    span = w.shape[-1]
    j = torch.arange(span, device=DEV)
    length = past[:, None, None]
    rank = torch.where((j < case["first"]) | (j >= length - case["recent"]), math.inf, w)
    rank = torch.where(j < length, rank, -math.inf)
    kept = torch.sort(rank, dim=-1, descending=True, stable=True).indices[..., :min(budget, span)].sort(-1).values
    slot = torch.arange(budget, device=DEV)
    full = torch.zeros(seqs, heads, budget, dtype=torch.int64, device=DEV)
    full[..., :kept.shape[-1]] = kept
    over = length > budget
    kept = torch.where(over, full, torch.where(slot < length, slot, -1).expand(seqs, heads, budget))
    out = state["weights_out"]
    taken = w.gather(-1, kept.clamp(min=0)) if budget <= span else w.gather(-1, kept[..., :span].clamp(min=0))
    wide = out.clone()
    wide[..., :taken.shape[-1]] = torch.where(kept[..., :taken.shape[-1]] >= 0, taken, wide[..., :taken.shape[-1]])
    out.copy_(wide)
    state["kept"].copy_(kept)
    state["left"].copy_(torch.where(past > budget, budget, past))
    # the bytes of the sequences that are cut, from their old places to the first ones
    rows = (past > budget).nonzero().squeeze(-1)
    table = state["table"].long()
    src = kept[rows].transpose(1, 2)                                     # [cut][budget][heads]
    from_slot = table[rows[:, None, None], src // page] * page + src % page
    to_slot = (table[rows][:, slot // page] * page + slot % page if rows.numel() else src[..., 0])
    to_slot = to_slot[..., None].expand(from_slot.shape)
    for side in ("k", "v"):
        codes, scales = state[side + "_codes"], state[side + "_scales"]
        a, b = _places(side, case, from_slot.reshape(-1, heads)), _places(side, case, to_slot.reshape(-1, heads))
        moved = codes[a[0]], scales[a[1]]
        codes.index_put_((b[0],), moved[0])
        scales.index_put_((b[1],), moved[1])
    return _evicted(state)


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
    data = codes if bits == 8 else codes[..., 0::2] | codes[..., 1::2] << 4
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
    codes = data if bits == 8 else torch.stack((data & 15, data >> 4), -1).flatten(-2)
    return _values(codes, scales.reshape(*lead, page, dim // 32), bits)


def _places(side, case, slot):
    """For tokens whose heads' vectors lie at `slot` [tokens][heads] (page * tokens of a page + place): the plane
    indexes [tokens][heads][bytes] of their code bytes and of their scale bytes."""
    bits, dim, page, heads = case[side + "_bits"], case["dim"], case["page"], case["heads"]
    row, blocks = dim * bits // 8, dim // 32
    shape, order = _unit_shape(side, dim, bits)
    unit = (slot // page * heads + torch.arange(heads, device=DEV)) * (page // 16) + slot % page // 16
    inner = torch.arange(16 * row, device=DEV).reshape(shape).permute(order).reshape(16, row)
    if side == "k":
        scale = torch.arange(16 * blocks, device=DEV).reshape(16, blocks)
    else:
        scale = torch.arange(16 * blocks, device=DEV).reshape(4, blocks, 4).transpose(1, 2).reshape(16, blocks)
    r = slot % 16
    return (unit * 16 * row)[..., None] + inner[r], (unit * 16 * blocks)[..., None] + scale[r]


# ------------------------------------------------------------------ in 64 bits

def exact(case, seed):
    state = prepare(case, seed)
    return {"rope": _rope_exact, "logprobs": _logprobs_exact, "weights": _weights_exact, "evict": _evict_exact}[case["op"]](case, state)


def _rope_exact(case, state):
    """The rotations as products of complex numbers."""
    got = {}
    pairs = case["rotary"] // 2
    turn = torch.stack([state["positions"][int(a)].double() * f for a, f in zip(state["axis"].tolist(), state["freqs"])], 1)
    turn = torch.polar(torch.full_like(turn, case["factor"]), turn)[:, None, :]
    for name in ("q", "k"):
        x = state[name].double().clone()
        even = torch.arange(pairs, device=DEV) * 2 if case["adjacent"] else torch.arange(pairs, device=DEV)
        odd = even + (1 if case["adjacent"] else pairs)
        z = torch.complex(x[..., even], x[..., odd]) * turn
        x[..., even], x[..., odd] = z.real, z.imag
        got[name] = x
    return got


def _logprobs_exact(case, state):
    z = state["logits"].double() * case["scale"]
    logp = torch.log_softmax(z, -1)
    p = logp.exp()
    return {"logp": logp.gather(1, state["tokens"].long()), "lse": torch.logsumexp(z, -1),
            "entropy": -(p * logp.clamp(min=-1e300)).sum(-1), "top_logp": torch.topk(logp, case["top"], -1).values,
            "top_index": None}


def _keys(case, state, s, total):
    """The keys of sequence s that the cache holds, float64 [heads][tokens][dim], code by code from the place of each
    byte."""
    bits, dim, page, heads = case["k_bits"], case["dim"], case["page"], case["heads"]
    used = state["table"][s, :-(-total // page)].long()
    row, blocks = dim * bits // 8, dim // 32
    r, d = torch.arange(16, device=DEV)[:, None], torch.arange(dim, device=DEV)[None, :]
    piece = min(16, row // 4)
    byte = d * bits // 8
    at = (byte // piece) * 16 * piece + r * piece + byte % piece
    data = state["k_codes"].view(-1, heads, page // 16, 16 * row)[used][..., at]
    power = state["k_scales"].view(-1, heads, page // 16, 16 * blocks)[used][..., r * blocks + d // 32]
    if bits == 4:
        data = torch.where(d % 2 == 0, data % 16, data // 16)
        grid = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=DEV)
    else:
        small = [m * 2.0 ** -9 for m in range(8)]
        grid = torch.tensor((small + [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8)])[:127],
                            dtype=torch.float64, device=DEV)
    half = 1 << (bits - 1)
    x = grid[(data % half).long()] * torch.where(data >= half, -1.0, 1.0).double()
    x = x * torch.pow(2.0, power.double() - 127)               # [pages][heads][units][16][dim]
    return x.permute(1, 0, 2, 3, 4).reshape(heads, -1, dim)[:, :total]


def _weights_exact(case, state):
    group = case["q_heads"] // case["heads"]
    got = state["weights"].double()
    at = 0
    for s, (n, past) in enumerate(_lengths(case)):
        k, hidden = _keys(case, state, s, n + past), _hidden(case, n, past)
        fresh = torch.zeros(case["heads"], n + past, dtype=torch.float64, device=DEV)
        for h in range(case["q_heads"]):
            z = state["q"][at:at + n, h].double() @ k[h // group].T * state["scale"]
            p = torch.exp(z - state["lse"][at:at + n, h, None].double()).masked_fill_(hidden, 0.0)
            fresh[h // group] += p.sum(0)
        fresh[:, :past] += got[s, :, :past] * case["decay"]
        got[s, :, :n + past] = fresh
        at += n
    return {"weights": got}


def _evict_exact(case, state):
    """The weights of the kept tokens; the bytes and the positions are whole numbers."""
    w = state["weights"].double().cpu()
    out = state["weights_out"].double().cpu()
    for s, (_, past) in enumerate(_lengths(case)):
        lo, hi = case["first"], past - case["recent"]
        take = case["budget"] - case["first"] - case["recent"]
        for h in range(case["heads"]):
            row = w[s, h, :past]
            if past > case["budget"]:
                inner = row[lo:hi].tolist()
                best = sorted(sorted(range(len(inner)), key=lambda i: (-inner[i], i))[:take])
                row = torch.cat((row[:lo], row[lo:hi][best], row[hi:]))
            out[s, h, :row.numel()] = row
    return {"kept": None, "left": None, "weights_out": out.to(DEV), "k_codes": None, "k_scales": None, "v_codes": None,
            "v_scales": None}
