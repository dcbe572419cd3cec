"""A decoder's rotary positions and its key-value cache in 8 bits, as a serving
program calls them, in two forms: elementary torch operations in float32
(`own` false) and the library's kernels (`own` true).

Four operators, in the order of a decoding step: queries and keys are turned
by their positions ("rope"), the new keys and values are written to a cache of
8-bit codes and read back as what they now stand for ("store"), requests' rows
are read back from it ("read"), and the new tokens attend to it ("attn"): one
token a request, or several after a cached prefix, each of which sees the
prefix and the new tokens up to itself.

Head counts are those of the decoders that the workloads name (16 query heads
over 8 key-value heads of 128; 12 heads of 64), with other groupings among the
drawn cases. Lengths differ between the requests of a batch: `_spread` fixes
the set of lengths by the case, the seed only their order.
"""

import math

import torch

own = False

DEVICE = "cuda"
_TYPES = {"f16": torch.float16, "f32": torch.float32}
_BYTES = {"f16": 2, "f32": 4}


def listed():
    return [
        # one decoding step of a few requests: latency
        {"name": "rope-step-8-f16", "op": "rope", "tokens": 8, "heads": 16, "kv_heads": 8, "dim": 128, "rot": 128,
         "interleaved": False, "base": 1e6, "factor": 1.0, "far": 16384, "dtype": "f16"},
        # prompts in float32, neighbours paired, half of each head turned, positions squeezed for a longer context
        {"name": "rope-prompts-9999-f32", "op": "rope", "tokens": 9999, "heads": 16, "kv_heads": 8, "dim": 128,
         "rot": 64, "interleaved": True, "base": 1e4, "factor": 4.0, "far": 131072, "dtype": "f32"},
        # one decoding step's keys and values of one layer
        {"name": "store-step-8-f16", "op": "store", "tokens": 8, "kv_heads": 8, "dim": 128, "page": 16,
         "dtype": "f16"},
        # 64 prompts of 410 rows
        {"name": "store-prompts-26240-f16", "op": "store", "tokens": 26240, "kv_heads": 8, "dim": 128, "page": 32,
         "dtype": "f16"},
        # one request leaves for another cache
        {"name": "read-1x452-f32", "op": "read", "batch": 1, "len_lo": 452, "len_hi": 452, "spare": 3, "kv_heads": 12,
         "dim": 64, "page": 16, "dtype": "f32"},
        # a server's requests, as rows for calls that take no pages
        {"name": "read-32-ragged-f16", "op": "read", "batch": 32, "len_lo": 62, "len_hi": 2001, "spare": 0,
         "kv_heads": 8, "dim": 128, "page": 16, "dtype": "f16"},
        # one request soon after its 30 s prompt: latency counts
        {"name": "attn-1x452-f16", "op": "attn", "batch": 1, "len_lo": 452, "len_hi": 452, "new_lo": 0, "new_hi": 0,
         "heads": 16, "kv_heads": 8, "dim": 128, "page": 16, "dtype": "f16"},
        # a server's ordinary step: 3.2 s commands and two-minute clips side by side
        {"name": "attn-32-ragged-f16", "op": "attn", "batch": 32, "len_lo": 62, "len_hi": 2001, "new_lo": 0,
         "new_hi": 0, "heads": 16, "kv_heads": 8, "dim": 128, "page": 16, "dtype": "f16"},
        # long contexts, the cache streamed from memory
        {"name": "attn-32-long-f16", "op": "attn", "batch": 32, "len_lo": 500, "len_hi": 16384, "new_lo": 0,
         "new_hi": 0, "heads": 16, "kv_heads": 8, "dim": 128, "page": 64, "dtype": "f16"},
        # float32 graphs, every head with keys of its own
        {"name": "attn-16-f32", "op": "attn", "batch": 16, "len_lo": 5, "len_hi": 1503, "new_lo": 0, "new_hi": 0,
         "heads": 12, "kv_heads": 12, "dim": 64, "page": 32, "dtype": "f32"},
        # chunks of 62 rows after cached prefixes of all lengths
        {"name": "attn-8-chunks-62-f16", "op": "attn", "batch": 8, "len_lo": 0, "len_hi": 2001, "new_lo": 62,
         "new_hi": 62, "heads": 16, "kv_heads": 8, "dim": 128, "page": 16, "dtype": "f16"},
        # prompts of 3.2 s to 30 s of audio entering together
        {"name": "attn-16-prompts-410-f16", "op": "attn", "batch": 16, "len_lo": 0, "len_hi": 0, "new_lo": 62,
         "new_hi": 410, "heads": 16, "kv_heads": 8, "dim": 128, "page": 16, "dtype": "f16"},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("rope", "store", "read", "attn", "attn", "attn"))
    heads, kv_heads = rng.choice(((16, 8), (12, 12), (32, 8), (8, 1), (16, 2)))
    dim = rng.choice((64, 128))
    dtype = rng.choice(("f16", "f16", "f32"))
    page = rng.choice((16, 32, 48, 64, 128))
    if op == "rope":
        most = 9999 * 24 * 128 * 4 // ((heads + kv_heads) * dim * _BYTES[dtype])
        return {"op": op, "tokens": _log_int(rng, 1, most), "heads": heads, "kv_heads": kv_heads, "dim": dim,
                "rot": rng.choice((dim, dim, dim // 2, dim // 4, 20)), "interleaved": rng.random() < 0.5,
                "base": rng.choice((1e4, 1e6)), "factor": rng.choice((1.0, 1.0, 2.5, 8.0)),
                "far": _log_int(rng, 1, 1 << 20), "dtype": dtype}
    if op == "store":
        most = 26240 * 8 * 128 * 2 // (kv_heads * dim * _BYTES[dtype])
        return {"op": op, "tokens": _log_int(rng, 1, min(26240, most)), "kv_heads": kv_heads, "dim": dim,
                "page": page, "dtype": dtype}
    if op == "read":
        len_hi = _log_int(rng, 1, 4000)
        most = max(1, 32 * 1032 * 8 * 128 * 2 // (kv_heads * dim * _BYTES[dtype] * len_hi))
        return {"op": op, "batch": _log_int(rng, 1, min(64, most)), "len_lo": rng.randint(0, len_hi), "len_hi": len_hi,
                "spare": rng.choice((0, 5)), "kv_heads": kv_heads, "dim": dim, "page": page, "dtype": dtype}
    if rng.random() < 0.5:
        len_hi, new_hi = _log_int(rng, 1, 16384), 0
        most = int(0.45e9) // (kv_heads * dim * len_hi)
    else:
        len_hi, new_hi = _log_int(rng, 1, 4096), _log_int(rng, 2, 410)
        most = min(int(16e9 if dtype == "f16" else 2e9) // (4 * new_hi * (len_hi + new_hi) * heads * dim),
                   int(0.45e9) // (kv_heads * dim * (len_hi + new_hi)))
    return {"op": op, "batch": _log_int(rng, 1, max(1, min(64, most))), "len_lo": rng.randint(0, len_hi),
            "len_hi": len_hi, "new_lo": rng.randint(0, new_hi), "new_hi": new_hi, "heads": heads,
            "kv_heads": kv_heads, "dim": dim, "page": page, "dtype": dtype}


def _spread(lo, hi, count):
    """`count` whole numbers from lo to hi, evenly spread, hi among them."""
    return [hi - (hi - lo) * i // max(1, count - 1) for i in range(count)]


def _lengths(lo, hi, count, order):
    return torch.tensor(_spread(lo, hi, count), dtype=torch.int32)[torch.randperm(count, generator=order)].to(DEVICE)


def _quantise(x):
    """Codes and scales of rows x [..., D], one scale a row; the quotients in
    64 bits, where codes next to a border are the right ones."""
    x = x.double()
    scale = (x.abs().amax(-1) / 127).float()
    codes = torch.round(x / scale.double()[..., None]).nan_to_num(0.0).clamp(-127, 127)
    return codes.to(torch.int8), scale


def prepare(case, seed):
    order = torch.Generator().manual_seed(seed)
    noise = torch.Generator(DEVICE).manual_seed(seed)
    return _PREPARE[case["op"]](case, order, noise)


def _prepare_rope(case, order, noise):
    # queries and keys as columns of the fused product's rows
    tokens, heads, kv_heads, dim = case["tokens"], case["heads"], case["kv_heads"], case["dim"]
    dtype = _TYPES[case["dtype"]]
    rows = torch.randn((tokens, (heads + 2 * kv_heads) * dim), dtype=dtype, device=DEVICE, generator=noise)
    rot = case["rot"]
    at = torch.arange(rot // 2, dtype=torch.float64, device=DEVICE)
    return {"op": "rope", "q": rows[:, :heads * dim].view(tokens, heads, dim),
            "k": rows[:, heads * dim:(heads + kv_heads) * dim].view(tokens, kv_heads, dim),
            "positions": torch.randint(0, case["far"], (tokens,), generator=order).to(torch.int32).to(DEVICE),
            "freqs": case["base"] ** (-2 * at / rot) / case["factor"], "interleaved": case["interleaved"],
            "gain": 0.1 * math.log(case["factor"]) + 1.0,
            "q_out": torch.empty((tokens, heads, dim), dtype=dtype, device=DEVICE),
            "k_out": torch.empty((tokens, kv_heads, dim), dtype=dtype, device=DEVICE)}


def _pool(blocks, case, noise):
    """A cache of codes and scales as earlier steps left them: channels of
    different size, a scale for every token and head."""
    shape = (blocks, case["kv_heads"], case["page"], case["dim"])
    state = {}
    for name in ("k", "v"):
        size = torch.exp(0.5 * torch.randn((case["kv_heads"], 1, case["dim"]), device=DEVICE, generator=noise))
        rows = torch.randn(shape, device=DEVICE, generator=noise) * size
        scale = rows.abs().amax(-1) / 127
        state[name + "_codes"] = torch.round(rows / scale[..., None]).to(torch.int8)
        state[name + "_scale"] = scale
    return state


def _prepare_store(case, order, noise):
    tokens, page, dtype = case["tokens"], case["page"], _TYPES[case["dtype"]]
    blocks = -(-tokens // page) + 8
    # runs of tokens in pages all over the pool
    first = torch.randperm(blocks, generator=order).to(DEVICE)
    at = torch.arange(tokens, device=DEVICE)
    shape = (tokens, case["kv_heads"], case["dim"])
    return _with_cache({"op": "store", "slots": first[at // page] * page + at % page, "dtype": dtype,
                        **_pool(blocks, case, noise),
                        "k": torch.randn(shape, dtype=dtype, device=DEVICE, generator=noise),
                        "v": torch.randn(shape, dtype=dtype, device=DEVICE, generator=noise),
                        "k_out": torch.empty(shape, dtype=dtype, device=DEVICE),
                        "v_out": torch.empty(shape, dtype=dtype, device=DEVICE)})


def _pages(lens, most, page, order):
    """(block table, blocks of the pool) of requests of these lengths, at most
    `most` each: blocks scattered, unused entries -1."""
    width = max(1, -(-most // page))
    held = ((lens + page - 1) // page).long()
    blocks = int(held.sum()) + 8
    place = torch.arange(width, device=DEVICE)
    rank = (torch.cumsum(held, 0) - held)[:, None] + place
    ids = torch.randperm(blocks, generator=order).to(torch.int32).to(DEVICE)
    return torch.where(place < held[:, None], ids[rank.clamp(max=blocks - 1)], -1), blocks


def _prepare_read(case, order, noise):
    page, dtype = case["page"], _TYPES[case["dtype"]]
    lens = _lengths(case["len_lo"], case["len_hi"], case["batch"], order)
    table, blocks = _pages(lens, case["len_hi"], page, order)
    # every request's slots in the order of its positions, then places that no token has
    total = sum(_spread(case["len_lo"], case["len_hi"], case["batch"]))
    ends = torch.cumsum(lens, 0)
    at = torch.arange(total, device=DEVICE)
    owner = torch.searchsorted(ends, at, right=True)
    position = at - (ends - lens)[owner]
    slots = torch.full((total + case["spare"],), -1, dtype=torch.int64, device=DEVICE)
    slots[:total] = table[owner, position // page].long() * page + position % page
    shape = (slots.numel(), case["kv_heads"], case["dim"])
    return _with_cache({"op": "read", "slots": slots, "dtype": dtype, **_pool(blocks, case, noise),
                        "k_out": torch.empty(shape, dtype=dtype, device=DEVICE),
                        "v_out": torch.empty(shape, dtype=dtype, device=DEVICE)})


def _prepare_attn(case, order, noise):
    batch, page, dtype = case["batch"], case["page"], _TYPES[case["dtype"]]
    lens = _lengths(case["len_lo"], case["len_hi"], batch, order)
    max_len, max_new, tokens, starts = case["len_hi"], 1, batch, None
    if case["new_hi"]:
        new = _lengths(case["new_lo"], case["new_hi"], batch, order)
        lens += new
        max_len, max_new = max_len + case["new_hi"], case["new_hi"]
        tokens = sum(_spread(case["new_lo"], case["new_hi"], batch))
        starts = torch.zeros(batch + 1, dtype=torch.int32, device=DEVICE)
        starts[1:] = torch.cumsum(new, 0)
    table, blocks = _pages(lens, max_len, page, order)
    q = torch.randn((tokens, case["heads"], case["dim"]), dtype=dtype, device=DEVICE, generator=noise)
    return _with_cache({"op": "attn", "q": q, "table": table, "lens": lens, "starts": starts, "max_len": max_len,
                        "max_new": max_new, "dtype": dtype, **_pool(blocks, case, noise), "out": torch.empty_like(q)})


def _with_cache(state):
    """The handle and the workspace that a program keeps from step to step."""
    if own:
        from block_wise_int4_amd import mnb
        state["cache"] = mnb.KvCacheI8(state["k_codes"], state["v_codes"], state["k_scale"], state["v_scale"],
                                       state["dtype"])
        if state["op"] == "attn":
            state["workspace"] = mnb.paged_attn_i8_workspace(state["q"], state["cache"], state["table"],
                                                             state["max_len"], state["max_new"])
    return state


_PREPARE = {"rope": _prepare_rope, "store": _prepare_store, "read": _prepare_read, "attn": _prepare_attn}


def run(state):
    return (_OWN if own else _PLAIN)[state["op"]](state)


def _own_rope(s):
    from block_wise_int4_amd import mnb
    return mnb.mnb_rope(s["q"], s["k"], s["positions"], s["freqs"], interleaved=s["interleaved"], gain=s["gain"],
                        q_out=s["q_out"], k_out=s["k_out"])


def _own_store(s):
    from block_wise_int4_amd import mnb
    mnb.mnb_kv_append_i8(s["k"], s["v"], s["slots"], s["cache"])
    k, v = mnb.mnb_kv_read_i8(s["slots"], s["cache"], k=s["k_out"], v=s["v_out"])
    return k, v, s["k_scale"], s["v_scale"]


def _own_read(s):
    from block_wise_int4_amd import mnb
    return mnb.mnb_kv_read_i8(s["slots"], s["cache"], k=s["k_out"], v=s["v_out"])


def _own_attn(s):
    from block_wise_int4_amd import mnb
    return mnb.mnb_paged_attn_i8(s["q"], s["cache"], s["table"], s["lens"], s["max_len"], starts=s["starts"],
                                 max_new=s["max_new"], workspace=s["workspace"], out=s["out"])


_OWN = {"rope": _own_rope, "store": _own_store, "read": _own_read, "attn": _own_attn}


def _turn(x, cos, sin, interleaved):
    """x [tokens, heads, dim] with its first 2 * cos.shape[2] dimensions turned."""
    rot = 2 * cos.shape[2]
    y = x[..., :rot].float()
    if interleaved:
        a, b = y[..., 0::2], y[..., 1::2]
        y = torch.stack((a * cos - b * sin, a * sin + b * cos), dim=-1).flatten(-2)
    else:
        a, b = y[..., :rot // 2], y[..., rot // 2:]
        y = torch.cat((a * cos - b * sin, a * sin + b * cos), dim=-1)
    return torch.cat((y.to(x.dtype), x[..., rot:]), dim=-1)


def _plain_rope(s):
    # (angles in 64 bits: a far position times a frequency loses its fraction of a turn in 32)
    angle = (s["positions"].double()[:, None] * s["freqs"])[:, None]
    cos, sin = (torch.cos(angle) * s["gain"]).float(), (torch.sin(angle) * s["gain"]).float()
    return _turn(s["q"], cos, sin, s["interleaved"]), _turn(s["k"], cos, sin, s["interleaved"])


def _place(s):
    page = s["k_codes"].shape[2]
    return s["slots"].clamp(min=0) // page, s["slots"].clamp(min=0) % page


def _values(s, name, block, offset):
    return s[name + "_codes"][block, :, offset].float() * s[name + "_scale"][block, :, offset][..., None]


def _plain_store(s):
    block, offset = _place(s)
    s["k_codes"][block, :, offset], s["k_scale"][block, :, offset] = _quantise(s["k"])
    s["v_codes"][block, :, offset], s["v_scale"][block, :, offset] = _quantise(s["v"])
    return *_plain_read(s), s["k_scale"], s["v_scale"]


def _plain_read(s):
    block, offset = _place(s)
    there = (s["slots"] >= 0)[:, None, None]
    return (torch.where(there, _values(s, "k", block, offset), 0.0).to(s["dtype"]),
            torch.where(there, _values(s, "v", block, offset), 0.0).to(s["dtype"]))


def _plain_attn(s):
    q, page = s["q"], s["k_codes"].shape[2]
    tokens, heads, dim = q.shape
    batch, kv_heads, group = s["lens"].numel(), s["k_codes"].shape[1], heads // s["k_codes"].shape[1]
    at = torch.arange(max(1, s["max_len"]), device=q.device)
    block, offset = s["table"][:, at // page].clamp(min=0).long(), (at % page).expand(batch, -1)
    k, v = _values(s, "k", block, offset).transpose(1, 2), _values(s, "v", block, offset).transpose(1, 2)
    # rows [batch, new, heads, dim], and how many keys each sees
    lens = s["lens"].long()
    new = torch.arange(s["max_new"], device=q.device)
    if s["starts"] is None:
        rows, sees = q[:, None], lens[:, None]
    else:
        first = s["starts"][:-1].long()
        sees = lens[:, None] - (s["starts"][1:].long() - first)[:, None] + new + 1
        rows = q[(first[:, None] + new).clamp(max=tokens - 1)]
    rows = rows.float().view(batch, -1, kv_heads, group, dim).permute(0, 2, 1, 3, 4).reshape(batch, kv_heads, -1, dim)
    valid = (at < sees[:, :, None]) & (at < lens[:, None, None])
    valid = valid.repeat_interleave(group, 1)[:, None]
    score = torch.matmul(rows * dim ** -0.5, k.transpose(2, 3)).masked_fill(~valid, -math.inf)
    top = score.amax(3, keepdim=True)
    weight = torch.exp(score - torch.where(top == -math.inf, 0.0, top))
    total = weight.sum(3, keepdim=True)
    mixed = torch.where(total == 0, 0.0, torch.matmul(weight, v) / total)
    mixed = mixed.view(batch, kv_heads, -1, group, dim).permute(0, 2, 1, 3, 4).reshape(batch, -1, heads, dim)
    if s["starts"] is None:
        return mixed[:, 0].to(q.dtype)
    row = torch.arange(tokens, device=q.device)
    owner = torch.searchsorted(s["starts"][1:].long(), row, right=True).clamp(max=batch - 1)
    return mixed[owner, row - first[owner]].to(q.dtype)


_PLAIN = {"rope": _plain_rope, "store": _plain_store, "read": _plain_read, "attn": _plain_attn}


def work(case):
    if case["op"] == "rope":
        heads, size = case["heads"] + case["kv_heads"], _BYTES[case["dtype"]]
        return {"bytes": case["tokens"] * (2 * heads * case["dim"] * size + 4) + 4 * case["rot"],
                "flops": 3 * case["tokens"] * heads * case["rot"]}
    # a token's keys and values of all heads: as numbers, and as codes with their scales
    wide = 2 * case["kv_heads"] * case["dim"] * _BYTES[case["dtype"]]
    narrow = 2 * case["kv_heads"] * (case["dim"] + 4)
    if case["op"] == "store":   # numbers in, codes out, numbers out; the scales are an output
        return {"bytes": case["tokens"] * (2 * wide + narrow + 16), "flops": 0}
    lens = _spread(case["len_lo"], case["len_hi"], case["batch"])
    if case["op"] == "read":
        return {"bytes": sum(lens) * (wide + narrow) + case["spare"] * wide + 8 * (sum(lens) + case["spare"]),
                "flops": 0}
    new = _spread(case["new_lo"], case["new_hi"], case["batch"]) if case["new_hi"] else [1] * case["batch"]
    keys, tokens = sum(lens), sum(new)
    if case["new_hi"]:
        # (which prefix meets which number of new tokens goes by the seed: their mean)
        seen = tokens * keys / case["batch"] + sum(n * (n + 1) // 2 for n in new)
        keys += tokens
    else:
        seen = keys
    size = 2 * tokens * case["heads"] * case["dim"] * _BYTES[case["dtype"]]
    return {"bytes": keys * narrow + size + 4 * keys / case["page"] + 8 * case["batch"],
            "flops": int(4 * seen * case["heads"] * case["dim"])}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        angle = torch.outer(s["positions"].double(), s["freqs"].double())
        factor = torch.polar(torch.full_like(angle, s["gain"]), angle)[:, None]
        out = []
        for x in (s["q"].double(), s["k"].double()):
            half = case["rot"] // 2
            pairs = x[..., :case["rot"]].unflatten(-1, (half, 2) if case["interleaved"] else (2, half))
            if not case["interleaved"]:
                pairs = pairs.transpose(-1, -2)
            turned = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * factor)
            if not case["interleaved"]:
                turned = turned.transpose(-1, -2)
            out.append(torch.cat((turned.flatten(-2), x[..., case["rot"]:]), dim=-1))
        return tuple(out)
    if case["op"] == "store":
        back, scales = [], []
        for name in ("k", "v"):
            x = s[name].double()
            step = (x.abs().amax(-1, keepdim=True) / 127).float().double()
            back.append(torch.round(x / step) * step)
            rows = s[name + "_scale"].double().permute(0, 2, 1).flatten(0, 1)
            rows.index_copy_(0, s["slots"], step[..., 0])
            scales.append(rows.unflatten(0, (-1, case["page"])).permute(0, 2, 1).contiguous())
        return (*back, *scales)
    if case["op"] == "read":
        out = []
        for name in ("k", "v"):
            rows = (s[name + "_codes"].double() * s[name + "_scale"].double()[..., None]).permute(0, 2, 1, 3)
            rows = rows.flatten(0, 1)
            rows = torch.cat((rows, torch.zeros_like(rows[:1])))   # (slot -1: the row of zeros behind them)
            out.append(rows[s["slots"]])
        return tuple(out)
    q = s["q"].double()
    out = torch.zeros_like(q)
    group = case["heads"] // case["kv_heads"]
    first = list(range(case["batch"] + 1)) if s["starts"] is None else s["starts"].tolist()
    for b, n in enumerate(s["lens"].tolist()):
        mine, count = slice(first[b], first[b + 1]), first[b + 1] - first[b]
        if n == 0 or count == 0:
            continue  # nothing to attend to: zeros
        pages = s["table"][b, : -(-n // case["page"])].long()
        k, v = ((s[c + "_codes"][pages].double() * s[c + "_scale"][pages].double()[..., None]).permute(1, 0, 2, 3)
                .flatten(1, 2)[:, :n] for c in ("k", "v"))
        x = q[mine].permute(1, 0, 2).reshape(case["kv_heads"], group * count, case["dim"])
        score = torch.bmm(x, k.transpose(1, 2).contiguous()) / math.sqrt(case["dim"])
        hidden = torch.ones((count, n), dtype=torch.bool, device=DEVICE).triu(n - count + 1).repeat(group, 1)
        p = torch.softmax(score.masked_fill(hidden, -math.inf), dim=2)
        out[mine] = torch.bmm(p, v.contiguous()).view(case["heads"], count, case["dim"]).permute(1, 0, 2)
    return out
