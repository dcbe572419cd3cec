"""GPU: rotary positions, the 8-bit key-value cache and the attention over it as a
decoder runs them, and the sizes at which their calls take another form, against
the float64 oracle. Codes, scales and what is read back are compared exactly,
attention outputs within the bound of `test_gpu_cache8`, whose derivation stands
there.
"""

import numpy as np
import pytest
import torch

import oracle
from block_wise_int4_amd import mnb
from test_gpu_cache8 import DEV, TD, _bound, _cache, _case, _check, _near, _np

pytestmark = pytest.mark.gpu

I32 = dict(dtype=torch.int32, device=DEV)
I64 = dict(dtype=torch.int64, device=DEV)


# ---------------------------------------------------------------------------
# a decoder's use of them
# ---------------------------------------------------------------------------

class Layer:
    """The attention half of one decoder layer: fused rows of queries, keys and
    values are given their positions, appended to an 8-bit cache, attended."""

    def __init__(self, dt, batch, heads, kv_heads, dim, page, max_len, seed):
        self.dt, self.heads, self.kv_heads, self.dim, self.page, self.max_len = dt, heads, kv_heads, dim, page, max_len
        self.gen = torch.Generator(DEV).manual_seed(seed)
        width = -(-max_len // page)
        self.cache = _cache(batch * width, kv_heads, page, dim, dt)
        self.table = torch.full((batch, width), -1, **I32)
        self.free = torch.randperm(batch * width, generator=self.gen, device=DEV).int()
        self.lens = torch.zeros(batch, **I32)
        self.freqs, self.gain = mnb.rope_frequencies(dim, base=1e4, device=DEV)

    def rows(self, tokens):
        width = (self.heads + 2 * self.kv_heads) * self.dim
        return torch.randn((tokens, width), device=DEV, generator=self.gen).to(TD[self.dt])

    def split(self, x):
        q, kv = self.heads * self.dim, self.kv_heads * self.dim
        return (x[:, :q].unflatten(1, (self.heads, -1)), x[:, q: q + kv].unflatten(1, (self.kv_heads, -1)),
                x[:, q + kv:].unflatten(1, (self.kv_heads, -1)))

    def place(self, added):
        slots = torch.empty(sum(added), **I64)
        lens, starts, _, taken = mnb.mnb_kv_tables(self.lens, torch.tensor(added, **I32), self.free, self.table,
                                                   self.page, slots)
        self.free, self.lens = self.free[int(taken):], lens
        return slots, starts


@pytest.mark.parametrize("dt,heads,kv_heads,dim,page", [("f16", 16, 8, 128, 16), ("f16", 8, 1, 64, 32),
                                                        ("f32", 6, 6, 64, 16), ("f32", 10, 2, 128, 48)])
def test_prompts_and_steps(dt, heads, kv_heads, dim, page):
    print(f"decoder {dt} {heads}/{kv_heads} dim={dim} page={page}", flush=True)
    d = Layer(dt, 4, heads, kv_heads, dim, page, 120, seed=1)
    prompts, steps = [33, 1, 70, 0], 3
    held = [[] for _ in prompts]      # rotated keys and values of each request, as they were appended
    for step in range(steps + 1):
        added = prompts if step == 0 else [1, 1, 1, 1]
        before = d.lens.tolist()
        slots, starts = d.place(added)
        x = d.rows(sum(added))
        q, k, v = d.split(x)
        positions = torch.tensor([before[b] + i for b, n in enumerate(added) for i in range(n)], **I32)
        plain = _np(q), _np(k)
        mnb.mnb_rope(q, k, positions, d.freqs, gain=d.gain, q_out=q, k_out=k)     # in place, columns of one buffer
        for got, old in zip((q, k), plain):
            want = oracle.rope(old, positions.tolist(), d.freqs.tolist(), False, d.gain)
            # cosine and sine 2^-23 each, products and their sum 3 roundings of 2^-24, the output's half step
            pair = np.abs(old).reshape(*old.shape[:-1], 2, -1).sum(axis=-2, keepdims=True)
            near = (pair * np.ones((2, 1))).reshape(old.shape)
            _near(_np(got), want, near * 2.0 ** -21 + np.abs(want) * torch.finfo(TD[dt]).eps / 2 + 2.0 ** -25, "rotated")
        mnb.mnb_kv_append_i8(k, v, slots, d.cache)
        at = 0
        for b, n in enumerate(added):
            held[b] += [(_np(k[at + i]), _np(v[at + i])) for i in range(n)]
            at += n
        if step == 0:
            out = mnb.mnb_paged_attn_i8(q, d.cache, d.table, d.lens, d.max_len, starts=starts, max_new=max(added))
            done = _check(out, q, d.cache, d.table, d.lens, starts, d.max_len, max(added), dt, what="prompts")
        else:
            out = mnb.mnb_paged_attn_i8(q, d.cache, d.table, d.lens, d.max_len)
            done = _check(out, q, d.cache, d.table, d.lens, None, d.max_len, 1, dt, what=f"step {step}")
        assert done == set(range(sum(added)))
    # every token is where its table says, quantized from what was appended
    frames = int(d.lens.max())
    slots = torch.full((4, frames), -1, **I64)
    for b, n in enumerate(d.lens.tolist()):
        at = torch.arange(n, device=DEV)
        slots[b, :n] = d.table[b, at // page].long() * page + at % page
    back = mnb.mnb_kv_read_i8(slots.view(-1), d.cache)
    for which, got in enumerate(back):
        got = _np(got).reshape(4, frames, kv_heads, dim)
        for b, rows in enumerate(held):
            codes, scales = oracle.quantize_rows(np.stack([r[which] for r in rows]))
            exact = codes.astype(np.float64) * scales.astype(np.float64)[..., None]
            assert np.array_equal(got[b, : len(rows)], exact.astype(np.float16 if dt == "f16" else np.float32))
            assert not got[b, len(rows):].any()
    # the rows read back, given to the attention over whole tensors, say what the cache says
    if dt == "f32":
        k, v = (x.view(4, frames, kv_heads, dim) for x in back)
        other = mnb.mnb_cross_attn(q.view(4, 1, heads, dim), k, v, d.lens).view(4, heads, dim)
        _check(other, q, d.cache, d.table, d.lens, None, d.max_len, 1, dt, what="read back")


def test_a_step_captured_and_replayed():
    d = Layer("f16", 5, 8, 4, 64, 16, 200, seed=2)
    prompts = [60, 16, 1, 100, 15]
    slots, starts = d.place(prompts)
    x = d.rows(sum(prompts))
    q, k, v = d.split(x)
    mnb.mnb_rope(q, k, torch.cat([torch.arange(n) for n in prompts]).int().to(DEV), d.freqs, q_out=q, k_out=k)
    mnb.mnb_kv_append_i8(k, v, slots, d.cache)
    work = mnb.paged_attn_i8_workspace(q[:5], d.cache, d.table, d.max_len)
    x, positions, slots = d.rows(5), torch.zeros(5, **I32), torch.zeros(5, **I64)
    lens, turned = torch.zeros(5, **I32), torch.zeros((5, 4, 64), dtype=torch.float16, device=DEV)
    turned_q, out = torch.zeros((2, 5, 8, 64), dtype=torch.float16, device=DEV)

    def step(cache):
        q, k, v = d.split(x)
        mnb.mnb_rope(q, k, positions, d.freqs, q_out=turned_q, k_out=turned)
        mnb.mnb_kv_append_i8(turned, v, slots, cache)
        return mnb.mnb_paged_attn_i8(turned_q, cache, d.table, lens, d.max_len, workspace=work, out=out)
    same = mnb.KvCacheI8(*(t.clone() for t in (d.cache.k, d.cache.v, d.cache.k_scale, d.cache.v_scale)), torch.float16)
    step(same)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(d.cache)
    same = mnb.KvCacheI8(*(t.clone() for t in (d.cache.k, d.cache.v, d.cache.k_scale, d.cache.v_scale)), torch.float16)
    for i in range(4):
        positions.copy_(d.lens)
        s, _ = d.place([1] * 5)
        slots.copy_(s)
        lens.copy_(d.lens)
        x.copy_(d.rows(5))
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        got = out.clone()
        want = step(same).clone()
        assert torch.equal(got, want) and torch.equal(d.cache.k, same.k) and torch.equal(d.cache.v, same.v), i
        _check(got, turned_q, same, d.table, lens, None, d.max_len, 1, "f16", what=f"replay {i}")


def test_two_graphs_of_one_workspace_in_turn():
    # few rows and many rows, in pieces, through one workspace
    ca, cb = (_case(s, [4000, 2100], 4, 2, 64, 16, "f16", new=n) for s, n in ((21, None), (22, [40, 60])))
    need = [mnb.paged_attn_i8_workspace(c[0], c[1], c[2], 4000, n) for c, n in ((ca, 1), (cb, 60))]
    work = max(need, key=lambda w: w.numel())
    assert min(w.numel() for w in need) > 0
    outs = [torch.zeros_like(c[0]) for c in (ca, cb)]

    def run(c, n, out):
        q, cache, table, ln, starts = c
        return mnb.mnb_paged_attn_i8(q, cache, table, ln, 4000, starts=starts, max_new=n, workspace=work, out=out)
    want = [run(c, n, torch.zeros_like(c[0])) for c, n in ((ca, 1), (cb, 60))]
    torch.cuda.synchronize()
    graphs = []
    for c, n, out in ((ca, 1, outs[0]), (cb, 60, outs[1])):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            run(c, n, out)
        graphs.append(g)
    for _ in range(3):
        for g, out in zip(graphs, outs):
            out.zero_()
            g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o, w) for o, w in zip(outs, want))


def test_two_streams_at_once():
    cases = [_case(s, [3000] * 6, 16, 8, 128, 16, "f16", new=n) for s, n in ((23, None), (24, [20] * 6))]
    want = [mnb.mnb_paged_attn_i8(q, cache, table, ln, 3000, starts=starts, max_new=20 if starts is not None else 1)
            for q, cache, table, ln, starts in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    got = [[], []]
    for _ in range(4):
        for i, (q, cache, table, ln, starts) in enumerate(cases):
            with torch.cuda.stream(streams[i]):
                got[i].append(mnb.mnb_paged_attn_i8(q, cache, table, ln, 3000, starts=starts,
                                                    max_new=20 if starts is not None else 1))
    torch.cuda.synchronize()
    assert all(torch.equal(x, want[i]) for i in range(2) for x in got[i])


# ---------------------------------------------------------------------------
# where calls change their form
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("dt", ["f16", "f32"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("rows", [2, 3, 5, 6, 16, 17, 32, 33, 64, 65, 128, 129])
def test_rows_around_the_forms_limits(rows, dim, dt):
    print(f"rows {rows} dim={dim} {dt}", flush=True)
    # as heads that share a key-value head, and as new tokens of one head
    q, cache, table, ln, _ = _case(rows, [100, 7], rows, 1, dim, 16, dt)
    _check(mnb.mnb_paged_attn_i8(q, cache, table, ln, 100), q, cache, table, ln, None, 100, 1, dt)
    q, cache, table, ln, starts = _case(rows, [200, rows], 1, 1, dim, 16, dt, new=[rows, rows - 1])
    got = mnb.mnb_paged_attn_i8(q, cache, table, ln, 200, starts=starts, max_new=rows)
    _check(got, q, cache, table, ln, starts, 200, rows, dt)


@pytest.mark.parametrize("dt,dim", [("f16", 128), ("f16", 64), ("f32", 64)])
@pytest.mark.parametrize("keys", [255, 256, 257, 384, 385, 511, 512, 513, 767, 769, 1024, 1025, 1537])
def test_keys_around_the_pieces_limits(keys, dt, dim):
    for heads, new in ((2, None), (8, None), (2, [20, 40])):
        print(f"keys {keys} {dt} dim={dim} heads={heads} new={new}", flush=True)
        q, cache, table, ln, starts = _case(keys + heads, [keys, keys // 3], heads, 1, dim, 16, dt, new=new)
        n = max(new) if new else 1
        for bound in (keys, keys + 1000):       # (what is cut are the keys that max_len allows)
            got = mnb.mnb_paged_attn_i8(q, cache, table, ln, bound, starts=starts, max_new=n)
            _check(got, q, cache, table, ln, starts, bound, n, dt, what=f"max_len {bound}")


@pytest.mark.parametrize("dt", ["f16", "f32"])
@pytest.mark.parametrize("page", [16, 48, 1024])
def test_pages_of_other_sizes_in_pieces(page, dt):
    for new in (None, [33]):
        q, cache, table, ln, starts = _case(page, [2500], 2, 1, 64, page, dt, new=new)
        got = mnb.mnb_paged_attn_i8(q, cache, table, ln, 2500, starts=starts, max_new=33 if new else 1)
        _check(got, q, cache, table, ln, starts, 2500, 33 if new else 1, dt)


@pytest.mark.parametrize("dt", ["f16", "f32"])
def test_many_requests_most_of_them_empty(dt):
    lens = [0] * 300
    lens[7], lens[150], lens[299] = 70, 1, 33
    new = [0] * 300
    new[7], new[150], new[299] = 50, 1, 3
    for n in (None, new):
        q, cache, table, ln, starts = _case(31, lens, 4, 2, 64, 16, dt, new=n)
        got = mnb.mnb_paged_attn_i8(q, cache, table, ln, 70, starts=starts, max_new=50 if n else 1)
        _check(got, q, cache, table, ln, starts, 70, 50 if n else 1, dt)


@pytest.mark.parametrize("dt", ["f16", "f32"])
@pytest.mark.parametrize("new", [None, 2])
def test_as_many_requests_as_a_call_takes(new, dt):
    # 65536 requests over 40 blocks that they share, a block each; against plain products in float64
    B, heads, kv_heads, dim = 65536, 2, 1, 64
    g = torch.Generator(DEV).manual_seed(6)
    cache = _cache(40, kv_heads, 16, dim, dt)
    rows = [torch.randn((640, kv_heads, dim), device=DEV, generator=g).to(TD[dt]) for _ in range(2)]
    mnb.mnb_kv_append_i8(*rows, torch.arange(640, device=DEV), cache)
    ids = torch.randint(0, 40, (B, 1), device=DEV, generator=g).int()
    lens = torch.randint(0, 17, (B,), device=DEV, generator=g).int()
    tokens = B * (new or 1)
    q = torch.randn((tokens, heads, dim), device=DEV, generator=g).to(TD[dt])
    starts = None if new is None else torch.arange(0, tokens + 1, new, **I32)
    got = mnb.mnb_paged_attn_i8(q, cache, ids, lens, 16, starts=starts, max_new=new or 1)
    k, v = ((c.double() * s.double()[..., None])[:, 0] for c, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)))
    at = ids[:, 0].long().repeat_interleave(new or 1)
    sees = lens.long() if new is None else (lens.long()[:, None] + torch.tensor([-1, 0], device=DEV)).clamp(min=0).flatten()
    score = (q.double()[:, :, None, :] * k[at][:, None]).sum(dim=-1) * dim ** -0.5
    hidden = torch.arange(16, device=DEV)[None, None, :] >= sees[:, None, None]
    w = torch.where(hidden, 0.0, torch.exp(score - score.amax(dim=-1, keepdim=True)))
    total = w.sum(dim=-1, keepdim=True)
    p = torch.where(total > 0, w / total, 0.0)
    want = (p[..., None] * v[at][:, None]).sum(dim=2)
    a = (p[..., None] * v[at][:, None].abs()).sum(dim=2)
    # the bound of one row, with |q|, |k| and |v| at their largest here
    u, s_abs = 2.0 ** -24, float((q.double().abs().amax() * k.abs().sum(dim=-1).amax()) * dim ** -0.5)
    rel = 2 * (2 * ((dim + 8) * u * s_abs + 4 * u * s_abs) + 2.0 ** -21 + 80 * u)
    tol = a * rel + 16 * 2.0 ** -21 * float(v.abs().amax()) + want.abs() * u + 1e-30
    if dt == "f16":
        tol += a * 2.0 ** -10 + 16 * 2.0 ** -25 * float(v.abs().amax()) + want.abs() * 2.0 ** -11 + 2.0 ** -25
    assert ((got.double() - want).abs() <= tol).all()
    assert not got[sees == 0].any()


def test_more_tokens_than_a_launch_has_workgroups_for():
    # 64 tokens a workgroup, 65536 workgroups: the rest in a second turn
    T = (1 << 22) + 12345
    g = torch.Generator(DEV).manual_seed(7)
    cache = _cache(-(-T // 16), 1, 16, 64, "f16")
    x = torch.randn((T, 1, 64), dtype=torch.float16, device=DEV, generator=g)
    slots = torch.randperm(T, device=DEV)
    mnb.mnb_kv_append_i8(x, x.neg(), slots, cache)
    back = mnb.mnb_kv_read_i8(slots, cache)
    for got, rows in zip(back, (x, -x)):
        # half a code's step, amax / 254, and half a step of float16 in what is read back, 2^-11 of at most
        # amax (1 + 1 / 254); the scale's rounding, 2^-24 of amax, with it: below 1 / 254 + 2^-11 + 2^-18
        most = rows.float().abs().amax(dim=-1, keepdim=True) * (1 / 254 + 2.0 ** -11 + 2.0 ** -18)
        assert ((got.float() - rows.float()).abs() <= most).all()
    some = torch.cat([torch.arange(5, device=DEV), torch.arange(T - 5, T, device=DEV),
                      torch.randint(0, T, (200,), device=DEV)])
    codes, scales = oracle.quantize_rows(_np(x[some]))
    at = slots[some]
    assert np.array_equal(cache.k[at // 16, :, at % 16].cpu().numpy(), codes)
    assert np.array_equal(cache.k_scale[at // 16, :, at % 16].cpu().numpy(), scales)


# ---------------------------------------------------------------------------
# far places, far scales, repeated slots
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("dt,dim", [("f16", 64), ("f16", 128), ("f32", 64), ("f32", 128)])
def test_rows_of_all_exponents(dt, dim):
    rng = np.random.default_rng(dim)
    low, high, most = (-149, 127, 3.4028234e38) if dt == "f32" else (-24, 15, 65504.0)
    x = rng.uniform(-1.9, 1.9, (600, 2, dim)) * 2.0 ** rng.uniform(low, high, (600, 2, 1))
    grid = 2.0 ** np.floor(rng.uniform(max(low, -120), high - 8, (86, 2, 1)))
    x[::7] = np.round(rng.uniform(-127.5, 127.5, (86, 2, dim)) * 2) / 2 * grid      # halves between codes
    rows = torch.from_numpy(np.clip(x, -most, most)).to(TD[dt]).to(DEV)
    cache, slots = _cache(38, 2, 16, dim, dt), torch.arange(600, device=DEV)
    mnb.mnb_kv_append_i8(rows, rows, slots, cache)
    codes, scales = oracle.quantize_rows(_np(rows))
    assert np.array_equal(cache.v.transpose(1, 2).reshape(-1, 2, dim)[:600].cpu().numpy(), codes)
    assert np.array_equal(cache.v_scale.transpose(1, 2).reshape(-1, 2)[:600].cpu().numpy(), scales)
    exact = codes.astype(np.float64) * scales.astype(np.float64)[..., None]
    assert np.array_equal(mnb.mnb_kv_read_i8(slots, cache)[0].cpu().numpy(),
                          exact.astype(np.float16 if dt == "f16" else np.float32))


@pytest.mark.parametrize("new", [None, [9, 4], [40, 50]])
def test_offsets_past_32_bits(new):
    # blocks 2^17 bytes apart, 40000 of them; scales 2^16 numbers apart; rows of q 2^26 bytes apart
    blocks, heads, page, dim = 40000, 2, 16, 128
    codes = torch.empty(blocks << 17, dtype=torch.int8, device=DEV)
    scales = torch.empty(blocks << 16, dtype=torch.float32, device=DEV)
    step, srow = (1 << 17, page * dim, dim, 1), (1 << 16, page, 1)
    k, v = (torch.as_strided(codes, (blocks, heads, page, dim), step, at) for at in (0, 1 << 16))
    ks, vs = (torch.as_strided(scales, (blocks, heads, page), srow, at) for at in (0, 1 << 15))
    cache = mnb.KvCacheI8(k, v, ks, vs, torch.float16)
    lens = [75, 50]
    table = torch.tensor([[39999, 16384, 16383, 32768, 3], [20000, 39998, 32767, 0, -1]], **I32)
    g = torch.Generator(DEV).manual_seed(3)
    at = [(b, t) for b, n in enumerate(lens) for t in range(n)]
    slots = torch.tensor([int(table[b, t // page]) * page + t % page for b, t in at], **I64)
    rows = [torch.randn((len(at), heads, dim), device=DEV, generator=g).half() for _ in range(2)]
    mnb.mnb_kv_append_i8(*rows, slots, cache)
    back = mnb.mnb_kv_read_i8(slots, cache)
    for got, x in zip(back, rows):
        c, s = oracle.quantize_rows(_np(x))
        assert np.array_equal(got.cpu().numpy(), (c * s.astype(np.float64)[..., None]).astype(np.float16))
    tokens = 2 if new is None else sum(new)
    wide = torch.empty(tokens << 25, dtype=torch.float16, device=DEV)
    q = torch.as_strided(wide, (tokens, 4, dim), (1 << 25, dim, 1))
    q.copy_(torch.randn((tokens, 4, dim), device=DEV, generator=g))
    n = max(new) if new else 1
    starts = None if new is None else torch.tensor([0, new[0], tokens], **I32)
    ln = torch.tensor(lens, **I32)
    got = mnb.mnb_paged_attn_i8(q, cache, table, ln, 80, starts=starts, max_new=n)
    # the oracle's cache: the blocks that are used, gathered
    ids = table.flatten()[table.flatten() >= 0].long()
    small = mnb.KvCacheI8(*(t[ids].contiguous() for t in (k, v, ks, vs)), torch.float16)
    where = {int(i): n for n, i in enumerate(ids)}
    renamed = torch.tensor([[where.get(int(i), -1) for i in row] for row in table], **I32)
    _check(got, q.contiguous(), small, renamed, ln, starts, 80, n, "f16")


@pytest.mark.parametrize("new", [None, [20, 40]])
def test_float16_scales_up_to_the_largest(new):
    # differences of scores are then far above any exponent: the largest key's value alone
    q, cache, table, ln, starts = _case(41, [300, 90], 2, 1, 64, 16, "f16", new=new)
    for b in range(2):
        cache.k[int(table[b, 0]), :, 5] = 127          # far above the others, in every query
        cache.k_scale[int(table[b, 0]), :, 5] = 1.0
    q.abs_().add_(0.5)
    n = 40 if new else 1
    for scale in (1e10, 1e24, 1e30, 3e38):
        got = mnb.mnb_paged_attn_i8(q, cache, table, ln, 300, starts=starts, max_new=n, scale=scale)
        at = 0
        for b in range(2):
            rows = got[at: at + (new[b] if new else 1)].double()
            at += rows.shape[0]
            where = int(table[b, 0]), 0, 5
            want = cache.v[where].double() * cache.v_scale[where].double()
            # one weight: its product with the value scale and the output, each rounded to float16
            assert ((rows - want).abs() <= want.abs() * (2.0 ** -10 + 2.0 ** -20) + 2.0 ** -25).all(), (scale, b)


@pytest.mark.parametrize("size", [1e2, 3e3, 1e5, 1e7, 1e9, 3e10])
@pytest.mark.parametrize("dt,new,keys", [("f16", None, 700), ("f16", [20, 20], 700), ("f16", [60, 40], 300),
                                         ("f16", [60, 40], 5000), ("f32", None, 700), ("f32", [60, 40], 300)])
def test_equal_scores_of_any_size_weigh_the_same(dt, new, keys, size):
    # keys of one score (half of them written as half the codes with twice the scale): the mean of
    # their values; a quarter of them far below, and none of it
    dim, heads = 64, 2
    for sign in (1, -1):
        q, cache, table, ln, starts = _case(51, [keys, keys // 2], heads, 1, dim, 16, dt, new=new)
        cache.k.fill_(64)
        cache.k[:, :, 1::2] = 32
        scale = torch.full_like(cache.k_scale, 1.0)
        scale[:, :, 1::2] = 2.0
        q.fill_(100.0)
        low = torch.zeros_like(scale, dtype=torch.bool)
        low[:, :, 3::4] = True
        cache.k_scale.copy_(torch.where(low, scale * (0.5 if sign > 0 else 2.0), scale))
        n = max(new) if new else 1
        by = sign * size / (dim * 100.0 * 64)
        got = _np(mnb.mnb_paged_attn_i8(q, cache, table, ln, keys, starts=starts, max_new=n, scale=by))
        vn, sn = _np(cache.v) * _np(cache.v_scale)[..., None], _np(cache.v_scale)
        rows = oracle.visible(q.shape[0], ln.tolist(), None if starts is None else starts.tolist(), keys, n)
        for b, t, m in rows:
            ids = table[b].cpu().numpy()
            v = oracle.paged_rows(vn, ids, m, 16)[:, 0]
            vs = oracle.paged_rows(sn[..., None], ids, m, 16)[:, 0, 0]
            keep = np.arange(m) % 4 != 3 if size > 50 else slice(None)
            v, vs = v[keep], vs[keep]
            want, a = v.mean(axis=0), np.abs(v).mean(axis=0)
            # sums of n terms; whole numbers of 21 bits of weights times value scales; the exponents' reference,
            # up to 2^12 a float32 number (2^-12 twice); float16: weights times value scales, and the output
            tol = a * (m + 64) * 2.0 ** -23 + 2.0 ** -21 * vs.max() * (np.abs(v) / vs[:, None]).mean(axis=0) + 2.0 ** -25
            tol += a * 2.0 ** -20 if dt == "f32" else a * (2.0 ** -11 + 2.0 ** -11) + np.abs(want) * 2.0 ** -11
            for h in range(heads):
                _near(got[t, h], want, tol, f"scores of {sign * size:g}, row {t} of {m} keys, head {h}")


@pytest.mark.parametrize("dt", ["f16", "f32"])
@pytest.mark.parametrize("new,keys", [(None, 300), ([20, 20], 300), ([60, 40], 300), ([60, 40], 2000)])
def test_values_of_zeros(dt, new, keys):
    q, cache, table, ln, starts = _case(52, [keys, 70], 2, 1, 64, 16, dt, new=new)
    cache.v_scale.zero_()
    got = mnb.mnb_paged_attn_i8(q, cache, table, ln, keys, starts=starts, max_new=max(new) if new else 1)
    assert not got.any()
    cache.v_scale.fill_(1.0)
    cache.v.zero_()
    cache.v_scale.view(-1)[::3] = 0.0
    assert not mnb.mnb_paged_attn_i8(q, cache, table, ln, keys, starts=starts, max_new=max(new) if new else 1).any()


@pytest.mark.parametrize("dt", ["f16", "f32"])
@pytest.mark.parametrize("new,keys", [(None, 300), ([20, 20], 300), ([60, 60], 300), ([60, 60], 2000)])
def test_large_values_of_little_or_no_weight(dt, new, keys):
    # values of 0.001 beside one of 60000 that a row does not see, or whose key lies far below the
    # others, before or behind them; and keys that rise, from large values to small ones
    n = max(new) if new else 1
    for at in ("last", 3, 100, keys - 70, "rising"):
        q, cache, table, ln, starts = _case(53, [keys, 250], 2, 1, 64, 16, dt, new=new)
        cache.v_scale.copy_(torch.where(torch.isfinite(cache.v_scale), cache.v_scale * 1e-3, cache.v_scale))
        q.copy_(q * 0.1 + 1.0)
        for b, held in enumerate((keys, 250)):
            def place(t):
                return int(table[b, t // 16]), 0, t % 16
            if at == "rising":      # values fall by 2^25 over the keys, scores rise by 2^40
                for t in range(held):
                    part = t / (held - 1)
                    cache.v_scale[place(t)] = 400.0 * 2.0 ** (-25 * part)
                    cache.k[place(t)] = 64
                    cache.k_scale[place(t)] = 40 * 0.6931 * part / 64 / 8
                continue
            t = held - 1 if at == "last" else at if at < held else 7
            cache.v[place(t)] = 127
            cache.v_scale[place(t)] = 60000.0 / 127
            if at != "last":
                cache.k[place(t)] = -127
                cache.k_scale[place(t)] = 60.0 / 127 / 8
        got = mnb.mnb_paged_attn_i8(q, cache, table, ln, keys, starts=starts, max_new=n)
        _check(got, q, cache, table, ln, starts, keys, n, dt, what=f"value at {at}")


@pytest.mark.parametrize("dt", ["f16", "f32"])
def test_the_same_slot_twice_and_requests_that_share_blocks(dt):
    cache = _cache(4, 2, 16, 64, dt, code=3, scale=0.5)
    g = torch.Generator(DEV).manual_seed(5)
    x = torch.randn((3, 2, 64), device=DEV, generator=g).to(TD[dt])
    rows = x[[0, 0, 1, 2, 2, 2]].contiguous()
    slots = torch.tensor([7, 7, 20, 63, 63, 63], **I64)
    mnb.mnb_kv_append_i8(rows, rows, slots, cache)       # equal rows: either is both
    c, s = oracle.quantize_rows(_np(x))
    for i, slot in enumerate((7, 20, 63)):
        assert np.array_equal(cache.k[slot // 16, :, slot % 16].cpu().numpy(), c[i])
        assert np.array_equal(cache.v_scale[slot // 16, :, slot % 16].cpu().numpy(), s[i])
    # a common prefix, held once
    q, cache, table, ln, _ = _case(42, [80, 80], 2, 1, 64, 16, dt)
    table[1, :3] = table[0, :3]
    got = mnb.mnb_paged_attn_i8(q, cache, table, ln, 80)
    _check(got, q, cache, table, ln, None, 80, 1, dt)


def test_a_row_of_the_bound_is_what_the_formula_gives():
    # the bound itself, planted with a mistake in the oracle: a key left out is seen
    q, cache, table, ln, _ = _case(43, [40], 1, 1, 64, 16, "f32")
    got = _np(mnb.mnb_paged_attn_i8(q, cache, table, ln, 40))[0, 0]
    k, v = (_np(c) * _np(s)[..., None] for c, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)))
    k, v, s = (oracle.paged_rows(x, table[0].cpu().numpy(), 40, 16)[:, 0] for x in (k, v, _np(cache.v_scale)[..., None]))
    tol = _bound(_np(q)[0, 0], k, v, s[:, 0], 0.125, "f32")
    assert (np.abs(got - oracle.attend(_np(q)[0, 0], k, v, 0.125)) <= tol).all()
    assert (np.abs(got - oracle.attend(_np(q)[0, 0], k[1:], v[1:], 0.125)) > tol).any()
