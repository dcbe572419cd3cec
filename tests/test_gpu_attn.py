"""GPU: the decoder's attention operators against the float64 oracle.

Tables, slots and the append are compared exactly. Attention outputs are
compared within a bound worked out per output from the inputs (`_bound`):
with u = 2^-24, n valid keys, S the largest sum of |scale q_i k_i| of a score
and A = sum p |v| / sum p,

  a score is a float32 dot product of D terms, scaled: off by (D + 4) u S;
  its difference from the maximum, times log2(e), rounded: 4 u S more;
  so a weight exp(s - m) is off by 2 (D + 8) u S relative, plus 2^-21 for the
  exponential and the joining factors, in the numerator and the denominator;
  sums of n weights, in any order: n u each, plus 64 u for the joins;

and for float16 also the weights' rounding to float16 (2^-11 relative, at
most 2^-25 absolute against a largest weight of at least 1) and the output's
(2^-11 relative, 2^-25 absolute).
"""

import numpy as np
import pytest
import torch

import oracle
from block_wise_int4_amd import mnb

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
TD = {"f16": torch.float16, "f32": torch.float32}
NAN, INF = float("nan"), float("inf")


def _bound(q, k, v, scale, dt):
    """Per-output bound for one query row q [D] over valid rows k, v [n, D]."""
    n, dim = k.shape
    if n == 0:
        return np.zeros(v.shape[1])
    u = 2.0 ** -24
    s_abs = (np.abs(k * q).sum(axis=1) * abs(scale)).max()
    score = (k * q).sum(axis=1) * scale
    p = np.exp(score - score.max())
    a = (p[:, None] * np.abs(v)).sum(axis=0) / p.sum()
    tol = a * 2 * (2 * (dim + 8) * u * s_abs + 2.0 ** -21 + (n + 64) * u) + 1e-30
    if dt == "f16":
        y = np.abs((p[:, None] * v).sum(axis=0)) / p.sum()
        tol += a * 2 * 2.0 ** -11 + n * 2.0 ** -25 * np.abs(v).max() + y * 2.0 ** -11 + 2.0 ** -25
    return tol


def _near(got, ref, tol, what=""):
    worst = np.max(np.abs(got - ref) / np.maximum(tol, 1e-300), initial=0.0)
    assert np.all(np.isfinite(got)) and worst <= 1.0, f"{what}: {worst:.3f} of the bound"


def _np(t):
    return t.cpu().double().numpy()


# ---------------------------------------------------------------------------
# tables
# ---------------------------------------------------------------------------

def _tables(cached, added, free, table, page, tokens):
    i32 = dict(dtype=torch.int32, device=DEV)
    t = torch.tensor(table, **i32)
    slots = torch.full((tokens,), -77, dtype=torch.int64, device=DEV)
    args = (torch.tensor(cached, **i32), torch.tensor(added, **i32), torch.tensor(free, **i32), t, page, slots)
    lens, starts, slots, taken = mnb.mnb_kv_tables(*args)
    first = [x.clone() for x in (t, lens, starts, slots, taken)]
    mnb.mnb_kv_tables(*args, lens=lens, starts=starts, taken=taken)   # on its own result
    torch.cuda.synchronize()
    for x, y in zip(first, (t, lens, starts, slots, taken)):
        assert torch.equal(x, y)
    return [_np(x).astype(np.int64) for x in (t, lens, starts, slots, taken)]


def _check_tables(cached, added, free, table, page, tokens):
    got = _tables(cached, added, free, table, page, tokens)
    ref = oracle.kv_tables(cached, added, free, table, page, tokens)
    for g, r, name in zip(got, ref, ("table", "lens", "starts", "slots", "taken")):
        assert np.array_equal(g, np.asarray(r).reshape(g.shape)), name


@pytest.mark.parametrize("batch", [1, 3, 64, 257, 1023, 1024, 1025, 2500])
@pytest.mark.parametrize("page,width", [(16, 20), (48, 7), (128, 3)])
def test_tables(batch, page, width):
    print(f"tables batch={batch} page={page} width={width}", flush=True)
    rng = np.random.default_rng(batch * 7 + page)
    cached = rng.integers(0, width * page + 1, batch)
    added = rng.integers(0, 60, batch) * (rng.random(batch) < 0.7)
    table = rng.integers(0, 10 ** 6, (batch, width))
    need = int(oracle.kv_tables(cached, added, [], table, page, 0)[4])
    total = int(added.sum())
    free = rng.permutation(need + 5) + 10 ** 6
    _check_tables(cached, added, free, table, page, total)            # enough
    _check_tables(cached, added, free[: need // 2], table, page, total + 33)   # the pool runs out, spare slots
    _check_tables(cached, added, free, table, page, total // 2)       # fewer slots than tokens


def test_tables_edges():
    # nobody adds; empty pool; negative counts; more tokens cached than the row is wide
    _check_tables([5, 0, 16], [0, 0, 0], [1, 2], [[4, -1], [-1, -1], [9, -1]], 16, 6)
    _check_tables([5, 0, 16], [30, 1, 1], [], [[4, -1], [-1, -1], [9, -1]], 16, 32)
    _check_tables([-3, 10 ** 6, 16], [4, 5, -7], [1, 2, 3], [[4, -1], [7, 7], [9, -1]], 16, 9)
    # one request whose prompt fills many blocks, over several workgroups
    _check_tables([3], [30000], list(range(2000, 4000)), [[11] + [-1] * 1999], 16, 30001)
    # no request, no slot
    i32 = dict(dtype=torch.int32, device=DEV)
    e, slots = torch.empty(0, **i32), torch.full((5,), 3, dtype=torch.int64, device=DEV)
    lens, starts, slots, taken = mnb.mnb_kv_tables(e, e, e, torch.empty((0, 4), **i32), 16, slots)
    assert lens.numel() == 0 and starts.tolist() == [0] and slots.tolist() == [-1] * 5 and taken.tolist() == [0]
    one = torch.tensor([20], **i32)
    out = mnb.mnb_kv_tables(one, one, one, torch.full((1, 4), 8, **i32), 16, slots[:0])
    assert [x.tolist() for x in out] == [[40], [0, 0], [], [1]]


# ---------------------------------------------------------------------------
# append
# ---------------------------------------------------------------------------

def _cache(blocks, heads, page, dim, dt, order="block-head-token", fill=NAN):
    """A cache of the given memory order, filled with one value."""
    if order == "block-head-token":
        k, v = (torch.full((blocks, heads, page, dim), fill, dtype=TD[dt], device=DEV) for _ in range(2))
    elif order == "block-token-head":
        k, v = (torch.full((blocks, page, heads, dim), fill, dtype=TD[dt], device=DEV).transpose(1, 2)
                for _ in range(2))
    else:   # one tensor holds both, keys and values of a block side by side
        both = torch.full((blocks, 2, heads, page, dim), fill, dtype=TD[dt], device=DEV)
        k, v = both[:, 0], both[:, 1]
    return mnb.KvCache(k, v)


ORDERS = ["block-head-token", "block-token-head", "interleaved"]


@pytest.mark.parametrize("order", ORDERS)
@pytest.mark.parametrize("dt,heads,dim,page,tokens", [("f16", 8, 128, 16, 1), ("f16", 12, 64, 48, 333),
                                                      ("f32", 1, 64, 16, 7), ("f32", 3, 128, 1024, 2100),
                                                      ("f16", 1, 64, 32, 4097)])
def test_append(dt, heads, dim, page, tokens, order):
    print(f"append {dt} heads={heads} dim={dim} page={page} tokens={tokens} {order}", flush=True)
    rng = np.random.default_rng(tokens)
    blocks = tokens // page + 3
    cache = _cache(blocks, heads, page, dim, dt, order, fill=0.25)
    slots = rng.permutation(blocks * page)[:tokens]
    skip = rng.random(tokens) < 0.2
    put = np.where(skip, rng.choice([-1, -10 ** 12, blocks * page, 2 ** 40]), slots)
    # keys and values as columns of one fused buffer, wider than both
    fused = torch.randn((tokens, 2 * heads * dim + 64), device=DEV).to(TD[dt])
    k, v = fused[:, 32: 32 + heads * dim], fused[:, 32 + heads * dim: 32 + 2 * heads * dim]
    mnb.mnb_kv_append(k, v, torch.from_numpy(put).to(DEV), cache)
    torch.cuda.synchronize()
    for t, new in ((cache.k, k), (cache.v, v)):
        ref = np.full((blocks, heads, page, dim), 0.25)
        for i in np.flatnonzero(~skip):
            ref[slots[i] // page, :, slots[i] % page] = _np(new[i]).reshape(heads, dim)
        assert np.array_equal(_np(t), ref)


def test_append_contiguous_rows_of_three_dimensions_and_nothing():
    cache = _cache(2, 2, 16, 64, "f16", fill=0.0)
    k = torch.randn((3, 2, 64), device=DEV).half()
    mnb.mnb_kv_append(k, -k, torch.tensor([31, 0, 5], device=DEV), cache)
    mnb.mnb_kv_append(k[:0], k[:0], torch.empty(0, dtype=torch.int64, device=DEV), cache)
    assert torch.equal(cache.k[1, :, 15], k[0]) and torch.equal(cache.v[0, :, 5], -k[2])
    with pytest.raises(ValueError, match="tokens"):
        mnb.mnb_kv_append(k, k[:2], torch.tensor([1, 2, 3], device=DEV), cache)
    with pytest.raises(ValueError, match="contiguous tokens"):
        mnb.mnb_kv_append(k[:, :1], k, torch.tensor([1, 2, 3], device=DEV), cache)


# ---------------------------------------------------------------------------
# paged attention
# ---------------------------------------------------------------------------

def _paged_case(seed, lens, heads, kv_heads, dim, page, dt, order="block-head-token", spread=1.0):
    """Random keys and values at the valid positions, NaN and infinities in
    every other place of the pool; blocks scattered, unused entries -1."""
    rng = np.random.default_rng(seed)
    width = max(1, max(-(-max(0, n) // page) for n in lens)) + 2
    held = [-(-max(0, n) // page) for n in lens]
    blocks = sum(held) + 3
    cache = _cache(blocks, kv_heads, page, dim, dt, order)
    cache.v[::2] = INF
    cache.k[1::2] = -INF
    ids = rng.permutation(blocks)
    table = np.full((len(lens), width), -1)
    slots, used = [], 0
    for b, n in enumerate(lens):
        table[b, : held[b]] = ids[used: used + held[b]]
        used += held[b]
        slots += [table[b, t // page] * page + t % page for t in range(n)]
    g = torch.Generator(DEV).manual_seed(seed)
    new = [torch.randn((len(slots), kv_heads, dim), device=DEV, generator=g).to(TD[dt]) for _ in range(2)]
    mnb.mnb_kv_append(new[0], new[1], torch.tensor(slots, dtype=torch.int64, device=DEV), cache)
    q = (spread * torch.randn((len(lens), heads, dim), device=DEV, generator=g)).to(TD[dt])
    i32 = dict(dtype=torch.int32, device=DEV)
    return q, cache, torch.tensor(table, **i32), torch.tensor(lens, **i32)


def _check_paged(got, q, cache, table, lens, max_len, dt, scale=None):
    scale = q.shape[-1] ** -0.5 if scale is None else scale
    qn, kn, vn, tn, ln = _np(q), _np(cache.k), _np(cache.v), table.cpu().numpy(), lens.tolist()
    ref = oracle.paged_attention(qn, kn, vn, tn, ln, max_len, scale)
    group = q.shape[1] // cache.kv_heads
    for b in range(q.shape[0]):
        n = min(ln[b], max_len)
        k, v = (oracle.paged_rows(c, tn[b], n, cache.page_size) for c in (kn, vn))
        for h in range(q.shape[1]):
            _near(_np(got[b, h]), ref[b, h], _bound(qn[b, h], k[:, h // group], v[:, h // group], scale, dt),
                  f"request {b} of {n} keys, head {h}")


LENS = [[0], [1], [15, 16, 17], [31, 32, 33, 0, 1], [63, 64, 65, 127], [500, 3, 0, 257, 129], [2049, 1023]]
HEADS = [(16, 8), (12, 12), (8, 1), (40, 2), (1, 1)]


@pytest.mark.parametrize("lens", LENS, ids=lambda x: "-".join(map(str, x)))
@pytest.mark.parametrize("heads,kv_heads", HEADS)
@pytest.mark.parametrize("dim,page,dt", [(128, 16, "f16"), (64, 48, "f16"), (64, 16, "f32"), (128, 64, "f32")])
def test_paged(lens, heads, kv_heads, dim, page, dt):
    print(f"paged {dt} lens={lens} heads={heads}/{kv_heads} dim={dim} page={page}", flush=True)
    q, cache, table, ln = _paged_case(sum(lens) + heads, lens, heads, kv_heads, dim, page, dt)
    got = mnb.mnb_paged_attn(q, cache, table, ln, max(lens))
    _check_paged(got, q, cache, table, ln, max(lens), dt)


@pytest.mark.parametrize("order", ORDERS)
@pytest.mark.parametrize("dt", ["f16", "f32"])
def test_paged_memory_orders_and_strided_queries(order, dt):
    q, cache, table, ln = _paged_case(3, [70, 300, 16], 4, 2, 128, 32, dt, order)
    fused = torch.full((3, 4 * 128 + 2 * 256), NAN, dtype=TD[dt], device=DEV)   # q beside k and v
    fused[:, :512] = q.reshape(3, 512)
    got = mnb.mnb_paged_attn(fused[:, :512].view(3, 4, 128), cache, table, ln, 300)
    _check_paged(got, q, cache, table, ln, 300, dt)


@pytest.mark.parametrize("dt", ["f16", "f32"])
def test_paged_long_caches_split_and_joined(dt):
    for lens, heads, kv_heads, dim in (([20000], 16, 8, 128), ([40001, 7, 9000], 4, 1, 64)):
        print(f"paged {dt} lens={lens} heads={heads}/{kv_heads} dim={dim}", flush=True)
        q, cache, table, ln = _paged_case(9, lens, heads, kv_heads, dim, 64, dt, spread=2.0)
        ws = mnb.paged_attn_workspace(q, cache, max(lens))
        got = []
        for junk in (0xFF, 0x00, 0x7F):      # the workspace's old contents do not matter
            if ws is not None:
                ws.fill_(junk)
            got.append(mnb.mnb_paged_attn(q, cache, table, ln, max(lens), workspace=ws).clone())
        assert torch.equal(got[0], got[1]) and torch.equal(got[0], got[2])
        _check_paged(got[0], q, cache, table, ln, max(lens), dt)


@pytest.mark.parametrize("dt", ["f16", "f32"])
def test_paged_lengths_beside_the_bounds(dt):
    lens = [100, 40, 64, 10]
    q, cache, table, ln = _paged_case(5, lens, 4, 2, 64, 16, dt)
    # a bound below some lengths cuts them
    _check_paged(mnb.mnb_paged_attn(q, cache, table, ln, 50), q, cache, table, ln, 50, dt)
    # a bound far above the lengths changes no more than the split of the sums
    _check_paged(mnb.mnb_paged_attn(q, cache, table, ln, 100000), q, cache, table, ln, 100000, dt)
    # negative lengths are empty; nothing is read past the table's width
    out = mnb.mnb_paged_attn(q, cache, table, ln - 64, 100)
    assert not out[1:].any()
    _check_paged(out, q, cache, table, ln - 64, 100, dt)
    narrow = table[:, :3].contiguous()
    _check_paged(mnb.mnb_paged_attn(q, cache, narrow, ln, 100), q, cache, narrow, ln, 100, dt)
    assert not mnb.mnb_paged_attn(q, cache, table, ln, 0).any()
    assert mnb.mnb_paged_attn(q[:0], cache, table[:0], ln[:0], 100).shape == (0, 4, 64)


@pytest.mark.parametrize("dt", ["f16", "f32"])
def test_paged_missing_blocks_are_left_out(dt):
    q, cache, table, ln = _paged_case(6, [200, 130, 33, 16], 6, 3, 128, 16, dt)
    table[0, 3] = -1
    table[0, 12] = cache.num_blocks
    table[1, 0] = 2 ** 31 - 1
    table[1, 1] = -2 ** 31
    table[2, :] = -5
    got = mnb.mnb_paged_attn(q, cache, table, ln, 200)
    assert not got[2].any()
    _check_paged(got, q, cache, table, ln, 200, dt)


@pytest.mark.parametrize("dt", ["f16", "f32"])
def test_paged_infinities_and_nan_in_valid_places(dt):
    q, cache, table, ln = _paged_case(7, [50, 50, 50, 50], 2, 2, 64, 16, dt)
    q.fill_(1.0)
    page = lambda b, t: (int(table[b, t // 16]), slice(None), t % 16)  # noqa: E731
    for t in range(50):
        cache.k[page(0, t)] = -INF                # every score -infinity: zeros
    cache.k[page(1, 20)] = -INF                   # one key of no weight, whose value is large
    cache.v[page(1, 20)] = 60000.0
    cache.k[page(2, 49)] = NAN                    # a NaN score: NaN
    cache.k[page(3, 4)] = INF                     # infinity less infinity: NaN
    got = mnb.mnb_paged_attn(q, cache, table, ln, 50)
    assert not got[0].any()
    assert torch.isnan(got[2]).all() and torch.isnan(got[3]).all()
    ref = oracle.paged_attention(_np(q), _np(cache.k), _np(cache.v), table.cpu().numpy(), ln.tolist(), 50, 0.125)
    keep = [t for t in range(50) if t != 20]
    for h in range(2):
        k, v = (oracle.paged_rows(_np(c), table[1].tolist(), 50, 16)[keep, h] for c in (cache.k, cache.v))
        _near(_np(got[1, h]), ref[1, h], _bound(_np(q[1, h]), k, v, 0.125, dt))


@pytest.mark.parametrize("dt,top", [("f16", 60000.0), ("f32", 1e30)])
def test_paged_sharp_and_flat_rows(dt, top):
    # one key far above the others anywhere in the row; keys of equal scores
    for at in (0, 31, 32, 299):
        q, cache, table, ln = _paged_case(8, [300], 2, 1, 64, 32, dt)
        cache.k.zero_()
        q.fill_(4.0)
        cache.k[int(table[0, at // 32]), :, at % 32] = 200.0 if dt == "f16" else 1e6
        got = mnb.mnb_paged_attn(q, cache, table, ln, 300)
        assert torch.equal(got[0, 0], cache.v[int(table[0, at // 32]), 0, at % 32])
    cache.k.zero_()
    cache.v.fill_(top)
    got = mnb.mnb_paged_attn(q, cache, table, ln, 300)
    _near(_np(got), np.full(got.shape, top), np.full(got.shape, top * 2 ** -10))


def test_paged_scale_and_lowest_value_keys():
    q, cache, table, ln = _paged_case(10, [90, 64], 4, 4, 64, 16, "f32")
    for scale in (0.0, -0.3, 1.7):
        _check_paged(mnb.mnb_paged_attn(q, cache, table, ln, 90, scale=scale), q, cache, table, ln, 90, "f32", scale)
    q.fill_(1.0)
    low = torch.finfo(torch.float32).min / 64       # scores at the type's lowest value, all of them
    cache.k.fill_(low)
    got = mnb.mnb_paged_attn(q, cache, table, ln, 90, scale=1.0)
    for b, n in enumerate((90, 64)):
        v = oracle.paged_rows(_np(cache.v), table[b].tolist(), n, 16)
        _near(_np(got[b]), v.mean(axis=0), np.abs(v).mean(axis=0) * 2 ** -16)


def test_paged_offsets_past_32_bits():
    # blocks whose byte offset, and whose element offset, pass 2^32
    dim, page, blocks = 128, 1024, 36000
    k = torch.empty((blocks, 1, page, dim), dtype=torch.float16, device=DEV)
    cache = mnb.KvCache(k, k.clone())
    ids = [35999, 0, 17000, 33000]
    assert ids[0] * page * dim > 2 ** 32
    g = torch.Generator(DEV).manual_seed(1)
    table = torch.tensor([ids], dtype=torch.int32, device=DEV)
    new = [torch.randn((3500, 1, dim), device=DEV, generator=g).half() for _ in range(2)]
    slots = torch.tensor([ids[t // page] * page + t % page for t in range(3500)], device=DEV)
    mnb.mnb_kv_append(new[0], new[1], slots, cache)
    q = torch.randn((1, 2, dim), device=DEV, generator=g).half()
    got = mnb.mnb_paged_attn(q, cache, table, torch.tensor([3500], dtype=torch.int32, device=DEV), 4096)
    kn, vn = _np(new[0][:, 0]), _np(new[1][:, 0])
    for h in range(2):
        x = _np(q[0, h])
        _near(_np(got[0, h]), oracle.attend(x, kn, vn, dim ** -0.5), _bound(x, kn, vn, dim ** -0.5, "f16"))


# ---------------------------------------------------------------------------
# cross attention
# ---------------------------------------------------------------------------

def _check_cross(got, q, k, v, lens, dt, scale=None, rows=None):
    scale = q.shape[-1] ** -0.5 if scale is None else scale
    qn, kn, vn = _np(q), _np(k), _np(v)
    group = q.shape[2] // k.shape[2]
    got = _np(got)
    for b in range(q.shape[0]):
        n = k.shape[1] if lens is None else max(0, min(lens[b], k.shape[1]))
        for t in range(q.shape[1]) if rows is None else rows:
            for h in range(q.shape[2]):
                x, kk, vv = qn[b, t, h], kn[b, :n, h // group], vn[b, :n, h // group]
                _near(got[b, t, h], oracle.attend(x, kk, vv, scale), _bound(x, kk, vv, scale, dt),
                      f"request {b}, row {t}, head {h}, {n} keys")


def _cross_case(seed, batch, queries, keys, heads, kv_heads, dim, dt):
    g = torch.Generator(DEV).manual_seed(seed)
    make = lambda *s: torch.randn(s, device=DEV, generator=g).to(TD[dt])  # noqa: E731
    return make(batch, queries, heads, dim), make(batch, keys, kv_heads, dim), make(batch, keys, kv_heads, dim)


@pytest.mark.parametrize("queries,keys", [(1, 1), (1, 1500), (3, 33), (4, 100), (16, 16), (17, 65), (33, 31), (62, 200),
                                          (130, 129), (5, 0)])
@pytest.mark.parametrize("heads,kv_heads,dim", [(12, 12, 64), (4, 2, 128), (6, 1, 64)])
@pytest.mark.parametrize("dt", ["f16", "f32"])
def test_cross(queries, keys, heads, kv_heads, dim, dt):
    print(f"cross {dt} queries={queries} keys={keys} heads={heads}/{kv_heads} dim={dim}", flush=True)
    q, k, v = _cross_case(queries + keys, 2, queries, keys, heads, kv_heads, dim, dt)
    rows = None if queries < 20 else sorted({0, 1, 15, 16, 17, queries // 2, queries - 2, queries - 1})
    got = mnb.mnb_cross_attn(q, k, v)
    _check_cross(got, q, k, v, None, dt, rows=rows)
    if keys:    # lengths, and whatever stands past them
        lens = [keys // 2, keys]
        k[0, lens[0]:], v[0, lens[0]:] = NAN, INF
        got = mnb.mnb_cross_attn(q, k, v, torch.tensor(lens, dtype=torch.int32, device=DEV))
        _check_cross(got, q, k, v, lens, dt, rows=rows)


@pytest.mark.parametrize("queries", [1, 3, 70])
@pytest.mark.parametrize("dt", ["f16", "f32"])
def test_cross_lengths(queries, dt):
    lens = [0, 1, -4, 31, 32, 33, 64, 150, 151, 10 ** 6]
    q, k, v = _cross_case(4, len(lens), queries, 151, 2, 2, 64, dt)
    for b, n in enumerate(lens):
        k[b, max(0, n):] = NAN
        v[b, max(0, n):] = -INF
    got = mnb.mnb_cross_attn(q, k, v, torch.tensor(lens, dtype=torch.int32, device=DEV))
    assert not got[0].any() and not got[2].any()
    _check_cross(got, q, k, v, lens, dt, rows=sorted({0, queries // 2, queries - 1}))


@pytest.mark.parametrize("queries", [2, 90])
@pytest.mark.parametrize("dt", ["f16", "f32"])
def test_cross_strides(queries, dt):
    heads, dim, keys = 4, 64, 77
    q, k, v = _cross_case(5, 3, queries, keys, heads, heads, dim, dt)
    ref = mnb.mnb_cross_attn(q, k, v)
    # head-major keys, values inside a fused buffer, queries and outputs with gaps
    kk = k.transpose(1, 2).contiguous().transpose(1, 2)
    fused = torch.full((3, keys, 2, heads, dim), NAN, dtype=TD[dt], device=DEV)
    fused[:, :, 1] = v
    wide = torch.full((3, queries, heads, 3 * dim), NAN, dtype=TD[dt], device=DEV)
    wide[..., dim: 2 * dim] = q
    out = torch.full((3, heads, queries, 2 * dim), 7.0, dtype=TD[dt], device=DEV)
    got = mnb.mnb_cross_attn(wide[..., dim: 2 * dim], kk, fused[:, :, 1], out=out[..., :dim].transpose(1, 2))
    assert torch.equal(got, ref)
    assert (out[..., dim:] == 7.0).all()
    # one encoder's states shared by the requests (beams)
    shared = mnb.mnb_cross_attn(q, k[:1].expand(3, -1, -1, -1), v[:1].expand(3, -1, -1, -1))
    assert torch.equal(shared[0], ref[0])
    _check_cross(shared, q, k[:1].expand(3, -1, -1, -1), v[:1].expand(3, -1, -1, -1), None, dt, rows=[0, queries - 1])


@pytest.mark.parametrize("dt", ["f16", "f32"])
def test_cross_infinities_and_nan_in_valid_places(dt):
    for queries in (1, 80):
        q, k, v = _cross_case(6, 3, queries, 90, 2, 2, 64, dt)
        q.fill_(1.0)
        k[0], k[1, 89], k[2, 3] = -INF, NAN, INF
        got = mnb.mnb_cross_attn(q, k, v)
        assert not got[0].any()
        assert torch.isnan(got[1]).all() and torch.isnan(got[2]).all()


@pytest.mark.parametrize("queries", [1, 64])
def test_cross_growing_scores(queries):
    # scores that rise along the keys by more than a float16 exponent range
    q, k, v = _cross_case(7, 1, queries, 600, 1, 1, 64, "f16")
    q.fill_(0.5)
    k[0, :, 0] = (torch.arange(600, device=DEV).float()[:, None] * 0.05 - 15).half().unsqueeze(1)[:, 0, :].repeat(1, 64)
    got = mnb.mnb_cross_attn(q, k, v, scale=1.0)
    _check_cross(got, q, k, v, None, "f16", 1.0, rows=[0, queries - 1])


# ---------------------------------------------------------------------------
# streams, graphs, refusals
# ---------------------------------------------------------------------------

def test_streams_and_graph_replays():
    q, cache, table, ln = _paged_case(11, [5000, 40, 1300], 16, 8, 128, 16, "f16")
    cq, ck, cv = _cross_case(12, 3, 2, 1500, 12, 12, 64, "f16")
    ws, cws = mnb.paged_attn_workspace(q, cache, 5000), mnb.cross_attn_workspace(cq, ck)
    i32 = dict(dtype=torch.int32, device=DEV)
    added, free = torch.ones(3, **i32), torch.tensor([1, 2, 0], **i32)
    grown, slots = torch.cat([table, torch.full((3, 1), -1, **i32)], 1), torch.empty(3, dtype=torch.int64, device=DEV)
    lens, starts, taken = torch.empty(3, **i32), torch.empty(4, **i32), torch.empty(1, **i32)
    out, cout = torch.empty_like(q), torch.empty_like(cq)

    def step():
        mnb.mnb_kv_tables(ln, added, free, grown, 16, slots, lens=lens, starts=starts, taken=taken)
        mnb.mnb_paged_attn(q, cache, table, ln, 5000, workspace=ws, out=out)
        mnb.mnb_cross_attn(cq, ck, cv, workspace=cws, out=cout)

    step()
    torch.cuda.synchronize()
    ref = [x.clone() for x in (out, cout, slots, lens, grown)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        out.fill_(NAN), cout.fill_(NAN), slots.fill_(0)
        step()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(ref, (out, cout, slots, lens, grown)))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(4):
        out.fill_(NAN), cout.fill_(NAN), slots.fill_(0)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(ref, (out, cout, slots, lens, grown))), i
        step()          # eager work between the replays
        torch.cuda.synchronize()


def test_binding_refusals():
    q, cache, table, ln = _paged_case(13, [40], 4, 2, 64, 16, "f16")
    bad = [(ValueError, "must be torch.float16", lambda: mnb.mnb_paged_attn(q.float(), cache, table, ln, 40)),
           (ValueError, "q must be", lambda: mnb.mnb_paged_attn(q[..., :32].contiguous(), cache, table, ln, 40)),
           (ValueError, "contiguous requests", lambda: mnb.mnb_paged_attn(
               torch.cat([q, q], 2)[..., :64], cache, table, ln, 40)),
           (ValueError, "must be torch.int32", lambda: mnb.mnb_paged_attn(q, cache, table.long(), ln, 40)),
           (ValueError, "elements", lambda: mnb.mnb_paged_attn(q, cache, table, torch.cat([ln, ln]), 40)),
           (ValueError, "is on", lambda: mnb.mnb_paged_attn(q.cpu(), cache, table, ln, 40)),
           (ValueError, "elements", lambda: mnb.mnb_paged_attn(q, cache, table, ln, 40, out=q[:, :3].contiguous())),
           (mnb.MnbError, "SHAPE", lambda: mnb.mnb_paged_attn(q[:, :3].contiguous(), cache, table, ln, 40)),
           (mnb.MnbError, "SHAPE", lambda: mnb.mnb_paged_attn(q, cache, table, ln, -1)),
           (mnb.MnbError, "INVALID", lambda: mnb.mnb_paged_attn(q, cache, table, ln, 40, scale=NAN)),
           (ValueError, "same shape and strides", lambda: mnb.KvCache(cache.k, cache.v[:-1]))]
    cq, ck, cv = _cross_case(1, 2, 3, 20, 4, 2, 64, "f32")
    bad += [(ValueError, "must be torch.float32", lambda: mnb.mnb_cross_attn(cq, ck.half(), cv)),
            (ValueError, "k and v must be", lambda: mnb.mnb_cross_attn(cq, ck, cv[:, :19])),
            (ValueError, "k and v must be", lambda: mnb.mnb_cross_attn(cq, ck[:1], cv[:1])),
            (ValueError, "contiguous", lambda: mnb.mnb_cross_attn(cq, ck.transpose(1, 3), cv.transpose(1, 3))),
            (ValueError, "q's shape", lambda: mnb.mnb_cross_attn(cq, ck, cv, out=cq[:, :2])),
            (ValueError, "elements", lambda: mnb.mnb_cross_attn(cq, ck, cv, ln)),
            (mnb.MnbError, "SHAPE", lambda: mnb.mnb_cross_attn(cq[:, :, :3].contiguous(), ck, cv)),
            (mnb.MnbError, "SHAPE", lambda: mnb.mnb_cross_attn(
                *(t[..., :32].contiguous() for t in (cq, ck, cv)))),
            (mnb.MnbError, "ALIGN", lambda: mnb.mnb_cross_attn(
                torch.zeros(2, 3, 4, 66, device=DEV)[..., :64], ck, cv))]
    out = torch.full_like(q, 3.0)
    for kind, text, call in bad:
        with pytest.raises(kind, match=text):
            call()
    torch.cuda.synchronize()
    assert (out == 3.0).all()
    # a workspace that is too small is refused, whatever the split
    long_q, long_cache, long_table, long_ln = _paged_case(14, [9000], 2, 2, 64, 64, "f16")
    need = mnb.mnb_paged_attn_workspace_bytes(1, 2, long_cache, 9000)
    if need:
        small = torch.empty(need - 1, dtype=torch.uint8, device=DEV)
        with pytest.raises(mnb.MnbError, match="INVALID"):
            mnb.mnb_paged_attn(long_q, long_cache, long_table, long_ln, 9000, workspace=small)


# ---------------------------------------------------------------------------
# cross attention with many rows (float16: the kernel whose tiles go through
# LDS), in both of its forms
# ---------------------------------------------------------------------------

MANY = [  # batch, queries, keys, heads, kv_heads, dim
    (24, 130, 200, 4, 2, 64), (24, 130, 257, 4, 2, 64), (24, 100, 333, 6, 2, 128), (13, 70, 100, 3, 3, 128),
    (64, 17, 31, 4, 4, 64), (64, 17, 65, 4, 4, 128), (40, 64, 32, 2, 1, 64), (40, 65, 33, 5, 5, 128),
    (100, 9, 96, 8, 2, 64), (200, 20, 1, 1, 1, 64),
]


def _many_rows(queries):
    return sorted({0, queries // 3, queries - 1})


@pytest.mark.parametrize("batch,queries,keys,heads,kv_heads,dim", MANY)
def test_cross_many(batch, queries, keys, heads, kv_heads, dim):
    print(f"cross many {batch}x{queries}x{keys} heads={heads}/{kv_heads} dim={dim}", flush=True)
    q, k, v = _cross_case(batch + keys, batch, queries, keys, heads, kv_heads, dim, "f16")
    got = mnb.mnb_cross_attn(q, k, v)
    pick = [0, batch // 2, batch - 1]
    _check_cross(got[pick], q[pick], k[pick], v[pick], None, "f16", rows=_many_rows(queries))
    # every length around the steps of 32 and 64 keys, garbage past it
    lens = [[keys, 0, 1, 31, 32, 33, 63, 64, 65, 95, 96, 97, 128, 129, -5, 10 ** 6][b % 16] for b in range(batch)]
    for b, n in enumerate(lens):
        k[b, max(0, n):], v[b, max(0, n):] = NAN, (INF if b % 2 else NAN)
    got = mnb.mnb_cross_attn(q, k, v, torch.tensor(lens, dtype=torch.int32, device=DEV))
    empty = [b for b, n in enumerate(lens) if n <= 0]
    assert not got[empty].any()
    pick = list(range(min(16, batch)))
    _check_cross(got[pick], q[pick], k[pick], v[pick], [lens[b] for b in pick], "f16", rows=_many_rows(queries))
    again = mnb.mnb_cross_attn(q, k, v, torch.tensor(lens, dtype=torch.int32, device=DEV))
    assert torch.equal(got, again)


@pytest.mark.parametrize("dim", [64, 128])
def test_cross_many_strides(dim):
    batch, queries, keys, heads = 40, 70, 77, 4
    q, k, v = _cross_case(15, batch, queries, keys, heads, heads, dim, "f16")
    ref = mnb.mnb_cross_attn(q, k, v)
    kk = k.transpose(1, 2).contiguous().transpose(1, 2)
    fused = torch.full((batch, keys, 2, heads, dim), NAN, dtype=torch.float16, device=DEV)
    fused[:, :, 1] = v
    wide = torch.full((batch, queries, heads, 3 * dim), NAN, dtype=torch.float16, device=DEV)
    wide[..., dim: 2 * dim] = q
    out = torch.full((batch, heads, queries, 2 * dim), 7.0, dtype=torch.float16, device=DEV)
    got = mnb.mnb_cross_attn(wide[..., dim: 2 * dim], kk, fused[:, :, 1], out=out[..., :dim].transpose(1, 2))
    assert torch.equal(got, ref)
    assert (out[..., dim:] == 7.0).all()
    shared = mnb.mnb_cross_attn(q, k[:1].expand(batch, -1, -1, -1), v[:1].expand(batch, -1, -1, -1))
    assert torch.equal(shared[0], ref[0])
    _check_cross(shared[-1:], q[-1:], k[:1], v[:1], None, "f16", rows=[0, 69])


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("keys", [90, 300])
def test_cross_many_scales_infinities_and_nan(keys, dim):
    batch, queries, heads = 40, 80, 4
    q, k, v = _cross_case(16, batch, queries, keys, heads, heads, dim, "f16")
    for scale in (0.0, -0.21, 0.9):
        got = mnb.mnb_cross_attn(q, k, v, scale=scale)
        _check_cross(got[:2], q[:2], k[:2], v[:2], None, "f16", scale, rows=[0, 63, 64, 79])
    # scores that rise along the keys by far more than the reference's slack
    q[0] = 0.5
    k[0] = (torch.arange(keys, device=DEV) * (30.0 / keys) - 15).half()[:, None, None]
    q[1:4] = 1.0
    k[1], k[2, keys - 1], k[3, 3] = -INF, NAN, INF
    got = mnb.mnb_cross_attn(q, k, v, scale=1.0)
    _check_cross(got[:1], q[:1], k[:1], v[:1], None, "f16", 1.0, rows=[0, 79])
    assert not got[1].any()
    assert torch.isnan(got[2]).all() and torch.isnan(got[3]).all()
    assert torch.isfinite(got[4:]).all()


def test_cross_many_rows_too_far_apart_for_32_bits():
    # keys 2^25 elements apart: the LDS kernel's 32-bit range does not reach
    batch, queries, keys, dim = 2, 3000, 40, 64
    buf = torch.zeros((keys - 1) * 2 ** 25 + 4 * dim, dtype=torch.float16, device=DEV)
    k = buf.as_strided((batch, keys, 1, dim), (dim, 2 ** 25, dim, 1))
    v = buf.as_strided((batch, keys, 1, dim), (dim, 2 ** 25, dim, 1), 2 * dim)
    g = torch.Generator(DEV).manual_seed(3)
    q = torch.randn((batch, queries, 1, dim), device=DEV, generator=g).half()
    k.copy_(torch.randn(k.shape, device=DEV, generator=g))
    v.copy_(torch.randn(v.shape, device=DEV, generator=g))
    got = mnb.mnb_cross_attn(q, k, v)
    _check_cross(got, q, k, v, None, "f16", rows=[0, 1500, 2999])


# ---------------------------------------------------------------------------
# rows that are cut, and the same rows whole where there are enough of them


@pytest.mark.parametrize("dim,page,dt,longest", [(128, 16, "f16", 1100), (64, 32, "f32", 1100), (64, 16, "f16", 2100)])
def test_paged_rows_cut_or_whole(dim, page, dt, longest):
    for requests in (23, 24):       # 184 and 192 rows of keys
        lens = [longest] + [(5 * b) % 37 for b in range(requests - 2)] + [longest - 1]
        print(f"paged {dt} dim={dim} {requests} requests, longest {longest}", flush=True)
        q, cache, table, ln = _paged_case(requests, lens, 8, 8, dim, page, dt)
        cut = mnb.mnb_paged_attn_workspace_bytes(requests, 8, cache, longest) > 0
        assert cut == (requests == 23)
        got = mnb.mnb_paged_attn(q, cache, table, ln, longest)
        _check_paged(got, q, cache, table, ln, longest, dt)


@pytest.mark.parametrize("queries", [1, 40])
@pytest.mark.parametrize("dt", ["f16", "f32"])
def test_cross_rows_that_overlap_in_memory(dt, queries):
    # rows 32 elements apart: the row after the last valid one shares half its
    # elements, a NaN among them that only dimension 42 may see
    batch, heads, rows, n = 8, 12, 20, 5
    gen = torch.Generator().manual_seed(3)
    values = torch.randn((batch, heads, 32 * (rows + 1)), generator=gen).to(TD[dt])
    values[:, :, 32 * (n - 1) + 42] = NAN
    values = values.to(DEV)
    v = values.as_strided((batch, rows, heads, 64), (heads * 32 * (rows + 1), 32, 32 * (rows + 1), 1))
    k = torch.randn((batch, rows, heads, 64), generator=gen).to(TD[dt]).to(DEV)
    q = torch.randn((batch, queries, heads, 64), generator=gen).to(TD[dt]).to(DEV)
    got = mnb.mnb_cross_attn(q, k, v, torch.full((batch,), n, dtype=torch.int32, device=DEV))
    nan = torch.isnan(got)
    assert nan[..., 42].all() and not nan[..., :42].any() and not nan[..., 43:].any()


# ---------------------------------------------------------------------------
# shapes of more row tiles, for the forms that only many of them take

MORE = [(70, 70, 100, 3, 3, 128), (100, 64, 32, 2, 1, 64), (600, 20, 1, 1, 1, 64), (2, 1100, 300, 4, 4, 128),
        (2, 1100, 129, 4, 4, 64), (64, 140, 70, 8, 8, 64)]


@pytest.mark.parametrize("batch,queries,keys,heads,kv_heads,dim", MORE)
def test_cross_more(batch, queries, keys, heads, kv_heads, dim):
    test_cross_many(batch, queries, keys, heads, kv_heads, dim)


def test_cross_more_rows_too_far_apart_for_32_bits():
    batch, queries, keys, dim = 2, 5000, 40, 64
    buf = torch.zeros((keys - 1) * 2 ** 25 + 4 * dim, dtype=torch.float16, device=DEV)
    k = buf.as_strided((batch, keys, 1, dim), (dim, 2 ** 25, dim, 1))
    v = buf.as_strided((batch, keys, 1, dim), (dim, 2 ** 25, dim, 1), 2 * dim)
    g = torch.Generator(DEV).manual_seed(3)
    q = torch.randn((batch, queries, 1, dim), device=DEV, generator=g).half()
    k.copy_(torch.randn(k.shape, device=DEV, generator=g))
    v.copy_(torch.randn(v.shape, device=DEV, generator=g))
    got = mnb.mnb_cross_attn(q, k, v)
    _check_cross(got, q, k, v, None, "f16", rows=[0, 2500, 4999])


def test_cross_more_rows_that_overlap_in_memory():
    test_cross_rows_that_overlap_in_memory("f16", 100)


@pytest.mark.parametrize("batch", [2047, 2048, 2049, 4100])
def test_tables_of_many_requests(batch):
    page, width = 16, 3
    rng = np.random.RandomState(batch)
    cached, added = rng.randint(-1, page * width + 2, batch), rng.randint(-1, 4, batch)
    free = rng.permutation(3 * batch)[:batch].astype(np.int32)      # too few for all
    table = rng.randint(-1, 50, (batch, width)).astype(np.int32)
    tokens = int(np.maximum(added, 0).sum()) + 3
    want = oracle.kv_tables(cached.tolist(), added.tolist(), free.tolist(), table, page, tokens)
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(DEV)
    got_table, slots = dev(table), torch.full((tokens,), 9, dtype=torch.int64, device=DEV)
    lens, starts, slots, taken = mnb.mnb_kv_tables(dev(cached), dev(added), dev(free), got_table, page, slots)
    for got, ref in zip((got_table, lens, starts, slots), want):
        assert np.array_equal(got.cpu().numpy(), ref)
    assert int(taken) == want[4]


@pytest.mark.parametrize("heads,dim,dt", [(1, 64, "f16"), (3, 64, "f16"), (1, 128, "f32"), (5, 64, "f32"), (16, 64, "f16"),
                                          (17, 64, "f16")])
@pytest.mark.parametrize("tokens", [1, 3, 77])
def test_append_of_narrow_tokens(heads, dim, dt, tokens):
    # several tokens a workgroup: two tokens' and one token's worth of threads,
    # tokens that do not fill the last one, slots that are left out
    page, blocks = 16, 7
    gen = torch.Generator().manual_seed(tokens)
    k, v = (torch.randn((tokens, heads, dim), generator=gen).to(TD[dt]).to(DEV) for _ in range(2))
    cache = mnb.KvCache(*(torch.full((blocks, heads, page, dim), 5.0, dtype=TD[dt], device=DEV) for _ in range(2)))
    slots = torch.randperm(blocks * page, generator=gen)[:tokens].long()
    slots[tokens // 2] = [-1, blocks * page, 1 << 40][heads % 3]
    mnb.mnb_kv_append(k, v, slots.to(DEV), cache)
    for new, got in ((k, cache.k), (v, cache.v)):
        want = torch.full((blocks, heads, page, dim), 5.0, dtype=TD[dt])
        for t, slot in enumerate(slots.tolist()):
            if 0 <= slot < blocks * page:
                want[slot // page, :, slot % page] = new[t].cpu()
        assert torch.equal(got.cpu(), want)


@pytest.mark.parametrize("requests,longest", [(101, 2000), (37, 4000)])
def test_paged_row_tiles_of_large_caches(requests, longest):
    # two row tiles a head, ordered by their keys: 202 rows of keys whole, 74 cut
    lens = [longest // 3, 0, 1, 700, 385] + [(7 * b) % 60 for b in range(requests - 5)]
    print(f"paged f16 {requests} requests, bound {longest}", flush=True)
    q, cache, table, ln = _paged_case(requests, lens, 40, 2, 128, 16, "f16")
    assert (mnb.mnb_paged_attn_workspace_bytes(requests, 40, cache, longest) > 0) == (requests == 37)
    got = mnb.mnb_paged_attn(q, cache, table, ln, longest)
    _check_paged(got, q, cache, table, ln, longest, "f16")


@pytest.mark.parametrize("dt,heads,queries", [("f32", 12, 40), ("f32", 3, 50)])
def test_cross_row_tiles_of_large_states(dt, heads, queries):
    # one encoder's states for all requests: their sizes alone order the tiles
    batch, keys, dim = 67, 1500, 64
    q, k, v = _cross_case(4, batch, queries, keys, heads, heads, dim, dt)
    k, v = k[:1].expand(batch, -1, -1, -1), v[:1].expand(batch, -1, -1, -1)
    lens = [(11 * b) % 71 for b in range(batch)]
    got = mnb.mnb_cross_attn(q, k, v, torch.tensor(lens, dtype=torch.int32, device=DEV))
    pick = [0, 1, 33, 65, 66]
    _check_cross(got[pick], q[pick], k[pick], v[pick], [lens[b] for b in pick], dt, rows=[0, 15, 16, queries - 1])


@pytest.mark.parametrize("dt", ["f16", "f32"])
@pytest.mark.parametrize("shared", [False, True])
def test_cross_one_token_of_large_states(dt, shared):
    # states past 32 MB (read past the caches, unless the requests share them)
    batch, heads, keys, dim = 30, 6, 1500, 64
    q, k, v = _cross_case(6, batch, 1, keys, heads, heads, dim, dt)
    if shared:
        k, v = k[:1].expand(batch, -1, -1, -1), v[:1].expand(batch, -1, -1, -1)
    lens = [(131 * b) % 1700 - 50 for b in range(batch)]
    got = mnb.mnb_cross_attn(q, k, v, torch.tensor(lens, dtype=torch.int32, device=DEV))
    pick = [0, 1, 7, 14, 29]
    _check_cross(got[pick], q[pick], k[pick], v[pick], [lens[b] for b in pick], dt, rows=[0])


@pytest.mark.parametrize("dim,dt,longest", [(64, "f16", 31), (64, "f16", 32), (128, "f16", 64), (64, "f32", 40), (128, "f32", 47)])
def test_paged_many_short_rows(dim, dt, longest):
    # more workgroups than the card holds, of fewer waves than usual
    requests, heads = 500, 4
    lens = [(b * 7) % (longest + 1) for b in range(requests)]
    q, cache, table, ln = _paged_case(longest, lens, heads, 2, dim, 16, dt)
    got = mnb.mnb_paged_attn(q, cache, table, ln, longest)
    pick = list(range(0, requests, 9))
    _check_paged(got[pick], q[pick], cache, table[pick], ln[pick], longest, dt)
