"""GPU: the 8-bit key-value cache and the attention over it, against the float64
oracle.

Codes, scales and what is read back are compared exactly. Attention outputs are
compared within a bound worked out per output from the inputs (`_bound`): the
oracle takes the stored codes and scales as they are; with u = 2^-24, n keys
seen, S = max_t sum_i |scale q_i k_ti|, Q = max_t |scale| amax|q| sum_i |k_ti|
and A = sum p |v| / sum p,

  a query may be held as whole numbers of 22 bits and a sign, relative to its
  largest: off by half a step, 2^-22 amax, which moves a score by 4 u Q;
  a score is a float32 sum of up to D terms, scaled twice: off by (D + 4) u S;
  its difference from the maximum, times log2(e): 4 u S more;
  so a weight is off by 2 ((D + 8) u S + 4 u Q) relative, plus 2^-21 for the
  exponential and the joining factors, in the numerator and the denominator;
  weights times value scales may be held as whole numbers of 21 bits, relative
  to the largest M = max_t p_t vs_t: off by 2^-21 M each, on codes |cv|;
  sums of n terms in any order, n u each, plus 64 u for the joins;

float16 adds the weights' rounding to float16 (2^-11 relative, at most 2^-25
absolute against a largest weight of at least 1, in the numerator and the
denominator) and the output's (2^-11 relative, 2^-25 absolute); float32 the
output's 2^-24.
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
ORDERS = ["block-head-token", "block-token-head", "interleaved"]


def _np(t):
    return t.cpu().double().numpy()


def _bound(q, k, v, vs, scale, dt):
    """Per-output bound of one query row q [D] over the rows k, v [n, D] it sees."""
    n, dim = k.shape
    if n == 0:
        return np.zeros(v.shape[1])
    u = 2.0 ** -24
    s_abs = (np.abs(k * q).sum(axis=1) * abs(scale)).max()
    q_abs = (np.abs(k).sum(axis=1) * abs(scale) * np.abs(q).max()).max()
    score = (k * q).sum(axis=1) * scale
    p = np.exp(score - score.max())
    a = (p[:, None] * np.abs(v)).sum(axis=0) / p.sum()
    y = np.abs((p[:, None] * v).sum(axis=0)) / p.sum()
    code = np.abs(v) / np.where(vs > 0, vs, 1.0)[:, None]
    tol = a * 2 * (2 * ((dim + 8) * u * s_abs + 4 * u * q_abs) + 2.0 ** -21 + (n + 64) * u) + 1e-30
    tol += 2.0 ** -21 * (p * vs).max() * code.sum(axis=0) / p.sum() + y * u
    if dt == "f16":
        tol += a * 2 * 2.0 ** -11 + n * 2.0 ** -25 * np.abs(v).max() + y * 2.0 ** -11 + 2.0 ** -25
    return tol


def _near(got, ref, tol, what=""):
    worst = np.max(np.abs(got - ref) / np.maximum(tol, 1e-300), initial=0.0)
    assert np.all(np.isfinite(got)) and worst <= 1.0, f"{what}: {worst:.3f} of the bound"


def _cache(blocks, heads, page, dim, dt, order="block-head-token", code=0, scale=NAN):
    """A cache of the given memory order, filled with one code and one scale."""
    def codes(*shape):
        return torch.full(shape, code, dtype=torch.int8, device=DEV)

    def scales(*shape):
        return torch.full(shape, scale, dtype=torch.float32, device=DEV)
    if order == "block-head-token":
        k, v = codes(blocks, heads, page, dim), codes(blocks, heads, page, dim)
        ks, vs = scales(blocks, heads, page), scales(blocks, heads, page)
    elif order == "block-token-head":
        k, v = (codes(blocks, page, heads, dim).transpose(1, 2) for _ in range(2))
        ks, vs = (scales(heads, blocks, page).transpose(0, 1) for _ in range(2))
    else:   # keys and values of a block side by side
        both, two = codes(blocks, 2, heads, page, dim), scales(blocks, 2, heads, page)
        k, v, ks, vs = both[:, 0], both[:, 1], two[:, 0], two[:, 1]
    return mnb.KvCacheI8(k, v, ks, vs, TD[dt])


# ---------------------------------------------------------------------------
# append and read
# ---------------------------------------------------------------------------

def _rows(dt, shape, seed):
    """Rows of all sizes: ordinary ones, tiny and huge ones, zeros, codes on the
    border between two."""
    g = torch.Generator(DEV).manual_seed(seed)
    x = torch.randn(shape, device=DEV, generator=g)
    size = torch.randn((*shape[:-1], 1), device=DEV, generator=g) * (3 if dt == "f16" else 20)
    x = x * torch.exp(size)
    flat = x.view(-1, shape[-1])
    flat[0] = 0.0
    if len(flat) > 1:
        flat[1] = torch.arange(shape[-1], device=DEV) - (shape[-1] - 0.5)
        flat[1, 0] = 63.5
    if len(flat) > 2:
        flat[2] = 6e-8 if dt == "f16" else 3e-45
    return x.clamp(-60000, 60000).to(TD[dt]) if dt == "f16" else x


@pytest.mark.parametrize("order", ORDERS)
@pytest.mark.parametrize("dt,heads,dim,page,tokens", [("f16", 8, 128, 16, 1), ("f16", 12, 64, 48, 333),
                                                      ("f32", 1, 64, 16, 7), ("f32", 3, 128, 1024, 2100),
                                                      ("f16", 1, 64, 32, 4097), ("f32", 5, 128, 16, 1001)])
def test_append_and_read(dt, heads, dim, page, tokens, order):
    print(f"append8 {dt} heads={heads} dim={dim} page={page} tokens={tokens} {order}", flush=True)
    rng = np.random.default_rng(tokens)
    blocks = tokens // page + 3
    cache = _cache(blocks, heads, page, dim, dt, order, code=5, scale=0.25)
    slots = rng.permutation(blocks * page)[:tokens]
    skip = rng.random(tokens) < (0.2 if tokens > 1 else 0.0)
    put = np.where(skip, rng.choice([-1, -10 ** 12, blocks * page, 2 ** 40]), slots)
    # keys and values as columns of one fused buffer, wider than both
    fused = torch.zeros((tokens, 2 * heads * dim + 64), dtype=TD[dt], device=DEV)
    k, v = fused[:, 32: 32 + heads * dim], fused[:, 32 + heads * dim: 32 + 2 * heads * dim]
    k.copy_(_rows(dt, (tokens, heads, dim), 1).view(tokens, -1))
    v.copy_(_rows(dt, (tokens, heads, dim), 2).view(tokens, -1))
    put_d = torch.from_numpy(put).to(DEV)
    mnb.mnb_kv_append_i8(k, v, put_d, cache)
    back = mnb.mnb_kv_read_i8(put_d, cache)
    torch.cuda.synchronize()
    for codes, scales, new, got in ((cache.k, cache.k_scale, k, back[0]), (cache.v, cache.v_scale, v, back[1])):
        want_c, want_s = oracle.quantize_rows(_np(new).reshape(tokens, heads, dim))
        ref_c = np.full((blocks, heads, page, dim), 5, dtype=np.int8)
        ref_s = np.full((blocks, heads, page), 0.25, dtype=np.float32)
        ref_c[slots[~skip] // page, :, slots[~skip] % page] = want_c[~skip]
        ref_s[slots[~skip] // page, :, slots[~skip] % page] = want_s[~skip]
        assert np.array_equal(scales.cpu().numpy(), ref_s)
        assert np.array_equal(codes.cpu().numpy(), ref_c)
        exact = want_c.astype(np.float64) * want_s.astype(np.float64)[..., None]
        exact[skip] = 0.0
        assert np.array_equal(got.cpu().numpy(), exact.astype(np.float16 if dt == "f16" else np.float32))


@pytest.mark.parametrize("dt", ["f16", "f32"])
def test_codes_next_to_their_borders(dt):
    # every multiple of half a step, and the numbers beside it
    amax = torch.tensor([127.0, 1.0, 0.37, 100.0, 3.0, 65504.0 if dt == "f16" else 3.4e38], device=DEV).to(TD[dt])
    rows = []
    for a in amax:
        half = (torch.arange(-127, 128, device=DEV).double() + 0.5) * (a.double() / 127)
        x = half.to(TD[dt])
        for y in (x, torch.nextafter(x, x + 1), torch.nextafter(x, x - 1)):
            rows.append(torch.cat((y.clamp(-a, a)[:255], a[None])).view(2, 128))
            rows[-1][0, 0] = a
    x = torch.cat(rows)[:, None].contiguous()
    tokens = x.shape[0]
    cache = _cache(tokens // 16 + 1, 1, 16, 128, dt)
    slots = torch.arange(tokens, device=DEV)
    mnb.mnb_kv_append_i8(x, -x, slots, cache)
    for codes, scales, new in ((cache.k, cache.k_scale, x), (cache.v, cache.v_scale, -x)):
        want_c, want_s = oracle.quantize_rows(_np(new)[:, 0])
        assert np.array_equal(scales.cpu().numpy().reshape(-1)[:tokens], want_s)
        assert np.array_equal(codes.cpu().numpy().reshape(-1, 128)[:tokens], want_c)


@pytest.mark.parametrize("dt", ["f16", "f32"])
def test_rows_that_are_not_finite_stand_for_nan(dt):
    cache = _cache(2, 2, 16, 64, dt, code=1, scale=1.0)
    x = torch.ones((4, 2, 64), dtype=TD[dt], device=DEV)
    x[0, 0, 5], x[1, 1, 63], x[2, 0, 0] = INF, NAN, -INF
    big = torch.finfo(TD[dt]).max
    x[3, 0, :2] = torch.tensor([big, -big], dtype=TD[dt])
    slots = torch.tensor([3, 17, 20, 31], device=DEV)
    mnb.mnb_kv_append_i8(x, x, slots, cache)
    for y in mnb.mnb_kv_read_i8(slots, cache):
        bad = torch.isnan(y).all(dim=2)
        assert bad.tolist() == [[True, False], [False, True], [True, False], [False, False]]
        assert torch.isfinite(y[~bad]).all() and (y[0, 1] == 1).all() and y[3, 0, 0] == -y[3, 0, 1]


def test_read_into_columns_of_one_buffer_and_nothing():
    cache = _cache(3, 2, 16, 64, "f16")
    x = torch.randn((5, 2, 64), device=DEV).half()
    slots = torch.tensor([40, 2, 0, 17, 5], device=DEV)
    mnb.mnb_kv_append_i8(x, -x, slots, cache)
    k, v = mnb.mnb_kv_read_i8(slots, cache)
    fused = torch.full((5, 3 * 128), 7.0, dtype=torch.float16, device=DEV)
    mnb.mnb_kv_read_i8(slots, cache, k=fused[:, :128], v=fused[:, 256:])
    assert torch.equal(fused[:, :128].view(5, 2, 64), k) and torch.equal(fused[:, 256:].view(5, 2, 64), v)
    assert (fused[:, 128:256] == 7).all() and torch.equal(k, -v)
    none = mnb.mnb_kv_read_i8(slots[:0], cache)
    mnb.mnb_kv_append_i8(x[:0], x[:0], slots[:0], cache)
    assert none[0].shape == (0, 2, 64)
    # the same slot any number of times
    assert torch.equal(mnb.mnb_kv_read_i8(slots[1:2].expand(9).contiguous(), cache)[0], k[1:2].expand(9, 2, 64))
    with pytest.raises(ValueError, match="tokens"):
        mnb.mnb_kv_append_i8(x, x[:2], slots, cache)
    with pytest.raises(ValueError, match="must be torch.float16"):
        mnb.mnb_kv_append_i8(x.float(), x, slots, cache)
    with pytest.raises(mnb.MnbError):
        mnb.mnb_kv_read_i8(slots, cache, k=k, v=k)


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------

def _case(seed, lens, heads, kv_heads, dim, page, dt, order="block-head-token", new=None, spread=1.0):
    """Random keys and values at the valid positions; codes of 127 with scales
    NaN and infinity in every other place of the pool; blocks scattered,
    unused entries -1. Returns q, cache, table, lens, starts."""
    rng = np.random.default_rng(seed)
    width = max(1, max(-(-max(0, n) // page) for n in lens)) + 2
    held = [-(-max(0, n) // page) for n in lens]
    blocks = sum(held) + 3
    cache = _cache(blocks, kv_heads, page, dim, dt, order, code=127)
    cache.v_scale[::2] = INF
    cache.k_scale[1::2] = -INF
    ids = rng.permutation(blocks)
    table = np.full((len(lens), width), -1)
    slots, used = [], 0
    for b, n in enumerate(lens):
        table[b, : held[b]] = ids[used: used + held[b]]
        used += held[b]
        slots += [table[b, t // page] * page + t % page for t in range(n)]
    g = torch.Generator(DEV).manual_seed(seed)
    rows = [torch.randn((len(slots), kv_heads, dim), device=DEV, generator=g) for _ in range(2)]
    # values of different sizes from token to token
    rows[1] *= torch.exp(torch.randn((len(slots), kv_heads, 1), device=DEV, generator=g))
    mnb.mnb_kv_append_i8(rows[0].to(TD[dt]), rows[1].to(TD[dt]), torch.tensor(slots, dtype=torch.int64, device=DEV),
                         cache)
    i32 = dict(dtype=torch.int32, device=DEV)
    starts = None if new is None else torch.tensor(np.concatenate([[0], np.cumsum(new)]), **i32)
    tokens = len(lens) if new is None else sum(new)
    q = (spread * torch.randn((tokens, heads, dim), device=DEV, generator=g)).to(TD[dt])
    return q, cache, torch.tensor(table, **i32), torch.tensor(lens, **i32), starts


def _check(got, q, cache, table, lens, starts, max_len, max_new, dt, scale=None, what=""):
    scale = q.shape[-1] ** -0.5 if scale is None else scale
    qn, tn, got = _np(q), table.cpu().numpy(), _np(got)
    kn, vn = (_np(c) * _np(s)[..., None] for c, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)))
    sn = _np(cache.v_scale)[..., None]
    group = q.shape[1] // cache.kv_heads
    rows = oracle.visible(q.shape[0], lens.tolist(), None if starts is None else starts.tolist(), max_len, max_new)
    claims = [t for _, t, _ in rows]
    for b, t, n in rows:
        if claims.count(t) > 1:
            continue   # (a row of two requests holds either's result)
        k, v, s = (oracle.paged_rows(c, tn[b], n, cache.page_size) for c in (kn, vn, sn))
        for h in range(q.shape[1]):
            ref = oracle.attend(qn[t, h], k[:, h // group], v[:, h // group], scale)
            _near(got[t, h], ref, _bound(qn[t, h], k[:, h // group], v[:, h // group], s[:, h // group, 0], scale, dt),
                  f"{what} request {b}, row {t} of {n} keys, head {h}")
    return set(claims)


LENS = [[0], [1], [15, 16, 17], [31, 32, 33, 0, 1], [63, 64, 65, 127], [500, 3, 0, 257, 129], [2049, 1023]]
HEADS = [(16, 8), (12, 12), (8, 1), (40, 2), (5, 1)]


@pytest.mark.parametrize("lens", LENS, ids=lambda x: "-".join(map(str, x)))
@pytest.mark.parametrize("heads,kv_heads", HEADS)
@pytest.mark.parametrize("dim,page,dt", [(128, 16, "f16"), (64, 48, "f16"), (64, 16, "f32"), (128, 64, "f32")])
def test_single_tokens(lens, heads, kv_heads, dim, page, dt):
    print(f"attn8 {dt} lens={lens} heads={heads}/{kv_heads} dim={dim} page={page}", flush=True)
    q, cache, table, ln, _ = _case(sum(lens) + heads, lens, heads, kv_heads, dim, page, dt)
    got = mnb.mnb_paged_attn_i8(q, cache, table, ln, max(lens))
    _check(got, q, cache, table, ln, None, max(lens), 1, dt)


# (cached, new) per request
ROWS = [[(0, 1)], [(0, 2)], [(0, 17), (5, 3)], [(70, 1), (0, 0), (0, 33), (300, 5)], [(0, 64), (16, 65)],
        [(130, 100), (0, 129), (1, 1)], [(700, 31)]]


@pytest.mark.parametrize("rows", ROWS, ids=lambda x: "-".join(f"{c}+{n}" for c, n in x))
@pytest.mark.parametrize("heads,kv_heads", [(16, 8), (3, 3), (8, 1)])
@pytest.mark.parametrize("dim,page,dt", [(128, 16, "f16"), (64, 48, "f16"), (64, 16, "f32"), (128, 64, "f32")])
def test_several_tokens(rows, heads, kv_heads, dim, page, dt):
    print(f"attn8 rows {dt} {rows} heads={heads}/{kv_heads} dim={dim} page={page}", flush=True)
    lens, new = [c + n for c, n in rows], [n for _, n in rows]
    q, cache, table, ln, starts = _case(sum(lens) + heads, lens, heads, kv_heads, dim, page, dt, new=new)
    got = mnb.mnb_paged_attn_i8(q, cache, table, ln, max(lens), starts=starts, max_new=max(new))
    assert _check(got, q, cache, table, ln, starts, max(lens), max(new), dt) == set(range(sum(new)))


@pytest.mark.parametrize("dt", ["f16", "f32"])
@pytest.mark.parametrize("new", [None, [7, 40, 1]])
def test_rows_of_no_request_and_past_the_bounds_stay(dt, new):
    # spare rows behind the last request; bounds below what the requests have; bad starts
    lens = [100, 40, 64]
    q, cache, table, ln, starts = _case(5, lens, 4, 2, 64, 16, dt, new=new)
    if new is None:
        _check(mnb.mnb_paged_attn_i8(q, cache, table, ln, 50), q, cache, table, ln, None, 50, 1, dt)
        _check(mnb.mnb_paged_attn_i8(q, cache, table, ln, 100000), q, cache, table, ln, None, 100000, 1, dt)
        out = mnb.mnb_paged_attn_i8(q, cache, table, ln - 64, 100)
        assert not out[1:].any()
        narrow = table[:, :3].contiguous()
        got = mnb.mnb_paged_attn_i8(q, cache, narrow, ln, 100)
        _check(got, q, cache, narrow, ln, None, 48, 1, dt)
        assert not mnb.mnb_paged_attn_i8(q, cache, table, ln, 0).any()
        return
    q = torch.cat((q, q[:5]))
    for s, max_new, max_len in (([0, 7, 47, 48], 40, 100), ([0, 7, 47, 48], 8, 100), ([0, 7, 47, 48], 40, 30),
                                ([-9, 3, 2, 1000], 60, 100), ([5, 5, 5, 9], 40, 1000), ([48, 7, 0, 0], 9, 100)):
        st = torch.tensor(s, dtype=torch.int32, device=DEV)
        out = torch.full_like(q, 7.0)
        got = mnb.mnb_paged_attn_i8(q, cache, table, ln, max_len, starts=st, max_new=max_new, out=out)
        done = _check(got, q, cache, table, ln, st, max_len, max_new, dt, what=f"starts {s}")
        rest = [t for t in range(q.shape[0]) if t not in done]
        assert (got[rest] == 7.0).all(), s


@pytest.mark.parametrize("order", ORDERS)
@pytest.mark.parametrize("dt", ["f16", "f32"])
def test_memory_orders_and_strided_queries(order, dt):
    for new in (None, [40, 66, 3]):
        q, cache, table, ln, starts = _case(3, [70, 300, 16], 4, 2, 128, 32, dt, order, new=new)
        T = q.shape[0]
        fused = torch.full((T, 4 * 128 + 2 * 256), NAN, dtype=TD[dt], device=DEV)   # q beside k and v
        fused[:, :512] = q.reshape(T, 512)
        got = mnb.mnb_paged_attn_i8(fused[:, :512].view(T, 4, 128), cache, table, ln, 300, starts=starts,
                                    max_new=66 if new else 1)
        _check(got, q, cache, table, ln, starts, 300, 66 if new else 1, dt)


@pytest.mark.parametrize("dt", ["f16", "f32"])
def test_long_caches_split_and_joined(dt):
    for lens, heads, kv_heads, dim, new in (([20000], 16, 8, 128, None), ([40001, 7, 9000], 4, 1, 64, None),
                                            ([20000, 300], 4, 2, 128, [3, 5])):
        print(f"attn8 {dt} lens={lens} heads={heads}/{kv_heads} dim={dim} new={new}", flush=True)
        q, cache, table, ln, starts = _case(9, lens, heads, kv_heads, dim, 64, dt, spread=2.0, new=new)
        n = max(new) if new else 1
        ws = mnb.paged_attn_i8_workspace(q, cache, table, max(lens), n)
        got = []
        for junk in (0xFF, 0x00, 0x7F):      # the workspace's old contents do not matter
            ws.fill_(junk)
            got.append(mnb.mnb_paged_attn_i8(q, cache, table, ln, max(lens), starts=starts, max_new=n,
                                             workspace=ws).clone())
        assert torch.equal(got[0], got[1]) and torch.equal(got[0], got[2])
        _check(got[0], q, cache, table, ln, starts, max(lens), n, dt)


@pytest.mark.parametrize("dt", ["f16", "f32"])
@pytest.mark.parametrize("new", [None, [100, 120, 20, 16]])
def test_missing_blocks_are_left_out(dt, new):
    q, cache, table, ln, starts = _case(6, [200, 130, 33, 16], 6, 3, 128, 16, dt, new=new)
    table[0, 3] = -1
    table[0, 12] = cache.num_blocks
    table[1, 0] = 2 ** 31 - 1
    table[1, 1] = -2 ** 31
    table[2, :] = -5
    got = mnb.mnb_paged_attn_i8(q, cache, table, ln, 200, starts=starts, max_new=120 if new else 1)
    assert not got[2 if new is None else slice(220, 240)].any()
    _check(got, q, cache, table, ln, starts, 200, 120 if new else 1, dt)


def _at(table, page, b, t):
    return int(table[b, t // page]), slice(None), t % page


@pytest.mark.parametrize("dt", ["f16", "f32"])
@pytest.mark.parametrize("new", [None, [40, 40, 40, 40]])
def test_scales_and_queries_that_are_not_finite(dt, new):
    q, cache, table, ln, starts = _case(7, [50, 50, 50, 50], 4, 2, 64, 16, dt, new=new)
    cache.k_scale[_at(table, 16, 0, 20)] = NAN        # a key of request 0: NaN for the rows that see it
    cache.v_scale[_at(table, 16, 1, 20)] = NAN        # a value of request 1
    per = 1 if new is None else 40
    for at in (2 * per + per // 2, 3 * per):
        q[at, 1, 7] = NAN if at == 3 * per else INF   # one head of one row of requests 2 and 3
    got = mnb.mnb_paged_attn_i8(q, cache, table, ln, 50, starts=starts, max_new=per)
    sees = [t for b in range(2) for t in range(b * per, (b + 1) * per) if 50 - per + t - b * per >= 20]
    bad = torch.zeros(got.shape[:2], dtype=torch.bool, device=DEV)
    bad[sees] = True
    bad[2 * per + per // 2, 1] = bad[3 * per, 1] = True
    assert torch.equal(torch.isnan(got).all(dim=2), bad) and torch.equal(torch.isnan(got).any(dim=2), bad)
    # the others are what they are without them
    cache.k_scale[_at(table, 16, 0, 20)] = cache.v_scale[_at(table, 16, 1, 20)] = 0.01
    q.nan_to_num_(1.0, 1.0, 1.0)
    clean = mnb.mnb_paged_attn_i8(q, cache, table, ln, 50, starts=starts, max_new=per)
    assert torch.equal(got[~bad], clean[~bad])


@pytest.mark.parametrize("dt", ["f16", "f32"])
def test_sharp_and_flat_rows(dt):
    # one key far above the others anywhere in the row; keys of equal scores; queries of zeros
    for new in (None, [50]):
        for at in (0, 31, 32, 63, 64, 240):
            q, cache, table, ln, starts = _case(8, [300], 2, 1, 64, 32, dt, new=new)
            cache.k.zero_()
            q.fill_(4.0)
            cache.k[_at(table, 32, 0, at)] = 127
            cache.k_scale[_at(table, 32, 0, at)] = 2.0
            got = mnb.mnb_paged_attn_i8(q, cache, table, ln, 300, starts=starts, max_new=50) if new else \
                mnb.mnb_paged_attn_i8(q, cache, table, ln, 300)
            block, _, offset = _at(table, 32, 0, at)
            want = (cache.v[block, 0, offset].double() * cache.v_scale[block, 0, offset].double())
            off = (got.double() - want).abs()
            # one weight of 1, times its value scale: the output's rounding, 2^-11 in float16; calls of many rows
            # round that product to float16 too (2^-11 more, (1 + 2^-11)^2 < 1 + 2^-10 + 2^-20)
            rel = 2.0 ** -19 if dt == "f32" else (2.0 ** -10 if new else 2.0 ** -11) + 2.0 ** -20
            assert (off <= want.abs() * rel + 2.0 ** -25).all()
        q.zero_()
        got = mnb.mnb_paged_attn_i8(q, cache, table, ln, 300, starts=starts, max_new=50 if new else 1)
        _check(got, q, cache, table, ln, starts, 300, 50, dt)


@pytest.mark.parametrize("dt", ["f16", "f32"])
def test_scales_of_scores_and_of_values(dt):
    for new in (None, [33, 64]):
        q, cache, table, ln, starts = _case(10, [90, 64], 4, 4, 64, 16, dt, new=new)
        n = 64 if new else 1
        for scale in (0.0, -0.3, 1.7, 30.0):
            got = mnb.mnb_paged_attn_i8(q, cache, table, ln, 90, starts=starts, max_new=n, scale=scale)
            _check(got, q, cache, table, ln, starts, 90, n, dt, scale, f"scale {scale}")
        # value rows from 2^-60 to 2^12 of their size beside one another, and rows of scale zero
        far = 2.0 ** torch.randint(-60 if dt == "f32" else -8, 12, cache.v_scale.shape, device=DEV).float()
        cache.v_scale.mul_(far * (torch.rand(far.shape, device=DEV) < 0.9)).nan_to_num_(0, 0, 0)
        got = mnb.mnb_paged_attn_i8(q, cache, table, ln, 90, starts=starts, max_new=n)
        _check(got, q, cache, table, ln, starts, 90, n, dt, what="scales of all sizes")


@pytest.mark.parametrize("dt", ["f16", "f32"])
def test_large_and_small_queries(dt):
    for new in (None, [33, 64]):
        for size in ((1e-3, 60000.0) if dt == "f16" else (1e-30, 1e30)):
            q, cache, table, ln, starts = _case(11, [90, 64], 2, 1, 128, 16, dt, new=new)
            q = (q / q.abs().amax() * size).to(TD[dt])
            scale = 0.5 / size
            n = 64 if new else 1
            got = mnb.mnb_paged_attn_i8(q, cache, table, ln, 90, starts=starts, max_new=n, scale=scale)
            _check(got, q, cache, table, ln, starts, 90, n, dt, scale, f"queries of {size}")


def test_one_flat_row_below_a_leading_key():
    # a key 17.7 above 16000 equal ones: these still hold 3e-4 of the weight
    n = 16000
    q, cache, table, ln, _ = _case(12, [n], 1, 1, 64, 64, "f32")
    cache.k.zero_()
    cache.v.fill_(100)
    cache.v_scale.fill_(1.0)
    q.fill_(1.0)
    block, _, offset = _at(table, 64, 0, 777)
    cache.k[block, 0, offset] = 127
    cache.k_scale.fill_(17.7 / (64 * 127 * 0.125))
    cache.v[block, 0, offset] = 0
    got = mnb.mnb_paged_attn_i8(q, cache, table, ln, n)
    w = np.exp(-float(cache.k_scale[block, 0, offset]) * 64 * 127 * 0.125) * (n - 1)
    # weights of one tile count against the leading key's 2^-21 only in that tile: 63 keys
    want = 100 * w / (1 + w)
    assert abs(float(got[0, 0, 0]) - want) <= want * 2.0 ** -15 + 100 * 64 * 2.0 ** -21


def test_the_same_bits_again_on_another_stream_and_replayed():
    for new in (None, [60, 100, 1, 0]):
        q, cache, table, ln, starts = _case(13, [3000, 100, 2, 700], 8, 4, 64, 16, "f16", new=new)
        n = 100 if new else 1
        ws = mnb.paged_attn_i8_workspace(q, cache, table, 3000, n)
        args = dict(starts=starts, max_new=n, workspace=ws)
        want = mnb.mnb_paged_attn_i8(q, cache, table, ln, 3000, **args)
        torch.cuda.synchronize()
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            got = mnb.mnb_paged_attn_i8(q, cache, table, ln, 3000, starts=starts, max_new=n)
        s.synchronize()
        assert torch.equal(got, want)
        out = torch.zeros_like(q)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            mnb.mnb_paged_attn_i8(q, cache, table, ln, 3000, out=out, **args)
        for step in range(3):
            q.neg_()
            ln -= 1
            out.zero_()
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, mnb.mnb_paged_attn_i8(q, cache, table, ln, 3000, starts=starts, max_new=n,
                                                          out=torch.zeros_like(q)))


def test_refused_calls_leave_the_outputs():
    q, cache, table, ln, starts = _case(14, [30, 20], 4, 2, 64, 16, "f16", new=[3, 2])
    out = torch.full_like(q, 5.0)
    with pytest.raises(ValueError, match="starts says"):
        mnb.mnb_paged_attn_i8(q, cache, table, ln, 30, out=out)
    with pytest.raises(mnb.MnbError):
        mnb.mnb_paged_attn_i8(q, cache, table, ln, 30, starts=starts, max_new=0, out=out,
                              workspace=torch.empty(0, dtype=torch.uint8, device=DEV))
    with pytest.raises(mnb.MnbError):
        mnb.mnb_paged_attn_i8(q, cache, table, ln, 30, starts=starts, max_new=3, scale=INF, out=out)
    with pytest.raises(ValueError, match="elements"):
        mnb.mnb_paged_attn_i8(q, cache, table, ln, 30, starts=starts[:2], max_new=3, out=out)
    with pytest.raises(ValueError, match="contiguous heads"):
        mnb.mnb_paged_attn_i8(q[:, :, :32], cache, table, ln, 30, starts=starts, max_new=3, out=out)
    with pytest.raises(ValueError, match="must be torch.float16"):
        mnb.mnb_paged_attn_i8(q.float(), cache, table, ln, 30, starts=starts, max_new=3, out=out)
    with pytest.raises(mnb.MnbError):
        mnb.mnb_paged_attn_i8(q, cache, table, ln, 30, starts=starts, max_new=3, out=q)
    torch.cuda.synchronize()
    assert (out == 5.0).all()
