"""GPU: attention at values where its arithmetic can go wrong, in every form of
the kernels. Each case is one query row over one run of keys, the same for all
requests, heads and query rows of a call whose sizes choose the form.

Where an output is finite, it is held to the bound of test_gpu_attn (`_bound`),
or to the one that the test derives.
"""

import numpy as np
import pytest
import torch

import oracle
import test_gpu_attn as base
from block_wise_int4_amd import mnb

pytestmark = pytest.mark.gpu

DEV, TD, NAN, INF, DIM = base.DEV, base.TD, float("nan"), float("inf"), 64

# form: (batch, query rows, heads, keys); the names are the kernels' forms
FORMS = {
    "paged": (3, 1, 2, 70),            # one token over pages, one workgroup a row
    "paged-short": (500, 1, 2, 20),    # fewer waves a workgroup
    "paged-cut": (1, 1, 2, 5000),      # chunks joined by a second launch
    "token": (3, 1, 2, 70),            # one token over an encoder's states
    "rows": (3, 20, 2, 70),            # two row tiles
    "many-4": (130, 20, 2, 70),        # float16: four waves of rows
    "many-2": (130, 20, 2, 300),       # float16: two groups of keys
}
F16_ONLY = ("many-4", "many-2")
ALL = [(form, dt) for form in FORMS for dt in ("f16", "f32") if not (form in F16_ONLY and dt == "f32")]


def _call(form, dt, q, k, v, n, scale):
    """All output rows [rows, DIM] (float64) of query q [DIM] over the first n
    of the rows k, v [keys, DIM], NaN and infinities in the places behind."""
    batch, queries, heads, keys = FORMS[form]
    q, k, v = (torch.as_tensor(t, dtype=torch.float64).to(TD[dt]).to(DEV) for t in (q, k, v))
    k, v = k.clone(), v.clone()
    k[n:], v[n:] = NAN, INF
    lens = torch.full((batch,), n, dtype=torch.int32, device=DEV)
    if form.startswith("paged"):
        blocks = -(-keys // 16)
        pages = [torch.full((blocks, heads, 16, DIM), NAN, dtype=TD[dt], device=DEV) for _ in range(2)]
        for page, rows in zip(pages, (k, v)):
            whole = torch.full((blocks * 16, DIM), NAN, dtype=TD[dt], device=DEV)
            whole[:keys] = rows
            page.copy_(whole.view(blocks, 1, 16, DIM).expand(-1, heads, -1, -1))
        cache = mnb.KvCache(*pages)
        table = torch.arange(blocks, dtype=torch.int32, device=DEV).repeat(batch, 1)
        cut = mnb.mnb_paged_attn_workspace_bytes(batch, heads, cache, keys) > 0
        assert cut == (form == "paged-cut")
        got = mnb.mnb_paged_attn(q.expand(batch, heads, DIM).contiguous(), cache, table, lens, keys, scale=scale)
    else:
        whole = [t.expand(batch, heads, keys, DIM).transpose(1, 2).contiguous() for t in (k, v)]
        got = mnb.mnb_cross_attn(q.expand(batch, queries, heads, DIM).contiguous(), *whole, lens, scale=scale)
    got = got.reshape(-1, DIM)
    torch.cuda.synchronize()
    assert torch.equal(got.nan_to_num(7.0, 8.0, 9.0), got[:1].expand_as(got).nan_to_num(7.0, 8.0, 9.0)), "rows differ"
    return got[0].cpu().double().numpy()


def _rand(seed, keys, dt):
    """q [DIM], k, v [keys, DIM] as float64, of values of the type."""
    g = torch.Generator().manual_seed(seed)
    return [torch.randn(s, generator=g).to(TD[dt]).double().numpy() for s in ((DIM,), (keys, DIM), (keys, DIM))]


def _say(form, dt, what):
    print(f"{form} {dt} {what}", flush=True)


# ---------------------------------------------------------------------------
# rows whose weights sum to zero

@pytest.mark.parametrize("form,dt", ALL)
def test_rows_without_weight_are_zeros_whatever_their_values(form, dt):
    _say(form, dt, "no weight")
    keys = FORMS[form][3]
    q, k, v = _rand(1, keys, dt)
    q[:], k[:] = 1.0, -INF
    v[1, 3], v[keys - 2, 5], v[0, 7], v[0, 8] = INF, NAN, -INF, NAN
    assert not _call(form, dt, q, k, v, keys - 1, 1.0).any()


# ---------------------------------------------------------------------------
# keys that are not valid, where the query is infinite

@pytest.mark.parametrize("form,dt", ALL)
def test_infinite_queries_do_not_reach_keys_that_are_not_valid(form, dt):
    _say(form, dt, "infinite query")
    keys = FORMS[form][3]
    q, k, v = _rand(2, keys, dt)
    q[5], k[:, 5] = -INF, np.abs(k[:, 5]) + 0.5       # every valid score is -infinity
    for n in (1, keys - 33 if keys > 33 else 3, keys - 1):
        assert not _call(form, dt, q, k, v, n, 0.125).any(), n


@pytest.mark.parametrize("dt", ["f16", "f32"])
@pytest.mark.parametrize("batch,keys", [(3, 20), (130, 20), (130, 300)])
def test_key_rows_that_overlap_in_memory(batch, keys, dt):
    # rows 32 elements apart: the row behind the last valid one starts with that
    # one's second half, which the query's first half meets with another sign
    queries, heads, n = 20, 2, 5
    g = torch.Generator().manual_seed(3)
    flat = torch.randn((32 * (keys + 1),), generator=g).to(TD[dt])
    flat[32 * (n - 1) + 40] = -INF
    q1 = torch.randn((DIM,), generator=g).to(TD[dt])
    q1[40], q1[8] = 1.0, -1.0
    v1 = torch.randn((keys, DIM), generator=g).to(TD[dt])
    k1 = flat.as_strided((keys, DIM), (32, 1))
    k = flat.to(DEV).as_strided((batch, keys, heads, DIM), (0, 32, 0, 1))
    v = v1.to(DEV)[None, :, None].expand(batch, -1, heads, -1).contiguous()
    q = q1.to(DEV).expand(batch, queries, heads, DIM).contiguous()
    got = mnb.mnb_cross_attn(q, k, v, torch.full((batch,), n, dtype=torch.int32, device=DEV)).reshape(-1, DIM)
    qn, kn, vn = (t.double().numpy() for t in (q1, k1[: n - 1], v1[: n - 1]))     # (the last one weighs nothing)
    ref, tol = oracle.attend(qn, kn, vn, DIM ** -0.5), base._bound(qn, kn, vn, DIM ** -0.5, dt)
    base._near(base._np(got), ref[None], tol[None], "overlapping keys")


# ---------------------------------------------------------------------------
# infinite values in valid places

@pytest.mark.parametrize("form,dt", ALL)
def test_infinite_values_in_valid_places(form, dt):
    _say(form, dt, "infinite values")
    keys = FORMS[form][3]
    for n in (1, 2, keys - 1):
        q, k, v = _rand(4, keys, dt)
        at = n - 1 if n > 1 else 0
        v[at, 3], v[0, 7], v[at, 7], v[at // 2, 60] = INF, -INF, -INF, -INF
        got = _call(form, dt, q, k, v, n, DIM ** -0.5)
        ref = oracle.attend(q, k[:n], v[:n], DIM ** -0.5)
        assert ref[3] == INF and ref[7] == ref[60] == -INF
        assert got[3] == INF and got[7] == -INF and got[60] == -INF, (n, got[[3, 7, 60]])
        rest = [d for d in range(DIM) if d not in (3, 7, 60)]
        base._near(got[rest], ref[rest], base._bound(q, k[:n], v[:n][:, rest], DIM ** -0.5, dt), f"{n} keys")


def _infinite_values_of_small_weight(form, dt):
    _say(form, dt, "infinite values, small weight")
    keys = FORMS[form][3]
    n = keys - 1
    q, k, v = _rand(5, keys, dt)
    q[:], k[:] = 1.0, 0.0
    k[n // 2] = 30.0 / DIM                       # 30 above the others: these weigh 1e-13, not nothing
    v[1, 3], v[n - 1, 9] = INF, -INF
    v[0, 20], v[n - 1, 20] = INF, -INF           # a sum of both
    v[2, 21] = NAN
    got = _call(form, dt, q, k, v, n, 1.0)
    assert got[3] == INF and got[9] == -INF and np.isnan(got[[20, 21]]).all(), got[[3, 9, 20, 21]]
    rest = [d for d in range(DIM) if d not in (3, 9, 20, 21)]
    ref = oracle.attend(q, k[:n], v[:n][:, rest], 1.0)
    base._near(got[rest], ref, base._bound(q, k[:n], v[:n][:, rest], 1.0, dt), "the other dimensions")


@pytest.mark.parametrize("form,dt", [f for f in ALL if f[0] not in F16_ONLY])
def test_infinite_values_of_small_weight_and_of_both_signs(form, dt):
    _infinite_values_of_small_weight(form, dt)


# ---------------------------------------------------------------------------
# the same in the form for many rows

@pytest.mark.parametrize("form", F16_ONLY)
def test_infinite_values_of_small_weight_among_many_rows(form):
    _infinite_values_of_small_weight(form, "f16")


# ---------------------------------------------------------------------------
# weights far below the largest

@pytest.mark.parametrize("form,dt", ALL)
def test_flat_tail_far_below_one_leading_key(form, dt):
    # A key of value 0 and n - 1 keys of value `top` 17.7 below it: the output is
    # the tail's share, whose weights (2^-25.5) may each be off by 2^-32 of the
    # row's reference, and by 2 (DIM + 8) u S + 2^-21 relative (see _bound, S =
    # 17.7); the sums are of equal terms, n u; then the output's own rounding.
    _say(form, dt, "flat tail")
    n = FORMS[form][3] - 1
    q, k, v = np.ones(DIM), np.zeros((n + 1, DIM)), np.zeros((n + 1, DIM))
    lead, top = 17.75, 32768.0
    k[0] = lead / DIM                            # (exact in float16)
    v[1:] = top
    got = _call(form, dt, q, k, v, n, 1.0)
    ref = oracle.attend(q, k[:n], v[:n], 1.0)
    u = 2.0 ** -24
    tol = ref * (2 * (DIM + 8) * u * lead + 2.0 ** -21 + 2 * (n + 64) * u) + 1e-30
    if dt == "f16":
        tol += n * 2.0 ** -32 * top + ref * 2.0 ** -11 + 2.0 ** -25
    base._near(got, ref, tol, f"{n} keys")


# ---------------------------------------------------------------------------
# float16 weights of the form for few rows: a pair of float16 numbers

@pytest.mark.parametrize("form", ["paged", "paged-short", "paged-cut", "token", "rows"])
def test_few_rows_keep_more_than_float16_weights(form):
    # Scores that are exact (small whole numbers, a scale of 1/8), values whose
    # weighted sum cancels: what is left shows the weights' own errors. Those are
    # 2^-22 relative for the pair, 2^-32 of the reference at least, |x| u twice
    # for a score x = s log2(e) and its difference (|s| <= 4), 2^-21 for the
    # exponential and the joins; sums of n terms n u, and 64 u for the joins.
    # Weights of 11 bits would be off by some 2^-12.3 / sqrt(n) of `a`.
    _say(form, "f16", "pairs")
    n = FORMS[form][3] - 1
    rng = np.random.default_rng(6)
    q, k, v = np.zeros(DIM), np.zeros((n + 1, DIM)), rng.standard_normal((n + 1, DIM))
    q[:32] = 1.0
    k[:, :32] = rng.integers(-1, 2, (n + 1, 32))
    k[:, 0] += rng.integers(-3, 4, n + 1)
    score = (k @ q / 8)[:n]
    assert np.abs(score).max() <= 4
    p = np.exp(score - score.max())
    v[:n] -= (p[:, None] * v[:n]).sum(axis=0) / p.sum()
    v = v.astype(np.float16).astype(np.float64)
    got = _call(form, "f16", q, k, v, n, 0.125)
    ref = oracle.attend(q, k[:n], v[:n], 0.125)
    a = (p[:, None] * np.abs(v[:n])).sum(axis=0) / p.sum()
    u = 2.0 ** -24
    tol = a * 2 * (2.0 ** -22 + 2 * 4 * 1.4427 * u * 2 + 2.0 ** -21 + (n + 64) * u)
    tol += n / p.sum() * 2.0 ** -32 * np.abs(v).max() + np.abs(ref) * 2.0 ** -11 + 2.0 ** -25
    base._near(got, ref, tol, f"{n} keys")


# ---------------------------------------------------------------------------
# scores of any size that finite float16 rows reach

@pytest.mark.parametrize("form,dt", ALL)
def test_scores_up_to_the_largest(form, dt):
    # rows whose products are exact in float32, and so are ties; the keys of the
    # largest score share the output, all others weigh nothing
    _say(form, dt, "large scores")
    keys = FORMS[form][3]
    _, _, v = _rand(8, keys, dt)
    for n in (1, keys - 1):
        for size, scale in ((300.0, 0.125), (3000.0, 0.125), (30000.0, 0.125), (30000.0, 1.7)):
            for sign in (1.0, -1.0):
                q = np.full(DIM, sign * size)
                k = np.repeat((np.arange(keys) % 7 + 1.0)[:, None] * size / 15, DIM, axis=1)
                score = k[:n, 0] * sign
                best = np.flatnonzero(score == score.max())
                got = _call(form, dt, q, k, v, n, scale)
                tol = base._bound(np.zeros(DIM), k[best], v[best], 1.0, dt)      # the mean of equal weights
                base._near(got, v[best].mean(axis=0), tol, f"{n} keys, {sign * size}, scale {scale}")


# ---------------------------------------------------------------------------
# scales at the ends of their range

@pytest.mark.parametrize("form,dt", ALL)
def test_scales_at_the_ends_of_their_range(form, dt):
    _say(form, dt, "scales")
    keys = FORMS[form][3]
    n = keys - 1
    q, k, v = _rand(7, keys, dt)
    zero = np.zeros(DIM)
    for scale in (3e38, -3e38, 1e-38, 0.0):
        got = _call(form, dt, zero, k, v, n, scale)        # every score is 0: the mean
        base._near(got, v[:n].mean(axis=0), base._bound(zero, k[:n], v[:n], 1.0, dt), f"scale {scale}")
    if dt == "f16":
        q[:], k[:] = 1.0, 0.0
        k[:, 0] = np.arange(keys) % 7 * 0.25
        k[n // 2, 0] = 2.0
        for scale in (1e38, 3e38):                         # the largest score takes all
            assert np.array_equal(_call(form, dt, q, k, v, n, scale), v[n // 2])
            worst = np.flatnonzero(k[:n, 0] == 0.0)
            got = _call(form, dt, q, k, v, n, -scale)
            base._near(got, v[worst].mean(axis=0), base._bound(zero, k[worst], v[worst], 1.0, dt), f"scale -{scale}")


# ---------------------------------------------------------------------------
# small weights in the denominator

@pytest.mark.parametrize("dt", ["f16", "f32"])
@pytest.mark.parametrize("batch,dim", [(3, 64), (130, 64), (130, 128), (1030, 64)])
@pytest.mark.parametrize("keys", [200, 65000])
def test_small_weights_count_in_both_sums(batch, dim, keys, dt):
    # one leading key and a flat row of weights 2^-23 below it, all values 1: the
    # output is 1 whatever the weights, if both sums have all of them. At 65000 keys
    # the flat row is 0.8% of the sums; each is of some keys / 2 float32 additions at
    # most of numbers below 2^-15 of it, off by less than 2^-11 of the whole (keys / 2
    # roundings of 2^-24 and a common factor), and the output's rounding is 2^-11.
    print(f"small weights {dt} batch={batch} dim={dim} keys={keys}", flush=True)
    queries, heads = 20, 2
    k = torch.zeros((1, keys, 1, dim), dtype=TD[dt], device=DEV)
    k[0, 0, 0] = 23 * float(np.log(2)) / dim
    v = torch.ones_like(k)
    q = torch.ones((batch, queries, heads, dim), dtype=TD[dt], device=DEV)
    k, v = (t.expand(batch, keys, heads, dim) for t in (k, v))
    got = mnb.mnb_cross_attn(q, k, v, scale=1.0)
    base._near(base._np(got), np.ones(got.shape), np.full(got.shape, keys / 2 * 2.0 ** -24 + 2.0 ** -11))
