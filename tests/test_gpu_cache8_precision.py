"""GPU: how finely the attention over the 8-bit cache holds weights times value
scales, in rows whose terms nearly cancel: an output is then far smaller than its
terms, and neither its own rounding nor a bound relative to it hides theirs.
"""

import numpy as np
import pytest
import torch

import oracle
from block_wise_int4_amd import mnb
from test_gpu_cache8 import DEV, TD, _bound, _cache, _case, _near, _np

pytestmark = pytest.mark.gpu

I32 = dict(dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("dt", ["f16", "f32"])
@pytest.mark.parametrize("new", [None, [5], [20], [60], [130]], ids=str)
@pytest.mark.parametrize("keys,dim", [(300, 64), (300, 128), (3000, 128)])
def test_terms_that_cancel(keys, dim, new, dt):
    # keys of one score; values 100 of scale 1 + 0.51 2^-10 and -100 of scale 1 + 0.49 2^-10, in turn: either
    # scale is half a float16 step from the number that float16 makes of it, to opposite sides, and the
    # result is 50 * 0.02 * 2^-10 instead of 50 * 2^-10
    q, cache, table, ln, starts = _case(61, [keys], 2, 1, dim, 16, dt, new=new)
    cache.k.zero_()
    cache.k_scale.fill_(1.0)
    cache.v.fill_(100)
    cache.v[:, :, 1::2] = -100
    cache.v_scale.fill_(1.0 + 0.51 * 2.0 ** -10)
    cache.v_scale[:, :, 1::2] = 1.0 + 0.49 * 2.0 ** -10
    got = _np(mnb.mnb_paged_attn_i8(q, cache, table, ln, keys, starts=starts, max_new=new[0] if new else 1))
    scales = cache.v_scale[0, 0, :2].tolist()
    tokens = got.shape[0]
    for t in range(tokens):
        n = keys - tokens + t + 1
        want = 100 * (scales[0] * ((n + 1) // 2) - scales[1] * (n // 2)) / n
        # weights of 1 exactly; 22-bit numbers (half a step of 2^-21 each) times codes of 100; sums of n
        # terms of 100.05, in pieces joined by factors of 1; the division, the output
        tol = 100.05 * (2.0 ** -21 + (n + 64) * 2.0 ** -24) + abs(want) * (2.0 ** -11 if dt == "f16" else 2.0 ** -22)
        tol += 2.0 ** -25
        assert np.abs(got[t] - want).max() <= tol, (t, n, np.abs(got[t] - want).max() / tol)


@pytest.mark.parametrize("heads", [4, 12, 40, 130])
@pytest.mark.parametrize("dim", [64, 128])
def test_two_keys_that_cancel(dim, heads):
    # float16, weights of every size: values of opposite sign whose products with the weights are a few
    # thousandths apart, for each of many query heads. The bound of a float32 call (weights within 2^-21 of the
    # tile's largest), the exponents' rounding beside a power of two up to 2^60 (four times half a step of
    # numbers below 128, 2^-18, of which a weight is moved by ln 2 times as much, in both sums), the output
    B = 8
    g = torch.Generator(DEV).manual_seed(dim + heads)
    cache = _cache(B, 1, 16, dim, "f16", code=0, scale=0.0)
    q = torch.randn((B, heads, dim), device=DEV, generator=g).half()
    cache.k[:, 0, :2] = torch.randint(-127, 128, (B, 2, dim), device=DEV, generator=g).to(torch.int8)
    cache.k_scale[:, 0, :2] = 0.02
    table = torch.arange(B, **I32)[:, None].contiguous()
    lens = torch.full((B,), 2, **I32)
    for head in range(min(heads, 4)):      # cancels for one head at a time
        k = _np(cache.k[:, 0, :2]) * float(cache.k_scale[0, 0, 0])
        score = (k * _np(q[:, head])[:, None]).sum(axis=2) * dim ** -0.5
        ratio = np.exp(score[:, 0] - score[:, 1])     # of the weights
        cache.v[:, 0, 0], cache.v[:, 0, 1] = 100, -100
        cache.v_scale[:, 0, 0] = 0.37
        cache.v_scale[:, 0, 1] = torch.from_numpy(0.37 * ratio * (1 + 2.0 ** -9)).to(DEV).float()
        got = _np(mnb.mnb_paged_attn_i8(q, cache, table, lens, 2))
        vn, sn = _np(cache.v) * _np(cache.v_scale)[..., None], _np(cache.v_scale)
        for b in range(B):
            v, vs = vn[b, 0, :2], sn[b, 0, :2]
            ref = oracle.attend(_np(q[b, head]), k[b], v, dim ** -0.5)
            p = np.exp(score[b] - score[b].max())
            a = (p[:, None] * np.abs(v)).sum(axis=0) / p.sum()
            tol = _bound(_np(q[b, head]), k[b], v, vs, dim ** -0.5, "f32") + a * 2 * 4 * 2.0 ** -18 * np.log(2)
            assert np.all(np.abs(ref) < a * 2.0 ** -8)
            _near(got[b, head], ref, tol + np.abs(ref) * 2.0 ** -11 + 2.0 ** -25, f"request {b}, head {head} of {heads}")


@pytest.mark.parametrize("size", [50, 3e3, 8e3, 1.1e4, 1.126e4, 1.128e4, 1.2e4, 1.6e4, 3e4])
@pytest.mark.parametrize("rise", [0, 12])
@pytest.mark.parametrize("new", [None, [10], [20], [60]], ids=str)
def test_equal_scores_of_different_steps_cancel(new, rise, size):
    # keys of one score, 64 with a value of 100, 64 with -100, in turn; with `rise` the first 128 are that much
    # lower, 64 of them twice. Calls of many float16 rows take a score less its reference as one multiply-add
    # while 128 times the codes' and the query's largest sum stays below 2^14 by log2(e): codes of 127 reach
    # scores of 11267 there. The reference and its difference from the factor's exponent are then float32
    # numbers up to 2^14, each off by 2^-11, which moves a step's weights by ln 2 times 2^-10 at most, in the
    # sum and in the total. Beyond that, and in the other calls, equal scores weigh the same.
    dim, keys = 64, 640
    one_fma = new is not None and 2 * new[0] >= 33 and size < 11267      # (two heads share the keys)
    for sign in (1, -1):
        q, cache, table, ln, starts = _case(62, [keys], 2, 1, dim, 16, "f16", new=new)
        q.fill_(100.0)
        cache.k.fill_(127)
        cache.k_scale.fill_(1.0)
        cache.v_scale.fill_(1.0)
        for t in range(keys):
            where = int(table[0, t // 16]), 0, t % 16
            cache.v[where] = 100 if t // 64 % 2 == 0 else -100
            if t < 128:
                cache.k_scale[where] = 1.0 - sign * rise * (2 - t // 64) / size
        by = sign * size / (dim * 100.0 * 127)
        got = _np(mnb.mnb_paged_attn_i8(q, cache, table, ln, keys, starts=starts, max_new=new[0] if new else 1, scale=by))
        ids, kn, vn = table[0].cpu().numpy(), _np(cache.k) * _np(cache.k_scale)[..., None], _np(cache.v)
        tokens = got.shape[0]
        for t in range(tokens):
            n = keys - tokens + t + 1
            k, v = (oracle.paged_rows(x, ids, n, 16)[:, 0] for x in (kn, vn))
            ref = oracle.attend(_np(q)[t, 0], k, v, by)
            # terms of 100 as 22-bit numbers, sums of n of them; the lower keys' weights, below e^-12 in all
            # but off by any part of themselves where scores are large; the output
            tol = 100 * (2.0 ** -20 + (n + 64) * 2.0 ** -24 + (2 * 2.0 ** -10 if one_fma else 0.0))
            tol += np.abs(ref) * 2.0 ** -11 + 2.0 ** -25
            if rise:
                tol += 100 * 64 * 2 * np.exp(-12.0) / (n - 128) * (size * 2.0 ** -22 if size > 100 else 2.0 ** -16)
            worst = (np.abs(got[t] - ref) / tol).max()
            assert worst <= 1.0, (sign, t, worst)


# Half a step of the whole numbers that stand for a row's queries, and for a tile's weights times value scales, to
# the largest of them: numbers below 2^23 (the largest at 0.99 2^22 or more).
HALF_STEP = 2.0 ** -23 / 0.99


@pytest.mark.parametrize("heads", [1, 4, 8, 40])
@pytest.mark.parametrize("dim", [64, 128])
def test_float32_weights_times_value_scales(dim, heads):
    # two keys of one score and nearly one value scale, codes of 100 and -100: the result is the difference of the
    # scales; each product may be off by half a step of the larger one's, the sum, its factor and the
    # division by a few roundings of the small result
    B = 2048
    g = torch.Generator(DEV).manual_seed(dim + heads)
    cache = _cache(B, 1, 16, dim, "f32", code=0, scale=0.0)
    cache.v[:, 0, 0], cache.v[:, 0, 1] = 100, -100
    first = 2.0 ** (20 * torch.rand((B,), device=DEV, generator=g).double() - 10)
    second = first * (1 - 2.0 ** -12 * torch.rand((B,), device=DEV, generator=g).double())
    cache.v_scale[:, 0, 0], cache.v_scale[:, 0, 1] = first.float(), second.float()
    q = torch.randn((B, heads, dim), device=DEV, generator=g)
    got = mnb.mnb_paged_attn_i8(q, cache, torch.arange(B, **I32)[:, None].contiguous(), torch.full((B,), 2, **I32), 2)
    first, second = cache.v_scale[:, 0, 0].double(), cache.v_scale[:, 0, 1].double()
    want = 50 * (first - second)
    tol = 100 * first * HALF_STEP + want.abs() * 2.0 ** -20
    worst = ((got.double() - want[:, None, None]).abs() / tol[:, None, None]).max()
    assert worst <= 1, float(worst)


@pytest.mark.parametrize("heads", [1, 4, 8, 40])
@pytest.mark.parametrize("dim", [64, 128])
def test_float32_queries(dim, heads):
    # rows of one large element, which meets codes of zero, and of small equal ones, which all are off alike:
    # a key of score about one and one of score zero, of values 100 and -100
    B = 2048
    u = 2.0 ** -24
    g = torch.Generator(DEV).manual_seed(dim + heads)
    cache = _cache(B, 1, 16, dim, "f32", code=0, scale=0.0)
    cache.k[:, 0, 0, 1:] = 127
    cache.k_scale[:, 0, :2] = 1.0
    cache.v[:, 0, 0], cache.v[:, 0, 1] = 100, -100
    cache.v_scale[:, 0, :2] = 1.0
    top = 1 + torch.rand((B, heads), device=DEV, generator=g)
    small = (2.0 ** -7 * (1 + torch.rand((B, heads), device=DEV, generator=g)))
    q = small[..., None].repeat(1, 1, dim)
    q[..., 0] = top
    scale = float(np.float32(2.0 ** 6 / (127 * dim)))
    got = mnb.mnb_paged_attn_i8(q, cache, torch.arange(B, **I32)[:, None].contiguous(), torch.full((B,), 2, **I32), 2,
                                scale=scale)
    s = small.double() * (dim - 1) * 127 * scale
    want = 100 * torch.tanh(s / 2)
    # the score moves the result by 50 times as much at most; off by the queries' half steps and float32's
    # roundings; the weights (2^-21 for the exponential, half a step) in numerator and denominator
    off = (dim - 1) * 127 * scale * top.double() * HALF_STEP + (dim + 8) * u * s
    tol = 50 * off + 200 * (2.0 ** -21 + HALF_STEP) + want * 8 * u
    worst = ((got.double() - want[..., None]).abs() / tol[..., None]).max()
    assert worst <= 1, float(worst)
