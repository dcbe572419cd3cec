"""GPU: attention over the 8-bit cache with scales that no float16 row gets by being
appended, which callers may write.
"""

import numpy as np
import pytest
import torch

from block_wise_int4_amd import mnb
from test_gpu_cache8 import DEV, _at, _case, _check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("new", [None, [20], [60], [130]], ids=str)
@pytest.mark.parametrize("exponent", [58, 60, 67, 68, 69, 100, 121])
def test_value_scales_past_float16(exponent, new):
    # a key of ordinary weight whose values are 2^exponent times its codes, half of them zero: infinity, the
    # largest float16 passed, where there is a code, and where there is none the other keys' sum, which may
    # count as zero beside it
    keys = 300
    n = new[0] if new else 1
    for at in (0, 100, keys - 10):
        q, cache, table, ln, starts = _case(71, [keys], 2, 1, 64, 16, "f16", new=new)
        clean = mnb.mnb_paged_attn_i8(q, cache, table, ln, keys, starts=starts, max_new=n)
        most = float((cache.v.abs() * cache.v_scale.nan_to_num(0, 0, 0)[..., None]).amax())
        where = _at(table, 16, 0, at)
        cache.v[where] = torch.tensor([1, 0, -3, 0] * 16, dtype=torch.int8, device=DEV)
        cache.v_scale[where] = 2.0 ** exponent
        got = mnb.mnb_paged_attn_i8(q, cache, table, ln, keys, starts=starts, max_new=n)
        sees = [t for t in range(n) if keys - n + t >= at]
        assert torch.equal(got[: n - len(sees)], clean[: n - len(sees)])
        part = got[n - len(sees):]
        assert (part[..., 0::4] == float("inf")).all() and (part[..., 2::4] == -float("inf")).all(), at
        assert torch.isfinite(part[..., 1::2]).all() and (part[..., 1::2].abs() <= most).all(), at


@pytest.mark.parametrize("new", [None, [20], [60]], ids=str)
@pytest.mark.parametrize("exponent", [68, 100, 121])
def test_large_value_scales_of_little_weight(exponent, new):
    # the same key's score so far below that its values are ordinary ones
    keys = 300
    n = new[0] if new else 1
    for at in (0, 100, keys - 70):
        for left in (-60, -10, 0, 5):    # its term's power of two
            q, cache, table, ln, starts = _case(72, [keys], 2, 1, 64, 16, "f16", new=new)
            cache.k.zero_()
            q.abs_().add_(0.5)
            q.fill_(1.0)
            where = _at(table, 16, 0, at)
            cache.k[where] = -127
            cache.k_scale[where] = (exponent - left) * np.log(2) / 127 / 8
            cache.v[where] = torch.tensor([1, 0, -3, 0] * 16, dtype=torch.int8, device=DEV)
            cache.v_scale[where] = 2.0 ** exponent
            got = mnb.mnb_paged_attn_i8(q, cache, table, ln, keys, starts=starts, max_new=n)
            _check(got, q, cache, table, ln, starts, keys, n, "f16", what=f"key {at}, 2^{left}")


@pytest.mark.parametrize("new", [None, [3], [40]], ids=str)
@pytest.mark.parametrize("size,keys_size,scale", [
    (2e-38, 1e38, 0.5), (1e-36, 1e34, 3.0), (3e-34, 1e36, 1 / 300), (3e-39, 1e38, 3.0), (1e38, 1e-41, 1 / 300),
    (1e-30, 1e-10, 1e38), (1e-42, 1e4, 3e38), (3e37, 1e-10, 1e-27),
    (3.4e38, 3e-38, 1 / 30), (3.4e38, 1e-10, 1e-28)])
def test_float32_products_of_far_sizes(size, keys_size, scale, new):
    # queries and keys whose products are ordinary numbers
    q, cache, table, ln, starts = _case(73, [90], 2, 1, 64, 16, "f32", new=new)
    n = new[0] if new else 1
    q = (q / q.abs().amax()).double().mul(size).float()
    ok = torch.isfinite(cache.k_scale)
    most = float((cache.k.abs().amax(dim=-1) * cache.k_scale.where(ok, torch.zeros_like(cache.k_scale))).amax())
    cache.k_scale.copy_(torch.where(ok, (cache.k_scale.double() / most * keys_size).float(), cache.k_scale))
    where = _at(table, 16, 0, 7)
    cache.k_scale[where], cache.k[where] = 0.0, 0      # a key of zeros among them
    got = mnb.mnb_paged_attn_i8(q, cache, table, ln, 90, starts=starts, max_new=n, scale=scale)
    _check(got, q, cache, table, ln, starts, 90, n, "f32", scale, f"{size} x {keys_size}")
