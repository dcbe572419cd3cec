"""How the attention over the 8-bit cache decides whether rows of keys stay whole: by what
the longest has over a CU's share, which changes little from one request to the next
(CPU only: a call that cuts nothing needs no workspace)."""

import pytest

from block_wise_int4_amd import mnb


def _longest(B, heads, kv_heads, dim):
    """The most keys a request may have so that its rows stay whole."""
    lo, hi = 0, 1 << 20
    while lo < hi:
        mid = (lo + hi + 1) // 2
        whole = mnb.lib().mnb_paged_attn_i8_workspace_bytes(B, heads, kv_heads, dim, mid, 1, mnb.MNB_F32) == 0
        lo, hi = (mid, hi) if whole else (lo, mid - 1)
    return lo


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("group", [1, 2, 3, 8, 16])
def test_the_longest_whole_row_grows_with_the_requests(group, dim):
    longest = [_longest(B, group, 1, dim) for B in range(1, 400)]
    assert all(a <= b for a, b in zip(longest, longest[1:]))
    # up to three quarters of the CUs a request more moves it by 1 in 64 at most (and a step of 512 keys, which a
    # workgroup's tiles are rounded to)
    assert all(b <= a * (1 + 1 / 64) + 512 for a, b in zip(longest[:192], longest[1:192]))
    # from a row a CU on, all rows of up to a megabyte
    assert set(longest[255:]) == {(1 << 20) // (2 * dim)}
    assert longest[0] <= (128 << 10) * 256 // 255 // (2 * dim)      # one row, all over its share: a join's time


def test_rows_of_a_prompt_are_counted_too():
    # 16 requests of 12 heads, and one request of 16 tokens of 12: the same rows of tiles
    need = mnb.lib().mnb_paged_attn_i8_workspace_bytes
    for keys in (700, 1500, 4000):
        assert (need(192, 16, 1, 64, keys, 1, mnb.MNB_F32) == 0) == (need(1, 192, 192, 64, keys, 16, mnb.MNB_F32) == 0)
