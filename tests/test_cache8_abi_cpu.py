"""Refusals of the 8-bit cache's, its attention's and the rotary positions'
entry points, on the host: every call returns its documented status before
anything would be enqueued (addresses are placeholders and never dereferenced;
calls with nothing to do return MNB_OK without a launch)."""

import ctypes

import pytest
import torch

from block_wise_int4_amd import mnb

OK, NULL, BITS, BLOCK, SHAPE, DTYPE, ALIGN, HIP, PLAN, INVALID = range(10)
# placeholders far apart: nothing of these sizes meets
A, B, C, D, E, F = (i << 40 for i in range(1, 7))


@pytest.fixture(scope="module")
def L():
    return mnb.lib()


def cache(**change):
    c = dict(k=1 << 20, v=2 << 20, k_scale=3 << 20, v_scale=4 << 20, num_blocks=64, kv_heads=8, page_size=16,
             head_dim=128, block_stride=8 * 16 * 128, head_stride=16 * 128, token_stride=128,
             scale_block_stride=8 * 16, scale_head_stride=16, dtype=1, reserved=0)
    c.update(change)
    return ctypes.byref(mnb.mnb_kv_cache_i8(*[c[f] for f, _ in mnb.mnb_kv_cache_i8._fields_]))


BAD_CACHES = [
    (dict(k=None), NULL), (dict(v=None), NULL), (dict(k_scale=None), NULL), (dict(v_scale=None), NULL),
    (dict(dtype=2), DTYPE), (dict(dtype=-1), DTYPE), (dict(num_blocks=0), SHAPE), (dict(num_blocks=1 << 31), SHAPE),
    (dict(kv_heads=0), SHAPE), (dict(kv_heads=1 << 31), SHAPE), (dict(page_size=0), SHAPE), (dict(page_size=8), SHAPE),
    (dict(page_size=24), SHAPE), (dict(page_size=1040), SHAPE), (dict(page_size=-16), SHAPE),
    (dict(head_dim=80), SHAPE), (dict(head_dim=0), SHAPE), (dict(block_stride=-128), SHAPE),
    (dict(token_stride=1 << 41), SHAPE), (dict(token_stride=(1 << 26) + 16), SHAPE), (dict(head_stride=2056), ALIGN),
    (dict(token_stride=136), ALIGN), (dict(scale_block_stride=-4), SHAPE), (dict(scale_head_stride=1 << 41), SHAPE),
    (dict(scale_block_stride=130), ALIGN), (dict(scale_head_stride=18), ALIGN), (dict(k=(1 << 20) + 8), ALIGN),
    (dict(v=(2 << 20) + 4), ALIGN), (dict(k_scale=(3 << 20) + 4), ALIGN), (dict(v_scale=(4 << 20) + 8), ALIGN),
    (dict(reserved=1), INVALID),
]


@pytest.mark.parametrize("change,status", BAD_CACHES)
def test_cache_descriptions(L, change, status):
    c = cache(**change)
    assert L.mnb_kv_append_i8(A, B, 1024, 1024, C, 4, c, None) == status
    assert L.mnb_kv_read_i8(C, 4, c, A, B, 1024, 1024, None) == status
    assert L.mnb_paged_attn_i8(A, 2048, c, B, C, None, 4, 4, 16 if change.get("kv_heads", 8) else 0, 8, 100, 1, 0.1,
                               None, 0, D, None) == status


TOKENS = [
    (dict(k=None), NULL), (dict(v=None), NULL), (dict(slots=None), NULL), (dict(T=-1), SHAPE),
    (dict(T=0x7FFFFFF1), SHAPE), (dict(ks=-8), SHAPE), (dict(vs=(1 << 40) + 8), SHAPE), (dict(ks=1028), ALIGN),
    (dict(vs=1028), ALIGN), (dict(k=A + 8), ALIGN), (dict(v=B + 2), ALIGN), (dict(slots=C + 4), ALIGN),
    (dict(T=1 << 30, ks=1 << 33), SHAPE), (dict(T=0, k=None, v=None, slots=None), OK),
]


@pytest.mark.parametrize("change,status", TOKENS)
def test_append_and_read_refusals(L, change, status):
    a = dict(k=A, v=B, ks=1024, vs=1024, slots=C, T=4)
    a.update(change)
    assert L.mnb_kv_append_i8(a["k"], a["v"], a["ks"], a["vs"], a["slots"], a["T"], cache(), None) == status
    assert L.mnb_kv_read_i8(a["slots"], a["T"], cache(), a["k"], a["v"], a["ks"], a["vs"], None) == status


@pytest.mark.parametrize("k,ks,v,vs", [
    (A, 1024, A, 1024),                 # one place for both
    (A, 1024, A + 4 * 1024, 1024),      # ranges that meet
    (A, 1000, B, 1024), (A, 1024, B, 0),      # rows nearer than they are long
    (A, 2048, A + 2 * 1000, 2048),      # columns of one buffer that overlap
    (A, 2048, A + 2 * 1024, 3 * 1024),  # strides that differ, within each other's range
])
def test_read_refuses_outputs_that_overlap(L, k, ks, v, vs):
    assert L.mnb_kv_read_i8(C, 4, cache(), k, v, ks, vs, None) == INVALID


def attn(L, q=A, q_stride=2048, desc=None, table=B, lens=C, starts=None, T=4, batch=4, heads=16, width=8, max_len=100,
         max_new=1, scale=0.1, ws=None, ws_bytes=0, out=D):
    return L.mnb_paged_attn_i8(q, q_stride, desc or cache(), table, lens, starts, T, batch, heads, width, max_len,
                               max_new, scale, ws, ws_bytes, out, None)


@pytest.mark.parametrize("change,status", [
    (dict(q=None), NULL), (dict(table=None), NULL), (dict(lens=None), NULL), (dict(out=None), NULL),
    (dict(batch=-1, T=-1), SHAPE), (dict(batch=65537, T=65537), SHAPE), (dict(heads=0), SHAPE), (dict(heads=12), SHAPE),
    (dict(heads=4), SHAPE), (dict(width=0), SHAPE), (dict(width=1 << 30), SHAPE), (dict(max_len=-1), SHAPE),
    (dict(max_len=(1 << 30) + 1), SHAPE), (dict(max_new=0), SHAPE), (dict(max_new=-5, starts=E), SHAPE),
    (dict(max_new=(1 << 30) + 1, starts=E), SHAPE), (dict(max_new=2), SHAPE), (dict(T=5), SHAPE), (dict(T=3), SHAPE),
    (dict(T=-1, starts=E), SHAPE), (dict(T=1 << 31, starts=E), SHAPE), (dict(q_stride=-8), SHAPE),
    (dict(q_stride=2052), ALIGN), (dict(T=1 << 30, starts=E, q_stride=1 << 33), SHAPE),
    (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID), (dict(q=A + 8), ALIGN),
    (dict(out=D + 8), ALIGN), (dict(table=B + 2), ALIGN), (dict(lens=C + 2), ALIGN), (dict(starts=E + 2), ALIGN),
    (dict(out=A), INVALID), (dict(out=A + 3 * 4096), INVALID), (dict(batch=0, T=0), OK),
    (dict(T=0, starts=E, q=None, out=None), OK), (dict(batch=0, T=0, q=None, table=None, lens=None, out=None), OK),
])
def test_attention_refusals(L, change, status):
    assert attn(L, **change) == status


def test_attention_workspace_is_asked_for_and_checked(L):
    need = L.mnb_paged_attn_i8_workspace_bytes(4, 16, 8, 128, 100000, 1, 1)
    if need == 0:
        pytest.skip("nothing is split")
    long = dict(max_len=100000, width=10000)
    assert attn(L, **long) == NULL
    assert attn(L, ws=E, ws_bytes=need - 1, **long) == INVALID
    assert attn(L, ws=E + 8, ws_bytes=need, **long) == ALIGN


def test_workspace_sizes_of_invalid_calls_are_zero(L):
    size = L.mnb_paged_attn_i8_workspace_bytes
    for bad in ((0, 16, 8, 128, 16384, 1, 1), (4, 16, 5, 128, 16384, 1, 1), (4, 16, 8, 96, 16384, 1, 1),
                (4, 16, 8, 128, -1, 1, 1), (4, 16, 8, 128, 16384, 0, 1), (4, 16, 8, 128, 16384, 1, 7),
                (65537, 16, 8, 128, 16384, 1, 1)):
        assert size(*bad) == 0


def rope(L, q=A, q_stride=2048, q_out=B, q_out_stride=2048, q_heads=16, k=C, k_stride=1024, k_out=D, k_out_stride=1024,
         k_heads=8, positions=E, freqs=F, T=4, dim=128, rot=128, layout=0, gain=1.0, dtype=1):
    return L.mnb_rope(q, q_stride, q_out, q_out_stride, q_heads, k, k_stride, k_out, k_out_stride, k_heads, positions,
                      freqs, T, dim, rot, layout, gain, dtype, None)


@pytest.mark.parametrize("change,status", [
    (dict(q=None), NULL), (dict(q_out=None), NULL), (dict(k=None), NULL), (dict(k_out=None), NULL),
    (dict(positions=None), NULL), (dict(freqs=None), NULL), (dict(dtype=3), DTYPE), (dict(T=-1), SHAPE),
    (dict(T=0x7FFFFFF1), SHAPE), (dict(q_heads=-1), SHAPE), (dict(k_heads=1 << 20), SHAPE), (dict(dim=0), SHAPE),
    (dict(dim=1032), SHAPE), (dict(dim=124, rot=124), SHAPE), (dict(rot=0), SHAPE), (dict(rot=63), SHAPE),
    (dict(rot=130), SHAPE), (dict(q_stride=-8), SHAPE), (dict(q_stride=2052), ALIGN), (dict(k_out_stride=1028), ALIGN),
    (dict(T=1 << 30, k_stride=1 << 33), SHAPE), (dict(layout=2), INVALID), (dict(gain=float("nan")), INVALID),
    (dict(gain=float("inf")), INVALID), (dict(q=A + 8), ALIGN), (dict(k_out=D + 2), ALIGN), (dict(positions=E + 2), ALIGN),
    (dict(freqs=F + 4), ALIGN),
    (dict(q_out=A, q_out_stride=4096), INVALID),        # its own place, another stride
    (dict(q_out=A + 4096), INVALID),                    # one token off its own place
    (dict(q_out=A + 64, q_stride=4096, q_out_stride=4096), INVALID), (dict(k_out=B), INVALID), (dict(q_out=C), INVALID),
    (dict(q_out_stride=2040), INVALID), (dict(k_out_stride=0), INVALID),
    (dict(T=0), OK), (dict(q_heads=0, k_heads=0), OK), (dict(T=0, q=None, k=None, positions=None), OK),
])
def test_rope_refusals(L, change, status):
    assert rope(L, **change) == status


def test_struct_layout_matches_the_header():
    # four pointers, nine 64-bit counts, two 32-bit fields
    assert ctypes.sizeof(mnb.mnb_kv_cache_i8) == 4 * 8 + 9 * 8 + 8


def test_binding_checks_tensors():
    codes, scales = torch.zeros(2, 8, 16, 128, dtype=torch.int8), torch.zeros(2, 8, 16)
    with pytest.raises(ValueError, match="on the GPU"):
        mnb.KvCacheI8(codes, codes, scales, scales, torch.float16)
    with pytest.raises(ValueError, match="unsupported dtype"):
        mnb.KvCacheI8(codes, codes, scales, scales, torch.bfloat16)
    with pytest.raises(ValueError, match="k must be torch.int8"):
        mnb.KvCacheI8(codes.half(), codes, scales, scales, torch.float16)
    with pytest.raises(ValueError, match="v_scale must be torch.float32"):
        mnb.KvCacheI8(codes, codes, scales, scales.half(), torch.float16)
    with pytest.raises(ValueError, match="contiguous"):
        mnb.KvCacheI8(codes, codes, scales.transpose(1, 2), scales, torch.float16)
    q, pos, freqs = torch.zeros(3, 2, 64), torch.zeros(3, dtype=torch.int32), torch.zeros(32, dtype=torch.float64)
    with pytest.raises(ValueError, match="on the GPU"):
        mnb.mnb_rope(q, None, pos, freqs)
    with pytest.raises(ValueError, match="q or k"):
        mnb.mnb_rope(None, None, pos, freqs)
    with pytest.raises(ValueError, match="positions has 3 elements"):
        mnb.mnb_rope(q[:2], None, pos, freqs)
    with pytest.raises(ValueError, match="freqs must be torch.float64"):
        mnb.mnb_rope(q, None, pos, freqs.float())
    with pytest.raises(ValueError, match="k must be"):
        mnb.mnb_rope(q, q[:2], pos, freqs)
    with pytest.raises(ValueError, match="contiguous heads"):
        mnb.mnb_rope(q.transpose(0, 1), None, pos[:2], freqs)
    with pytest.raises(ValueError, match="q_out must have"):
        mnb.mnb_rope(q, None, pos, freqs, q_out=q[:, :1])
    with pytest.raises(ValueError, match="unsupported dtype"):
        mnb.mnb_rope(q.bfloat16(), None, pos, freqs)
