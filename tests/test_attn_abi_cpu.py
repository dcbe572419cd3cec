"""Refusals of the attention entry points' C ABI, on the host: every call
returns its documented status before anything would be enqueued (addresses
are placeholders and never dereferenced; calls with nothing to do return
MNB_OK without a launch)."""

import ctypes

import pytest

from block_wise_int4_amd import mnb

OK, NULL, BITS, BLOCK, SHAPE, DTYPE, ALIGN, HIP, PLAN, INVALID = range(10)
A, B, C, D, E = (ctypes.c_void_p(i << 20) for i in range(1, 6))
ODD = ctypes.c_void_p((1 << 20) + 8)
ODD2 = ctypes.c_void_p((1 << 20) + 2)


@pytest.fixture(scope="module")
def L():
    return mnb.lib()


def cache(**change):
    c = dict(k=1 << 20, v=2 << 20, num_blocks=64, kv_heads=8, page_size=16, head_dim=128, block_stride=8 * 16 * 128,
             head_stride=16 * 128, token_stride=128, dtype=1, reserved=0)
    c.update(change)
    return ctypes.byref(mnb.mnb_kv_cache(*[c[f] for f, _ in mnb.mnb_kv_cache._fields_]))


BAD_CACHES = [
    (dict(k=None), NULL), (dict(v=None), NULL), (dict(dtype=2), DTYPE), (dict(dtype=-1), DTYPE),
    (dict(num_blocks=0), SHAPE), (dict(num_blocks=1 << 31), SHAPE), (dict(kv_heads=0), SHAPE),
    (dict(page_size=0), SHAPE), (dict(page_size=8), SHAPE), (dict(page_size=24), SHAPE),
    (dict(page_size=1040), SHAPE), (dict(page_size=-16), SHAPE), (dict(head_dim=80), SHAPE), (dict(head_dim=0), SHAPE),
    (dict(block_stride=-128), SHAPE), (dict(token_stride=1 << 41), SHAPE), (dict(head_stride=2052), ALIGN),
    (dict(token_stride=4), ALIGN), (dict(k=(1 << 20) + 8), ALIGN), (dict(v=(2 << 20) + 4), ALIGN),
    (dict(reserved=1), INVALID),
]


@pytest.mark.parametrize("change,status", BAD_CACHES)
def test_cache_descriptions(L, change, status):
    c = cache(**change)
    assert L.mnb_kv_append(A, B, 1024, 1024, C, 4, c, None) == status
    assert L.mnb_paged_attn(A, 2048, c, B, C, 4, 16 if change.get("kv_heads", 8) else 0, 8, 100, 0.1, None, 0, D,
                            None) == status


def tables(L, cached=A, added=B, free=C, n_free=10, batch=4, page=16, width=8, T=9, table=D, lens=E, starts=A, slots=B,
           taken=C):
    return L.mnb_kv_tables(cached, added, free, n_free, batch, page, width, T, table, lens, starts, slots, taken, None)


@pytest.mark.parametrize("change,status", [
    (dict(cached=None), NULL), (dict(added=None), NULL), (dict(free=None), NULL), (dict(table=None), NULL),
    (dict(lens=None), NULL), (dict(starts=None), NULL), (dict(slots=None), NULL), (dict(taken=None), NULL),
    (dict(batch=-1), SHAPE), (dict(batch=65537), SHAPE), (dict(n_free=-1), SHAPE), (dict(T=-1), SHAPE),
    (dict(T=0x7FFFFFF1), SHAPE), (dict(page=0), SHAPE), (dict(page=20), SHAPE), (dict(page=2048), SHAPE),
    (dict(width=0), SHAPE), (dict(width=(1 << 30) // 16 + 1), SHAPE), (dict(batch=65536, width=1 << 15), SHAPE),
    (dict(cached=ODD2), ALIGN), (dict(added=ODD2), ALIGN), (dict(free=ODD2), ALIGN), (dict(table=ODD2), ALIGN),
    (dict(lens=ODD2), ALIGN), (dict(starts=ODD2), ALIGN), (dict(taken=ODD2), ALIGN),
    (dict(slots=ctypes.c_void_p((1 << 20) + 4)), ALIGN),
])
def test_tables_refusals(L, change, status):
    assert tables(L, **change) == status


@pytest.mark.parametrize("args,status", [
    ((None, B, 1024, 1024, C, 4), NULL), ((A, None, 1024, 1024, C, 4), NULL), ((A, B, 1024, 1024, None, 4), NULL),
    ((A, B, 1024, 1024, C, -1), SHAPE), ((A, B, 1024, 1024, C, 0x7FFFFFF1), SHAPE), ((A, B, -8, 1024, C, 4), SHAPE),
    ((A, B, 1028, 1024, C, 4), ALIGN), ((ODD, B, 1024, 1024, C, 4), ALIGN), ((A, ODD, 1024, 1024, C, 4), ALIGN),
    ((A, B, 1024, 1024, ctypes.c_void_p((1 << 20) + 4), 4), ALIGN), ((None, None, 0, 0, None, 0), OK),
])
def test_append_refusals(L, args, status):
    assert L.mnb_kv_append(*args, cache(), None) == status


def paged(L, q=A, q_stride=2048, desc=None, table=B, lens=C, batch=4, heads=16, width=8, max_len=100, scale=0.1,
          ws=None, ws_bytes=0, out=D):
    return L.mnb_paged_attn(q, q_stride, desc or cache(), table, lens, batch, heads, width, max_len, scale, ws,
                            ws_bytes, out, None)


@pytest.mark.parametrize("change,status", [
    (dict(q=None), NULL), (dict(table=None), NULL), (dict(lens=None), NULL), (dict(out=None), NULL),
    (dict(batch=-1), SHAPE), (dict(batch=65537), SHAPE), (dict(heads=0), SHAPE), (dict(heads=12), SHAPE),
    (dict(heads=4), SHAPE), (dict(width=0), SHAPE), (dict(width=1 << 30), SHAPE), (dict(max_len=-1), SHAPE),
    (dict(max_len=(1 << 30) + 1), SHAPE), (dict(q_stride=-8), SHAPE), (dict(q_stride=2052), ALIGN),
    (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID), (dict(q=ODD), ALIGN),
    (dict(out=ODD), ALIGN), (dict(table=ODD2), ALIGN), (dict(lens=ODD2), ALIGN), (dict(batch=0), OK),
    (dict(batch=0, q=None, table=None, lens=None, out=None), OK),
])
def test_paged_refusals(L, change, status):
    assert paged(L, **change) == status


def view(data=1 << 20, batch=1500 * 768, row=768, head=64):
    return ctypes.byref(mnb.mnb_attn_view(data, batch, row, head))


def cross(L, q=True, k=True, v=True, out=True, lens=None, batch=4, queries=3, keys=1500, heads=12, kv_heads=12, dim=64,
          scale=0.1, dtype=1, ws=None, ws_bytes=0):
    q, k, v, out = (view() if t is True else t for t in (q, k, v, out))
    return L.mnb_cross_attn(q, k, v, lens, batch, queries, keys, heads, kv_heads, dim, scale, dtype, ws, ws_bytes, out,
                            None)


@pytest.mark.parametrize("change,status", [
    (dict(q=None), NULL), (dict(k=None), NULL), (dict(v=None), NULL), (dict(out=None), NULL),
    (dict(q=view(None)), NULL), (dict(k=view(None)), NULL), (dict(v=view(None)), NULL), (dict(out=view(None)), NULL),
    (dict(batch=-1), SHAPE), (dict(batch=65537), SHAPE), (dict(queries=-1), SHAPE), (dict(queries=0x7FFFFFF1), SHAPE),
    (dict(keys=-1), SHAPE), (dict(keys=(1 << 30) + 1), SHAPE), (dict(heads=0), SHAPE), (dict(kv_heads=0), SHAPE),
    (dict(heads=12, kv_heads=5), SHAPE), (dict(heads=6), SHAPE), (dict(dim=96), SHAPE), (dict(dtype=2), DTYPE),
    (dict(batch=65536, queries=0x7FFFFFF0, heads=1 << 30, kv_heads=1 << 30), SHAPE),
    (dict(queries=0x7FFFFFF0, heads=64, kv_heads=1), SHAPE),
    (dict(scale=float("-inf")), INVALID), (dict(q=view(row=-64)), SHAPE), (dict(k=view(head=68)), ALIGN),
    (dict(v=view(batch=1 << 41)), SHAPE), (dict(out=view(row=772)), ALIGN), (dict(q=view((1 << 20) + 8)), ALIGN),
    (dict(out=view((1 << 20) + 4)), ALIGN), (dict(lens=ODD2), ALIGN), (dict(batch=0), OK), (dict(queries=0), OK),
])
def test_cross_refusals(L, change, status):
    assert cross(L, **change) == status


def test_workspace_sizes_of_invalid_calls_are_zero(L):
    assert L.mnb_paged_attn_workspace_bytes(0, 16, 8, 128, 16384, 1) == 0
    assert L.mnb_paged_attn_workspace_bytes(4, 16, 5, 128, 16384, 1) == 0
    assert L.mnb_paged_attn_workspace_bytes(4, 16, 8, 96, 16384, 1) == 0
    assert L.mnb_paged_attn_workspace_bytes(4, 16, 8, 128, -1, 1) == 0
    assert L.mnb_paged_attn_workspace_bytes(4, 16, 8, 128, 16384, 7) == 0
    assert L.mnb_cross_attn_workspace_bytes(4, 0, 1500, 12, 12, 64, 1) == 0
    assert L.mnb_cross_attn_workspace_bytes(4, 1, 1500, 12, 0, 64, 1) == 0


def test_struct_layouts_match_the_header():
    # eight pointers or 64-bit counts, then two 32-bit fields
    assert ctypes.sizeof(mnb.mnb_kv_cache) == 9 * 8 + 8
    assert ctypes.sizeof(mnb.mnb_attn_view) == 4 * 8


def test_binding_checks_tensors():
    import torch
    half = torch.zeros(2, 8, 16, 128, dtype=torch.float16)
    with pytest.raises(ValueError, match="on the GPU"):
        mnb.KvCache(half, half)
    with pytest.raises(ValueError, match="must be torch.float16"):
        mnb.KvCache(half, half.float())
    with pytest.raises(ValueError, match="unsupported dtype"):
        mnb.KvCache(half.bfloat16(), half.bfloat16())
    with pytest.raises(ValueError, match="contiguous"):
        mnb.KvCache(half.transpose(2, 3), half.transpose(2, 3))
    i = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError, match="elements"):
        mnb.mnb_kv_tables(i, i[:3], i, i.view(4, 1), 16, torch.zeros(1, dtype=torch.int64))
    with pytest.raises(ValueError, match="must be torch.int64"):
        mnb.mnb_kv_tables(i, i, i, i.view(4, 1), 16, i)
    with pytest.raises(ValueError, match="max_blocks"):
        mnb.mnb_kv_tables(i, i, i, i, 16, torch.zeros(1, dtype=torch.int64))
    q = torch.zeros(1, 1, 12, 64, dtype=torch.float16)
    with pytest.raises(ValueError, match="on the GPU"):
        mnb.mnb_cross_attn(q, q, q)
