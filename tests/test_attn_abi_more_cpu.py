"""More of the attention entry points' C ABI, on the host (see
test_attn_abi_cpu): calls that must not be refused are told by their status,
MNB_OK or, without a GPU to launch on, MNB_ERR_HIP."""

import ctypes

import pytest
import torch

from test_attn_abi_cpu import A, B, C, D, E, INVALID, OK, HIP, L, tables  # noqa: F401 (L is a fixture)

no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="the addresses are placeholders: nothing may be launched")


def at(base, nbytes):
    return ctypes.c_void_p(base.value + nbytes)


@no_gpu
@pytest.mark.parametrize("change", [
    dict(slots=at(D, 16), T=0), dict(slots=at(A, 8), T=0),          # no slots, at an address inside another array
    dict(free=at(D, 16), n_free=0), dict(free=at(E, 8), n_free=0),  # no free blocks
])
def test_tables_empty_arrays_overlap_nothing(L, change):  # noqa: F811
    args = dict(cached=A, added=B, free=C, table=D, lens=E, starts=at(A, 4096), slots=at(B, 4096), taken=at(C, 4096))
    assert tables(L, **{**args, **change}) in (OK, HIP)


def test_tables_arrays_that_overlap_are_still_refused(L):  # noqa: F811
    args = dict(cached=A, added=B, free=C, table=D, lens=E, starts=at(A, 4096), slots=at(B, 4096), taken=at(C, 4096))
    assert tables(L, **{**args, "slots": at(D, 16), "T": 1}) == INVALID
    assert tables(L, **{**args, "free": at(D, 16), "n_free": 1}) == INVALID


def test_package_exports_what_an_attention_step_calls():
    import block_wise_int4_amd as package
    for name in ("KvCache", "mnb_kv_tables", "mnb_kv_append", "mnb_paged_attn", "mnb_cross_attn",
                 "mnb_paged_attn_workspace_bytes", "mnb_cross_attn_workspace_bytes", "paged_attn_workspace",
                 "cross_attn_workspace"):
        assert getattr(package, name) is getattr(package.mnb, name), name
