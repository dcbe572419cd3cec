"""GPU: a refused attention call enqueues nothing: the outputs it was given stay
as they were."""

import pytest
import torch

import test_gpu_attn as base
from block_wise_int4_amd import mnb

pytestmark = pytest.mark.gpu

DEV, NAN = base.DEV, float("nan")
I32 = dict(dtype=torch.int32, device=DEV)


def _refused(calls, outputs):
    before = [t.clone() for t in outputs]
    for name, call in calls.items():
        print(name, flush=True)
        with pytest.raises((ValueError, mnb.MnbError)):
            call()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(before, outputs)), name


def test_refused_paged_calls_leave_the_output():
    q, cache, table, ln = base._paged_case(21, [40, 9], 4, 2, 64, 16, "f16")
    long_q, long_cache, long_table, long_ln = base._paged_case(22, [9000], 2, 2, 64, 64, "f16")
    need = mnb.mnb_paged_attn_workspace_bytes(1, 2, long_cache, 9000)
    assert need > 0
    out, long_out = torch.full_like(q, 3.0), torch.full_like(long_q, 3.0)
    bytes_ = lambda n: torch.empty(n, dtype=torch.uint8, device=DEV)  # noqa: E731
    _refused({
        "query type": lambda: mnb.mnb_paged_attn(q.float(), cache, table, ln, 40, out=out),
        "heads": lambda: mnb.mnb_paged_attn(q[:, :3].contiguous(), cache, table, ln, 40, out=out[:, :3].contiguous()),
        "bound": lambda: mnb.mnb_paged_attn(q, cache, table, ln, -1, out=out),
        "scale": lambda: mnb.mnb_paged_attn(q, cache, table, ln, 40, scale=NAN, out=out),
        "table type": lambda: mnb.mnb_paged_attn(q, cache, table.long(), ln, 40, out=out),
        "lengths": lambda: mnb.mnb_paged_attn(q, cache, table, ln[:1], 40, out=out),
        "output size": lambda: mnb.mnb_paged_attn(q[:1], cache, table[:1], ln[:1], 40, out=out),
        "small workspace": lambda: mnb.mnb_paged_attn(long_q, long_cache, long_table, long_ln, 9000,
                                                      workspace=bytes_(need - 1), out=long_out),
        "no workspace": lambda: mnb.mnb_paged_attn(long_q, long_cache, long_table, long_ln, 9000,
                                                   workspace=bytes_(0), out=long_out),
        "workspace off by 8": lambda: mnb.mnb_paged_attn(long_q, long_cache, long_table, long_ln, 9000,
                                                         workspace=bytes_(need + 16)[8:], out=long_out),
    }, [out, long_out])


@pytest.mark.parametrize("dt", ["f16", "f32"])
def test_refused_cross_calls_leave_the_output(dt):
    q, k, v = base._cross_case(23, 2, 3, 20, 4, 2, 64, dt)
    ln = torch.tensor([20, 5], **I32)
    out = torch.full_like(q, 3.0)
    wide = torch.zeros((2, 3, 4, 68), dtype=q.dtype, device=DEV)
    _refused({
        "key type": lambda: mnb.mnb_cross_attn(q, k.double(), v, ln, out=out),
        "value rows": lambda: mnb.mnb_cross_attn(q, k, v[:, :19], ln, out=out),
        "requests": lambda: mnb.mnb_cross_attn(q, k[:1], v[:1], ln, out=out),
        "lengths": lambda: mnb.mnb_cross_attn(q, k, v, ln[:1], out=out),
        "scale": lambda: mnb.mnb_cross_attn(q, k, v, ln, scale=float("inf"), out=out),
        "heads": lambda: mnb.mnb_cross_attn(q[:, :, :3].contiguous(), k, v, ln, out=out[:, :, :3]),
        "output shape": lambda: mnb.mnb_cross_attn(q, k, v, ln, out=out[:, :2]),
        "alignment": lambda: mnb.mnb_cross_attn(wide[..., 2:66], k, v, ln, out=out),
    }, [out])


def test_refused_tables_and_append_calls_leave_their_outputs():
    cached, added, free = (torch.tensor(t, **I32) for t in ([5, 16], [1, 1], [3, 4]))
    table, slots = torch.tensor([[1, -1], [2, -1]], **I32), torch.full((2,), 9, dtype=torch.int64, device=DEV)
    lens, starts, taken = torch.full((2,), 7, **I32), torch.full((3,), 7, **I32), torch.full((1,), 7, **I32)
    outs = dict(lens=lens, starts=starts, taken=taken)
    cache = mnb.KvCache(*(torch.full((4, 2, 16, 64), 0.5, dtype=torch.float16, device=DEV) for _ in range(2)))
    k = torch.ones((2, 2, 64), dtype=torch.float16, device=DEV)
    _refused({
        "page": lambda: mnb.mnb_kv_tables(cached, added, free, table, 24, slots, **outs),
        "lengths over the cached ones": lambda: mnb.mnb_kv_tables(cached, added, free, table, 16, slots,
                                                                  **{**outs, "lens": cached}),
        "counts": lambda: mnb.mnb_kv_tables(cached, added[:1], free, table, 16, slots, **outs),
        "slot type": lambda: mnb.mnb_kv_tables(cached, added, free, table, 16, slots.int(), **outs),
        "token count": lambda: mnb.mnb_kv_append(k, k[:1], slots, cache),
        "token type": lambda: mnb.mnb_kv_append(k.float(), k, slots, cache),
        "token heads": lambda: mnb.mnb_kv_append(k[:, :1], k, slots, cache),
        "slots": lambda: mnb.mnb_kv_append(k, k, slots.int(), cache),
    }, [table, slots, lens, starts, taken, cached, cache.k, cache.v])
