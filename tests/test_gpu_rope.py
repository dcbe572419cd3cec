"""GPU: rotary positions against the float64 oracle.

Tolerance per output, from the formula: the fraction of a turn, at most a half,
is rounded to float32 (2^-26 turns: 2 pi 2^-26 radians at most), its float64
product and reduction add 2^-51 of the angle, cosine, sine, gain and the two
terms of the sum a few float32 roundings (2^-21 covers ten), each on terms of
size gain (|x0| + |x1|); and the output is rounded to its type (half of
finfo.eps, 2^-25 absolute for float16's subnormals).
"""

import numpy as np
import pytest
import torch

import oracle
from block_wise_int4_amd import mnb

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
TD = {"f16": torch.float16, "f32": torch.float32}


def _np(t):
    return t.cpu().double().numpy()


def _check(got, x, positions, freqs, interleaved, gain, what=""):
    x, got, pos, f = _np(x), _np(got), positions.cpu().numpy().astype(np.int64), _np(freqs)
    ref = oracle.rope(x, pos, f, interleaved, gain)
    size = np.abs(oracle.rope(np.abs(x), pos * 0, f * 0, interleaved, 1.0))
    half = len(f)
    a = np.arange(half) * 2 if interleaved else np.arange(half)
    b = a + 1 if interleaved else a + half
    pair = size[..., a] + size[..., b]
    angle = np.abs(pos[:, None] * f[None, :])
    rel = 2 * np.pi * 2.0 ** -26 + angle * 2.0 ** -51 + 2.0 ** -21
    tol = np.zeros(x.shape)
    for d in (a, b):
        tol[..., d] = abs(gain) * pair * rel[:, None, :]
    eps = 2.0 ** -11 if what.startswith("f16") else 2.0 ** -24
    rounded = np.zeros(x.shape)
    rounded[..., : 2 * half] = np.abs(ref[..., : 2 * half]) * eps + (2.0 ** -25 if eps > 2.0 ** -20 else 2.0 ** -149)
    worst = np.max(np.abs(got - ref) - (tol + rounded), initial=-1.0)
    assert np.isfinite(got).all() and worst <= 0, f"{what}: {worst} past the bound"
    assert np.array_equal(got[..., 2 * half:], x[..., 2 * half:]), what


@pytest.mark.parametrize("interleaved", [False, True], ids=["half", "interleaved"])
@pytest.mark.parametrize("dt,dim,rot", [("f16", 128, 128), ("f16", 64, 32), ("f16", 128, 20), ("f32", 64, 64),
                                        ("f32", 128, 64), ("f32", 4, 2), ("f16", 80, 80), ("f32", 1024, 1024),
                                        ("f16", 72, 24), ("f16", 256, 10)])
def test_rope(dt, dim, rot, interleaved):
    for T, heads, kv in ((1, 16, 8), (7, 3, 1), (130, 12, 12)):
        print(f"rope {dt} T={T} heads={heads}/{kv} dim={dim} rot={rot} interleaved={interleaved}", flush=True)
        g = torch.Generator(DEV).manual_seed(T + dim)
        fused = torch.randn((T, (heads + 2 * kv) * dim), device=DEV, generator=g).to(TD[dt])
        q = fused[:, : heads * dim].view(T, heads, dim)
        k = fused[:, heads * dim: (heads + kv) * dim].view(T, kv, dim)
        pos = torch.randint(0, 40000, (T,), device=DEV, generator=g, dtype=torch.int32)
        pos[0] = 0 if T > 1 else 5
        freqs, _ = mnb.rope_frequencies(rot, 1e4, device=DEV)
        before = fused.clone()
        qo, ko = mnb.mnb_rope(q, k, pos, freqs, interleaved=interleaved)
        torch.cuda.synchronize()
        assert torch.equal(fused, before)
        _check(qo, q, pos, freqs, interleaved, 1.0, f"{dt} q")
        _check(ko, k, pos, freqs, interleaved, 1.0, f"{dt} k")
        # in place, beside the values
        mnb.mnb_rope(q, k, pos, freqs, interleaved=interleaved, q_out=q, k_out=k)
        torch.cuda.synchronize()
        assert torch.equal(q, qo) and torch.equal(k, ko)
        assert torch.equal(fused[:, (heads + kv) * dim:], before[:, (heads + kv) * dim:])
        # one of the two
        assert torch.equal(mnb.mnb_rope(None, before[:, heads * dim: (heads + kv) * dim].view(T, kv, dim), pos, freqs,
                                        interleaved=interleaved)[1], ko)


@pytest.mark.parametrize("dt", ["f16", "f32"])
def test_far_and_negative_positions_and_gains(dt):
    pos = torch.tensor([2 ** 31 - 1, -2 ** 31, 2 ** 30, -1, 1, 999999, 0], dtype=torch.int32, device=DEV)
    x = torch.randn((7, 2, 128), device=DEV).to(TD[dt])
    for kw in (dict(base=1e6, linear=2.5), dict(stretch=8.0), dict(by_parts=(4.0, 2048, 1.0, 32.0))):
        freqs, gain = mnb.rope_frequencies(128, device=DEV, **kw)
        for g in (gain, -2.0, 0.0):
            _check(mnb.mnb_rope(x, None, pos, freqs, gain=g)[0], x, pos, freqs, False, g, f"{dt} {kw} {g}")
    # turned and turned back
    freqs, _ = mnb.rope_frequencies(128, device=DEV)
    there = mnb.mnb_rope(x, None, pos // 2, freqs)[0]
    back = mnb.mnb_rope(there, None, -(pos // 2), freqs)[0]
    # two calls, each off by half a step of its output and 2^-20 of the pair, sizes up to |x0| + |x1|
    pair = x.float().abs()[..., :64] + x.float().abs()[..., 64:]
    off = (back.float() - x.float()).abs()
    assert (off <= (torch.finfo(TD[dt]).eps * 2 + 2.0 ** -18) * torch.cat((pair, pair), dim=-1)).all()


@pytest.mark.parametrize("dt,dim,rot", [("f16", 128, 64), ("f16", 128, 20)])
def test_infinities_and_nan_stay_in_their_pairs(dt, dim, rot):
    x = torch.ones((1, 3, dim), device=DEV).to(TD[dt])
    x[0, 0, 3], x[0, 1, 3], x[0, 2, dim - 1] = float("inf"), float("nan"), float("inf")
    pos = torch.tensor([1], dtype=torch.int32, device=DEV)
    y = mnb.mnb_rope(x, None, pos, mnb.rope_frequencies(rot, device=DEV)[0])[0]
    bad = (~torch.isfinite(y[0])).nonzero().tolist()
    assert bad == [[0, 3], [0, 3 + rot // 2], [1, 3], [1, 3 + rot // 2], [2, dim - 1]]


def test_many_heads_and_empty_calls():
    freqs = mnb.rope_frequencies(64, device=DEV)[0]
    x = torch.randn((3, 400, 64), device=DEV).half()
    pos = torch.tensor([3, 70, 7], dtype=torch.int32, device=DEV)
    _check(mnb.mnb_rope(x, None, pos, freqs)[0], x, pos, freqs, False, 1.0, "f16 400 heads")
    q, k = mnb.mnb_rope(x[:0], x[:0], pos[:0], freqs)
    assert q.shape == k.shape == (0, 400, 64)


def test_on_another_stream_and_replayed():
    freqs = mnb.rope_frequencies(128, device=DEV)[0]
    x = torch.randn((9, 24, 128), device=DEV).half()
    pos = torch.arange(9, dtype=torch.int32, device=DEV)
    want = mnb.mnb_rope(x, None, pos, freqs)[0]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = mnb.mnb_rope(x, None, pos, freqs)[0]
    s.synchronize()
    assert torch.equal(got, want)
    out = torch.empty_like(x)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        mnb.mnb_rope(x, None, pos, freqs, q_out=out)
    for step in range(3):
        pos += 1
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, mnb.mnb_rope(x, None, pos, freqs)[0])
