"""GPU: rotary positions of more tokens than one launch takes (its threads, 64 a token,
are counted in 32 bits)."""

import pytest
import torch

from block_wise_int4_amd import mnb
from test_gpu_rope import DEV, _check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tokens,dt,dim,rot,interleaved", [
    ((1 << 25) + 3, torch.float16, 8, 6, False),        # one launch and the rest
    ((1 << 26) + 77, torch.float32, 4, 4, True),        # past 2^32 threads
    ((1 << 26) + (1 << 20) + 5, torch.float16, 8, 8, False)])
def test_more_tokens_than_a_launch_takes(tokens, dt, dim, rot, interleaved):
    print(f"rope {dt} T={tokens} dim={dim} rot={rot}", flush=True)
    g = torch.Generator(DEV).manual_seed(rot)
    q = torch.randn((tokens, 1, dim), device=DEV, generator=g, dtype=dt)
    k = torch.randn((tokens, 1, dim), device=DEV, generator=g, dtype=dt)
    pos = torch.randint(0, 40000, (tokens,), device=DEV, generator=g, dtype=torch.int32)
    freqs, _ = mnb.rope_frequencies(rot, 1e4, device=DEV)
    q_out, k_out = mnb.mnb_rope(q, k, pos, freqs, interleaved=interleaved)
    torch.cuda.synchronize()
    name = "f16" if dt == torch.float16 else "f32"
    # the places around whole launches against the oracle, all of them against calls of fewer tokens
    for at in (0, (1 << 24) - 4, (1 << 25) - 4, (1 << 26) - 4, tokens - 9):
        at = slice(at, min(at + 9, tokens))
        _check(q_out[at], q[at], pos[at], freqs, interleaved, 1.0, f"{name} {at}")
        _check(k_out[at], k[at], pos[at], freqs, interleaved, 1.0, f"{name} {at}")
    for at in range(0, tokens, 10000000):
        at = slice(at, at + 10000000)
        some = mnb.mnb_rope(q[at], k[at], pos[at], freqs, interleaved=interleaved)
        assert torch.equal(some[0], q_out[at]) and torch.equal(some[1], k_out[at]), at
    # keys alone, in place
    assert mnb.mnb_rope(None, k, pos, freqs, interleaved=interleaved, k_out=k)[0] is None
    assert torch.equal(k, k_out)
