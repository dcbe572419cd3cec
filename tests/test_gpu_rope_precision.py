"""GPU: how near rotary positions' cosines and sines come in float32: pairs (1, 0) turn into
them, and (0, 1)."""

import numpy as np
import pytest
import torch

from block_wise_int4_amd import mnb

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.mark.parametrize("interleaved", [False, True], ids=["half", "interleaved"])
@pytest.mark.parametrize("far", [1000, 1 << 20])
def test_cosines_and_sines(far, interleaved):
    tokens, dim = 8192, 128
    g = torch.Generator(DEV).manual_seed(far)
    pos = torch.randint(-far, far, (tokens,), device=DEV, generator=g, dtype=torch.int32)
    freqs, _ = mnb.rope_frequencies(dim, 1e4, device=DEV)
    x = torch.zeros((tokens, 2, dim), device=DEV)
    first = slice(0, None, 2) if interleaved else slice(0, 64)
    second = slice(1, None, 2) if interleaved else slice(64, None)
    x[:, 0, first], x[:, 1, second] = 1.0, 1.0
    y = mnb.mnb_rope(x, None, pos, freqs, interleaved=interleaved)[0].cpu().double().numpy()
    angle = pos.cpu().numpy().astype(np.float64)[:, None] * freqs.cpu().numpy()[None, :]
    c, s = np.cos(angle), np.sin(angle)
    # a cosine and a sine within a unit in the last place of numbers below one (2^-24), and one rounding
    # (2^-25) where they are turned on by what float32 leaves of the angle; the float64 angle's rounding
    tol = 2.0 ** -24 + 2.0 ** -25 + np.abs(angle) * 2.0 ** -51
    for head, want in ((0, (c, s)), (1, (-s, c))):
        for part, ref in zip((first, second), want):
            off = np.abs(y[:, head, part] - ref)
            assert (off <= tol).all(), (off / tol).max()
