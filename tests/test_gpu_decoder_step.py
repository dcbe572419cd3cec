"""GPU: a decoder's attention half as workloads/decoder_step.py runs it, against
the same wiring in plain float64: dequantized weights, every request's own keys
and values in one list each, no pages.

Tolerance, per element of the residual rows x (standard normal at the start;
weights of deviation 0.02 on 768 inputs, so that a product's rows deviate
0.55 times its input): a value row is within 2e-3 of its largest element, some
2.5, of the exact product (the bound the products are held to), and so is the
attention's output that averages them, 5e-3; the o product passes that on
0.55-fold, four deviations at most (1.1e-2), and adds 2e-3 of its own largest
element, below 1 (2e-3). Two such updates a layer, two layers: 5.2e-2; and the
sums are rounded to float16 four times at up to 4 (2^-9 each): 8e-3. Errors that
reach q and k move the weights by less than a hundredth part of this. So 6e-2,
while what the attention adds to x is several tenths at its largest.
"""

import pytest
import torch

from block_wise_int4_amd import mnb
from workloads import decoder_step as ds

pytestmark = pytest.mark.gpu


def _attend(q, k, v):
    """q [heads, dim] over k, v [n, heads, dim], float64."""
    w = torch.softmax(torch.einsum("hd,nhd->hn", q, k) * ds.DIM ** -0.5, dim=1)
    return torch.einsum("hn,nhd->hd", w, v)


def _reference(d, prompts, x_prompt, xs, states, frames):
    """Residual rows after each step, float64 on the CPU."""
    w = [{n: mnb.mnb_dequant(getattr(l, n)).cpu().double() for n in
          ("q", "k", "v", "o", "cross_q", "cross_k", "cross_v", "cross_o")} for l in d.layers]
    split = lambda t: t.view(-1, ds.HEADS, ds.DIM)
    keys = [[[] for _ in prompts] for _ in w]
    values = [[[] for _ in prompts] for _ in w]
    at = 0
    for b, n in enumerate(prompts):
        rows = x_prompt[at:at + n]
        at += n
        for l, m in enumerate(w):
            keys[l][b] += list(split(rows @ m["k"].T))
            values[l][b] += list(split(rows @ m["v"].T))
    out = []
    for x in xs:
        x = x.clone()
        for l, m in enumerate(w):
            for b in range(len(prompts)):
                row = x[b:b + 1].clone()
                keys[l][b] += list(split(row @ m["k"].T))
                values[l][b] += list(split(row @ m["v"].T))
                a = _attend(split(row @ m["q"].T)[0], torch.stack(keys[l][b]), torch.stack(values[l][b]))
                row = row + a.reshape(1, -1) @ m["o"].T
                s = states[b, :frames[b]]
                if len(s):
                    a = _attend(split(row @ m["cross_q"].T)[0], split(s @ m["cross_k"].T), split(s @ m["cross_v"].T))
                    row = row + a.reshape(1, -1) @ m["cross_o"].T
                x[b] = row[0]
        out.append(x)
    return out


def test_decoder_step_against_plain_attention():
    gen = torch.Generator().manual_seed(5)
    prompts, frames, steps = [1, 15, 38], [70, 0, 33], 4      # the steps cross pages of 16
    x_prompt = torch.randn((sum(prompts), ds.WIDTH), generator=gen).half()
    xs = [torch.randn((3, ds.WIDTH), generator=gen).half() for _ in range(steps)]
    states = torch.randn((3, 70, ds.WIDTH), generator=gen).half()
    d = ds.Decoder(3, 48, page=16, layers=2)
    d.encode(states.cuda(), torch.tensor(frames, dtype=torch.int32, device="cuda"))
    d.prompt(x_prompt.cuda(), prompts)
    got = [d.step(x.cuda()).cpu().double() for x in xs]
    assert d.lens.tolist() == [n + steps for n in prompts] == d.host_lens
    held = [-(-n // 16) for n in d.host_lens]
    blocks = d.table[d.table >= 0].tolist()
    assert (d.table >= 0).sum(dim=1).tolist() == held and len(set(blocks)) == sum(held)
    ref = _reference(d, prompts, x_prompt.double(), [x.double() for x in xs], states.double(), frames)
    for g, r, x in zip(got, ref, xs):
        assert (g - r).abs().max().item() <= 6e-2
        assert (r - x.double()).abs().max().item() > 0.2      # the attention is no small part
