"""GPU: the decoder example refuses tokens past the bound it was made for, before
anything changes: its tables would have no place for them, and the host would
count blocks that nobody took."""

import pytest
import torch

from workloads import decoder_step as ds

pytestmark = pytest.mark.gpu


def test_decoder_refuses_tokens_past_its_bound():
    d = ds.Decoder(2, 20, page=16, layers=1)          # two pages each: 32 tokens
    x = torch.randn((64, ds.WIDTH), device="cuda").half()
    d.prompt(x[:41], [31, 10])
    free, table, lens = d.free.clone(), d.table.clone(), d.lens.clone()
    d.place([1, 0])                                    # the last place
    with pytest.raises(ValueError, match="32 tokens"):
        d.place([1, 1])
    with pytest.raises(ValueError, match="32 tokens"):
        d.prompt(x[:23], [0, 23])
    assert d.host_lens == [32, 10] == d.lens.tolist()
    assert torch.equal(d.free, free) and torch.equal(d.table, table) and lens.tolist() == [31, 10]
    assert len(d.place([0, 22])) == 22 and d.lens.tolist() == [32, 32] and d.free.numel() == 0
