"""Keys of the verify block that are NaN, by their values or by their page's scale: they reach the
rows that see them, and no others."""
import math

import pytest
import torch

from tests.test_gpu_accumulate_weights import Case, clean_status, vsd  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("P_max", [40, 40000])                # held in registers, and read again
def test_scale_of_a_page(vsd, P_max):  # noqa: F811
    """Keys 0 and 1 end one page, 2 and 3 begin the next, whose scale for head 1 is NaN."""
    c = Case([30, P_max - 10], P_max, R=4, C=2, G=2, Hkv=2, d=64, quant=True, seed=3)
    c.check(c.call(vsd), (0, 3))
    c.scales[int(c.table[0, 2]), 1] = math.nan
    got = c.call(vsd).cpu()
    want = c.call(vsd, rows=(0, -1)).cpu()
    assert torch.isnan(got[0, 1, :30]).all() and torch.equal(got[0, 1, 30:], c.weights[0, 1, 30:])
    assert not torch.isnan(got[0, 0]).any() and not torch.isnan(got[1]).any()
    assert torch.isfinite(want).all()                         # row 0 sees key 0 alone
    assert vsd.vsd_read_device_status() == 0


@pytest.mark.parametrize("P_max", [40, 40000])
@pytest.mark.parametrize("quant", [False, True])
def test_value_of_a_key(vsd, P_max, quant):  # noqa: F811
    c = Case([30, P_max - 10], P_max, R=4, C=2, G=2, Hkv=2, d=64, quant=quant, seed=4)
    c.check(c.call(vsd), (0, 3))
    page = int(c.table[0, 2])
    if quant:
        c.codes[page, 1, 0, 5] = 0x7F
    else:
        c.keys[page, 1, 0, 5] = math.nan
    got, want = c.call(vsd).cpu(), c.call(vsd, rows=(0, -1)).cpu()
    assert torch.isnan(got[0, 1, :30]).all() and torch.equal(got[0, 1, 30:], c.weights[0, 1, 30:])
    assert not torch.isnan(got[0, 0]).any() and not torch.isnan(got[1]).any() and torch.isfinite(want).all()
    assert vsd.vsd_read_device_status() == 0


@pytest.mark.parametrize("quant", [False, True])
def test_page_outside_the_cache_is_left_out(vsd, quant):  # noqa: F811
    """... with its flag, whatever the keys beside it: the sums are those of the others."""
    c = Case([30], 40, R=4, C=2, G=2, Hkv=2, d=64, quant=quant, seed=5)
    table = c.table.clone()
    table[0, 2] = -1
    got = c.call(vsd, table=table.cuda()).cpu()
    assert vsd.vsd_read_device_status() == vsd.DEV_BAD_BLOCK
    seen = c.block_logits((0, 3))
    seen[0][1] = seen[0][1][:, :2]
    from tests import cache_life_ref as life
    want, bound = life.accumulated(c.weights.double(), c.logits, seen, (0, 3), c.prefix, c.G)
    assert torch.all((got.double() - want).abs() <= bound)
