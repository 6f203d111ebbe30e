"""Norms without an epsilon: right where fp32 holds the squares; rows of zeros are no numbers."""
import math

import pytest
import torch

from tests import cache_life_ref as life
from tests import quant_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def vsd():
    import sparse_attention_speculative_gb300 as m
    m.load()
    m.vsd_read_device_status()
    return m


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("by", [1.0, 2.0 ** 55, 2.0 ** -50])
def test_rows_without_an_epsilon(vsd, d, by):
    g = torch.Generator().manual_seed(d)
    n, H = 21, 3
    x = (torch.randn((1, n, H, d), generator=g) * by).to(torch.bfloat16)
    x[0, 5, 1] = 0
    w = (1 + 0.2 * torch.randn(d, generator=g)).to(torch.bfloat16)
    freq = life.inv_freq(d, 10000.0)
    pos = torch.tensor([7], dtype=torch.int32, device="cuda")
    got, _ = vsd.vsd_norm_rope(x.cuda(), None, vsd.vsd_rope_turns(freq), pos, q_weight=w.cuda(), eps=0.0)
    want, off = life.turned(x[0].double(), w, 0.0, list(range(7, 7 + n)), freq, False)
    zero = torch.zeros((n, H, d), dtype=torch.bool)
    zero[5, 1] = True
    got = got[0].cpu().double()
    assert torch.isnan(got[5, 1]).all()
    assert torch.all(((got - want).abs() <= life.bf16_bound(want, off)) | zero)


@pytest.mark.parametrize("d", [64, 128])
def test_rows_of_zeros_in_an_8_bit_page(vsd, d):
    """... become NaN codes, and set no scale for the page's others."""
    g = torch.Generator().manual_seed(d)
    n, H = 20, 2
    x = torch.randn((1, n, H, d), generator=g).to(torch.bfloat16)
    x[0, 3, 1] = 0
    w = (1 + 0.2 * torch.randn(d, generator=g)).to(torch.bfloat16).cuda()
    table = torch.tensor([[1, 0]], dtype=torch.int32, device="cuda")
    out = []
    for eps in (0.0, 1e-6):
        cache = [torch.zeros((2, H, 16, d), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn) for _ in range(2)]
        scale = [torch.zeros((2, H), device="cuda") for _ in range(2)]
        vsd.vsd_norm_rope_append_kv_quant(x.cuda(), x.cuda(), x.cuda(), *cache, *scale, table,
                                          torch.zeros(1, dtype=torch.int32, device="cuda"), None, k_weight=w, eps=eps)
        rows = [ref.decode(c.view(torch.uint8).cpu()) * s.cpu().double()[:, :, None, None] for c, s in zip(cache, scale)]
        out.append([r[[1, 0]].transpose(1, 2).reshape(-1, H, d)[:n] for r in rows])
    zero = torch.zeros((n, H, d), dtype=torch.bool)
    zero[3, 1] = True
    assert torch.equal(torch.isnan(out[0][0]), zero) and not torch.isnan(out[1][0]).any()
    # (an epsilon of 1e-6 beside squares of order one: below 2^-19 of a value, a step of a code at most)
    a, b = out[0][0][~zero], out[1][0][~zero]
    assert torch.all((a - b).abs() <= 2.0 ** -3 * b.abs() + 2.0 ** -9)
    assert torch.equal(out[0][1], out[1][1])
    assert vsd.vsd_read_device_status() == 0 and math.isfinite(float(a.sum()))
