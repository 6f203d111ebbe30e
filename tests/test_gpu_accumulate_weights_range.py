"""Queries near bf16's last binade over small key scales: logits of order one, whose products with the
codes alone leave fp32."""
import pytest
import torch

from tests.test_gpu_accumulate_weights import Case, clean_status, vsd  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("P_max", [300, 40000])                 # held in registers, and read again
@pytest.mark.parametrize("by", [2.0 ** 118, 2.0 ** 60, 2.0 ** -60, 2.0 ** -100])
def test_queries_and_scales_apart(vsd, P_max, by):  # noqa: F811
    """A power of two from the scales to the queries: the same logits, so the same sums, bit for bit."""
    c = Case([P_max - 20, 9], P_max, R=5, C=2, G=4, Hkv=2, d=128, quant=True, seed=6)
    want = c.call(vsd)
    c.check(want, (0, 4))
    c.q, c.scales = (c.q.double() * by).to(torch.bfloat16), c.scales / by
    assert torch.isfinite(c.q).all() and (c.scales >= 2.0 ** -126).all() and torch.isfinite(c.scales).all()
    got = c.call(vsd)
    c.check(got, (0, 4))
    assert torch.equal(got, want)
    assert vsd.vsd_read_device_status() == 0


def test_scales_that_are_subnormal_or_zero(vsd):  # noqa: F811
    """Keys that a scale below 2^-126 or of zero makes next to nothing: logits of zero."""
    c = Case([100], 100, R=4, C=2, G=2, Hkv=2, d=64, quant=True, seed=7)
    for s in (0.0, 2.0 ** -149, 2.0 ** -130):
        c.scales.fill_(s)
        c.check(c.call(vsd), (0, 3))
    assert vsd.vsd_read_device_status() == 0
