"""Eviction beside rows of sums that are shorter than a prefix, or as long as a stride may be."""
import pytest
import torch

from tests.test_gpu_compact_kv import Case, clean_status, int32, vsd  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("quant", [False, True])
@pytest.mark.parametrize("heads", [False, True])
@pytest.mark.parametrize("where", ["same", "other"])
@pytest.mark.parametrize("weights", ["new", "place"])
@pytest.mark.parametrize("stride", [300, 70])
def test_indices_without_a_sum(vsd, quant, heads, where, weights, stride):  # noqa: F811
    """Prefixes longer than the rows of sums: indices that have none are flagged and their rows stay,
    in K and V alike; the others move."""
    c = Case([400, 90, 64], 60, 2, 64, quant, heads, seed=stride, where=where)
    full, c.weights = c.weights, c.weights[..., :stride].contiguous()
    got = c.run(vsd, weights=weights)
    assert vsd.vsd_read_device_status() == vsd.DEV_BAD_INDEX
    # the same, with the rows that were refused put back
    c.weights = torch.where(torch.arange(full.shape[2]) < stride, full, 0.0)
    want = c.want()
    lists = c.idx.expand(-1, c.Hkv, -1)
    refused = (lists >= stride)
    assert refused[0].any() and not refused[1 if stride == 300 else 2].all()
    for b in range(3):
        for g in range(c.Hkv):
            n = int(c.n[b, g if heads else 0])
            for i in range(n):
                page = int(c.dst[b, i // 16])
                for kv in range(2):
                    row = got[0][kv][page, g, i % 16]
                    if refused[b, g, i]:
                        assert torch.equal(row, c.caches[kv][page, g, i % 16])
                    elif not refused[b, g, i // 16 * 16:i // 16 * 16 + 16].any():
                        same = row == want[0][kv][page, g, i % 16]
                        assert torch.all(same | (((row & 0x7F) == 0x7F) if quant else torch.tensor(False)))
                assert got[2][b, g, i] == (0.0 if refused[b, g, i] else want[2][b, g, i])
            assert torch.all(got[2][b, g, n:] == 0)


@pytest.mark.parametrize("quant", [False, True])
def test_indices_below_the_stride_need_no_more_of_it(vsd, quant):  # noqa: F811
    c = Case([400, 400], 60, 2, 64, quant, False, seed=1, where="other")
    c.idx[:, :, :60] = torch.arange(0, 120, 2, dtype=torch.int32)
    got = c.run(vsd)
    c.weights = c.weights[..., :119].contiguous()
    again = c.run(vsd)
    assert vsd.vsd_read_device_status() == 0
    c.check(again)
    assert all(torch.equal(a, b) for a, b in zip(got[0] + got[1] + [got[2]], again[0] + again[1] + [again[2]]))


def test_the_longest_stride(vsd):  # noqa: F811
    """Zeros to the end of a row of 2^31 - 1 sums (its positions and the step past them in 32 bits)."""
    stride = 2 ** 31 - 1
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("8.6 GB for the sums and their comparison")
    c = Case([50], 20, 1, 64, False, False, seed=2, where="other")
    out = torch.ones((1, 1, stride), device="cuda")
    dev = [x.cuda().view(torch.bfloat16) for x in c.caches]
    vsd.vsd_compact_kv(*dev, c.table.cuda(), c.dst.cuda(), int32([50]), *c.lists(), weights=c.weights.cuda(), weights_out=out)
    assert vsd.vsd_read_device_status() == 0
    n = int(c.n[0, 0])
    assert torch.equal(out[0, 0, :n].cpu(), c.want()[2][0, 0, :n])
    assert int(torch.count_nonzero(out[0, 0, n:])) == 0
    del out
    torch.cuda.empty_cache()


@pytest.mark.parametrize("quant", [False, True])
@pytest.mark.parametrize("heads", [False, True])
def test_lists_of_no_index(vsd, quant, heads):  # noqa: F811
    """k = 0: nothing moves, and the sums that are returned have no elements."""
    c = Case([40, 0], 0, 2, 64, quant, heads, seed=3)
    for weights, shape in (("new", (2, 2, 0)), ("none", None), ("place", c.weights.shape)):
        got = c.run(vsd, weights=weights)
        assert all(torch.equal(a, b) for a, b in zip(got[0] + got[1], c.caches + c.scales))
        assert got[2] is None if shape is None else got[2].shape == shape and not got[2].any()
    assert vsd.vsd_read_device_status() == 0


def test_sums_of_no_position(vsd):  # noqa: F811
    """Rows of sums without elements beside lists that have some: refused, not ignored."""
    c = Case([40], 16, 2, 64, False, False, seed=4)
    c.weights = c.weights[..., :0]
    with pytest.raises(vsd.VsdError):
        c.run(vsd)
