"""Selection on rows that one CTA writes: cuts inside a few and inside many keys that share their
upper bits, ties among them, rows of one CTA and of several."""
import pytest
import torch

import sparse_attention_speculative_gb300 as pkg

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def vsd():
    pkg.load()
    return pkg


def kept(score, P, k, n_sink, n_recent):
    """Positions of the sinks, the recent window and the highest scores between, ascending."""
    if k >= P:
        return list(range(P))
    sinks, recent = list(range(n_sink)), list(range(P - n_recent, P))
    rest = sorted(range(n_sink, P - n_recent), key=lambda j: (-score[j], j))
    return sorted(sinks + recent + rest[:k - n_sink - n_recent])


@pytest.mark.parametrize("P", [400, 2048, 2049, 5000, 16384, 20000, 32768])
@pytest.mark.parametrize("close", [1, 2, 127, 128, 129, 350])
@pytest.mark.parametrize("step", [0.0, 2.0 ** -20, 2.0 ** -12])
def test_cut_among_close_keys(vsd, P, close, step):
    g = torch.Generator().manual_seed(P + close)
    high = (P - close) // 3
    # `high` scores from 2 up, `close` ones at 1 + small steps (several equal), the others below 1/2
    x = torch.cat([2 + torch.rand(high, generator=g),
                   1 + step * torch.randint(0, 1 + close // 2, (close,), generator=g),
                   torch.rand(P - close - high, generator=g) / 2])
    rows = []
    for r in range(9 if P == 2049 else 3):      # (nine rows: clusters of eight at most)
        rows.append(x[torch.randperm(P, generator=g)])
    score = torch.stack(rows)
    n_sink, n_recent = 3, 5
    for take in sorted({0, 1, close // 2, close - 1, close}):
        k = min(P, high + take + n_sink + n_recent)
        idx, n, _ = vsd.vsd_select_topk(score[:, None].cuda(), torch.full((len(rows),), P, dtype=torch.int32).cuda(),
                                        k=k, n_sink=n_sink, n_recent=n_recent)
        assert n.tolist() == [k] * len(rows)
        for r, row in enumerate(rows):
            assert idx[r].tolist() == kept(row.tolist(), P, k, n_sink, n_recent)
    assert vsd.vsd_read_device_status() == 0


@pytest.mark.parametrize("P", [600, 32768])
def test_one_value(vsd, P):
    """Every score the same: the lowest positions."""
    score = torch.zeros((2, 1, P), device="cuda")
    idx, n, _ = vsd.vsd_select_topk(score, torch.tensor([P, P - 1], dtype=torch.int32).cuda(), k=300, n_sink=0,
                                    n_recent=10)
    assert idx[0].tolist() == list(range(290)) + list(range(P - 10, P))
    assert idx[1].tolist() == list(range(290)) + list(range(P - 11, P - 1))


@pytest.mark.parametrize("P", [1500, 20000, 60000])
@pytest.mark.parametrize("count", [101, 5000])
def test_histogram_of_other_scores(vsd, P, count):
    """A histogram that names fewer keys than the boundary bin has: positions of the row, in order,
    and nothing outside the buffers."""
    score = torch.ones((2, P), device="cuda")
    key = (0x80000000 | 0x3F800000) >> 20          # (of 1.0: the order-preserving key's upper 12 bits)
    hist = torch.zeros((2, 4096), dtype=torch.int32, device="cuda")
    hist[:, key] = count
    idx, n = vsd.vsd_select_topk_scored(score, hist, torch.full((2,), P, dtype=torch.int32).cuda(), k=100, n_sink=0,
                                        n_recent=0)
    torch.cuda.synchronize()
    vsd.vsd_read_device_status()
    assert n.tolist() == [100, 100]
    for row in idx.tolist():
        assert all(0 <= a < b < P for a, b in zip(row, row[1:]))
