"""The hybrid budget where a thread's positions lie in two words of the first pass's bitmap: slices of
a row that are no power of two (12, 20, 24 and 28 positions a thread)."""
import numpy as np
import pytest
import torch

import oracle
import sparse_attention_speculative_gb300 as pkg
from tests.parity_utils import fp32_row_sum

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def vsd():
    pkg.load()
    pkg.vsd_read_device_status()
    return pkg


@pytest.mark.parametrize("n_rows,P_max", [(9, 40000), (1, 80000), (9, 80001), (8, 98000), (9, 110000), (2, 200000)])
def test_candidates_of_the_first_pass_are_taken(vsd, n_rows, P_max):
    rng = np.random.default_rng(P_max)
    prefix = rng.integers(P_max // 2, P_max + 1, size=n_rows).astype(np.int32)
    prefix[0] = P_max
    target = rng.integers(-4, 5, size=(n_rows, 2, P_max)).astype(np.float32)  # ties
    draft = rng.normal(size=(n_rows, 1, P_max)).astype(np.float32)
    on_gpu = [torch.tensor(x, device="cuda") for x in (target, draft, prefix)]
    for k, m, n_sink, n_recent in [(4096, 2000, 16, 256), (500, 500, 0, 0), (3000, 1, 4, 64)]:
        idx, n_sel = vsd.vsd_select_topk_hybrid(*on_gpu, k=k, m=m, n_sink=n_sink, n_recent=n_recent)
        torch.cuda.synchronize()
        assert vsd.vsd_read_device_status() == 0
        want, n = oracle.select_hybrid(fp32_row_sum(target), fp32_row_sum(draft), prefix, k=k, m=m, n_sink=n_sink,
                                       n_recent=n_recent)
        np.testing.assert_array_equal(n_sel.cpu().numpy(), n)
        for r in range(n_rows):
            np.testing.assert_array_equal(idx[r].cpu().numpy()[:n[r]], want[r, :n[r]])
            assert torch.all(idx[r, n[r]:] == -1)
