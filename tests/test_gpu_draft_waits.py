"""Draft steps of very unequal lists on the warp-specialised kernel: most of its items have no
work, so its consumers' warps pass many stages in a row, each at its own pace."""
import numpy as np
import pytest
import torch

import oracle
from tests.parity_utils import assert_attn_close

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d,Hq,Hkv", [(128, 32, 8), (64, 64, 8)])
def test_stages_without_work_are_handed_back_by_every_warp(d, Hq, Hkv):
    """300 steps, some of them gathering early: no wait gives up, every step gives the same
    bits, and they are the definition's."""
    import sparse_attention_speculative_gb300 as vsd
    from sparse_attention_speculative_gb300 import build
    from sparse_attention_speculative_gb300.synth import host_arrays, make_batch, to_u16
    from sparse_attention_speculative_gb300.workloads import Workload
    build.build()
    oracle.build()
    n_per = [4096, 1, 130, 0, 2, 2500, 1, 1, 129, 3, 1, 40]
    prefix = tuple(max(n + 200, 300) for n in n_per)
    w = Workload("waits", B=len(n_per), P=max(prefix), Hq=Hq, Hkv=Hkv, d=d, gamma=3, k=4096, n_sink=0, n_recent=0,
                 seed=31, prefix_lens=prefix)
    batch = make_batch(w, "cuda")
    rng = np.random.default_rng(32)
    idx = torch.full((w.B, w.k), -1, dtype=torch.int32, device="cuda")
    for b, (P, n) in enumerate(zip(prefix, n_per)):
        if n:
            idx[b, :n] = torch.from_numpy(np.sort(rng.choice(P, size=n, replace=False)).astype(np.int32)).cuda()
    n_sel = torch.tensor(n_per, dtype=torch.int32, device="cuda")
    tail, seq = batch.prefix_len.clone(), batch.prefix_len + 1
    q = batch.q_draft[0]
    args = (q, batch.k_cache, batch.v_cache, batch.block_table, idx, n_sel, tail, seq)
    vsd.vsd_read_device_status()
    first = vsd.vsd_sparse_decode_attn(*args, scale=w.scale, max_tail=4)
    for i in range(300):
        out = vsd.vsd_sparse_decode_attn_step(*args, scale=w.scale, max_tail=4,
                                              flags=vsd.STEP_EARLY_GATHER if i & 1 else 0)
        if i % 20 == 0:
            assert torch.equal(out, first)
    torch.cuda.synchronize()
    assert vsd.vsd_read_device_status() == 0
    assert torch.equal(out, first)
    h = host_arrays(batch)
    want = oracle.sparse_decode(to_u16(q), h["k_cache"], h["v_cache"], h["block_table"], idx.cpu().numpy(),
                                n_sel.cpu().numpy(), tail.cpu().numpy(), seq.cpu().numpy(), scale=w.scale)
    assert_attn_close(first.float().cpu().numpy(), want, "draft step of unequal lists")
