"""The 8-bit cache's calls where they could go wrong between calls and at the ends of their
ranges."""
import threading

import pytest
import torch

from tests import quant_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def vsd():
    from sparse_attention_speculative_gb300 import build
    build.build()
    import sparse_attention_speculative_gb300 as m
    m.vsd_read_device_status()
    return m


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------ host threads
def test_first_calls_of_a_host_thread(vsd):
    """A thread whose first use of CUDA is one of these calls, with every output and the
    workspace given: the calls do not rely on an earlier one that made the device's context
    current."""
    cache = ref.Cache([900, 300], 2, 64, seed=1)
    kc, vc, ks, vs, bt = cache.cuda()
    q = torch.randn((2, 3, 8, 64), generator=cache.gen).bfloat16().cuda()
    pl, out = i32([890, 290]), torch.empty_like(q)
    ws = torch.zeros(32 << 20, dtype=torch.uint8, device="cuda")
    stream = torch.cuda.current_stream()
    kb = torch.zeros(kc.shape, dtype=torch.bfloat16, device="cuda")

    def quant():
        vsd.vsd_verify_attn_collect_quant(q, kc, vc, ks, vs, bt, pl, P_max=896, scale=0.1, collect=False, out=out,
                                          workspace=ws, stream=stream)

    def bf16():
        vsd.vsd_verify_attn_collect(q, kb, kb, bt, pl, P_max=896, scale=0.1, collect=False, out=out, workspace=ws,
                                    stream=stream)
    for call in (quant, bf16):
        ws.zero_()
        call()
        torch.cuda.synchronize()
        want, bad = out.clone(), []
        ws.zero_()
        out.zero_()
        torch.cuda.synchronize()

        def work():
            try:
                call()
            except Exception as e:  # noqa: BLE001 (reported below)
                bad.append(e)
        th = threading.Thread(target=work)
        th.start()
        th.join()
        assert not bad
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    assert vsd.vsd_read_device_status() == 0
