"""The 8-bit cache's calls where they could go wrong between calls and at the ends of their
ranges."""
import ctypes
import threading
import time

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


# ------------------------------------------------------------------ scratch of the calls
@pytest.fixture()
def recorded(vsd):
    """The extension module with stand-ins for the two attention calls of the library: they
    launch nothing, stay inside for a while and list every scratch address that a second
    call brings while a first one still has it."""
    from sparse_attention_speculative_gb300 import _lib
    lib = _lib.load()
    inside, seen, shared, lock = [], [], [], threading.Lock()
    P, I, F, SZ = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t

    def body(ws, size):
        with lock:
            if ws in inside:
                shared.append(ws)
            inside.append(ws)
            seen.append((ws, size))
        time.sleep(0.02)
        with lock:
            inside.remove(ws)
        return 0
    VERIFY = ctypes.CFUNCTYPE(I, P, I, P, P, P, P, P, P, P, I, I, I, F, P, P, P, P, I, I, P, P, SZ, P)
    SPARSE = ctypes.CFUNCTYPE(I, P, P, P, P, P, P, P, P, P, I, P, P, I, F, P, P, SZ, P)
    verify = VERIFY(lambda *a: body(a[20], a[21]))
    sparse = SPARSE(lambda *a: body(a[15], a[16]))
    addr = lambda f: ctypes.cast(f, ctypes.c_void_p).value  # noqa: E731
    module = _lib._bound()
    module.attach(vsd.VsdError, addr(lib.vsd_append_kv_quant), addr(lib.vsd_read_kv_quant),
                  addr(lib.vsd_verify_quant_workspace_size), addr(verify),
                  addr(lib.vsd_sparse_quant_workspace_size), addr(sparse))
    yield seen, shared
    _lib._bound()  # (the library's own calls again)


@pytest.mark.parametrize("same_stream", [True, False])
def test_calls_from_two_threads_have_scratch_of_their_own(vsd, recorded, same_stream):
    """A call is two launches that hand partial results on in its scratch: no other call may
    have that memory before both are made, whichever thread makes it and on which stream."""
    seen, shared = recorded
    cache = ref.Cache([900, 300], 2, 64, seed=1)
    args = cache.cuda()
    q = torch.zeros((2, 3, 8, 64), dtype=torch.bfloat16, device="cuda")
    idx = torch.zeros((2, 257), dtype=torch.int32, device="cuda")
    ns, pl, seq = i32([257, 200]), i32([890, 290]), i32([893, 295])
    streams = [torch.cuda.Stream()] * 2 if same_stream else [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    bad = []

    def work(stream):
        try:
            with torch.cuda.stream(stream):
                for _ in range(5):
                    vsd.vsd_verify_attn_collect_quant(q, *args, pl, P_max=896, scale=0.1, collect=False)
                    vsd.vsd_sparse_decode_attn_quant(q[:, 0].contiguous(), *args, idx, ns, pl, seq, scale=0.1,
                                                     max_tail=8)
        except Exception as e:  # noqa: BLE001 (reported below)
            bad.append(e)
    threads = [threading.Thread(target=work, args=(s,)) for s in streams]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    assert not bad
    assert len(seen) == 20 and all(ws and size for ws, size in seen)
    assert not shared


def test_calls_keep_no_memory(vsd):
    """What a call without a workspace allocates goes back to torch's allocator."""
    cache = ref.Cache([4000], 2, 64, seed=2)
    args, pl = cache.cuda(), i32([3990])
    q = torch.zeros((1, 8, 8, 64), dtype=torch.bfloat16, device="cuda")
    out = torch.empty_like(q)
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    with torch.cuda.stream(stream):
        vsd.vsd_verify_attn_collect_quant(q, *args, pl, P_max=3990, scale=0.1, collect=False, out=out)
    stream.synchronize()
    assert torch.cuda.memory_allocated() == before
    assert vsd.vsd_read_device_status() == 0
