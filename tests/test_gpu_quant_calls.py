"""The 8-bit cache's calls as programs make them: the scored selection, several streams,
captured graphs, caches past 2^31 bytes, waits that run out."""
import ctypes
import math
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


@pytest.mark.parametrize("Hq,Hkv,R,d", [(4, 1, 3, 64), (16, 2, 6, 128), (6, 3, 1, 64)])
def test_scored_verification_feeds_the_selection(vsd, Hq, Hkv, R, d):
    """The score is the fp32 sum of the partial scores in group order, its histogram counts
    the candidates, and the selection from them is the selection from the partial scores."""
    prefix, P_max, k, sink, recent = [700, 0, 33, 640], 704, 64, 4, 16
    cache = ref.Cache([p + R for p in prefix], Hkv, d, seed=41)
    q = torch.randn((4, R, Hq, d), generator=cache.gen).bfloat16().cuda()
    pl = i32(prefix)
    out, _, partial, score, hist = vsd.vsd_verify_attn_collect_scored_quant(
        q, *cache.cuda(), pl, P_max=P_max, scale=0.1, n_sink=sink, n_recent=recent)
    plain = vsd.vsd_verify_attn_collect_quant(q, *cache.cuda(), pl, P_max=P_max, scale=0.1)
    assert vsd.vsd_read_device_status() == 0
    assert torch.equal(out, plain[0])
    for b, P in enumerate(prefix):
        assert torch.equal(partial[b, :, :P], plain[2][b, :, :P])
        want = torch.zeros(P, device="cuda")
        for g in range(Hkv):
            want = want + partial[b, g, :P]
        assert torch.equal(score[b, :P], want)
        lo = min(sink, P)
        bits = want[lo:max(P - recent, lo)].view(torch.int32).long() & 0xFFFFFFFF
        key = torch.where(bits >= 2 ** 31, 0xFFFFFFFF - bits, bits + 2 ** 31)
        assert torch.equal(torch.bincount(key >> 20, minlength=4096), hist[b].long())
    a = vsd.vsd_select_topk(partial, pl, k=k, n_sink=sink, n_recent=recent)
    b = vsd.vsd_select_topk_scored(score, hist, pl, k=k, n_sink=sink, n_recent=recent)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def _calls(vsd, seed, stream=None):
    """Inputs of one verification and one draft step, and a function that makes both."""
    cache = ref.Cache([900, 300], 2, 128, seed=seed)
    args = cache.cuda()
    g = torch.Generator(device="cuda").manual_seed(seed)
    q = torch.randn((2, 3, 8, 128), generator=g, device="cuda").bfloat16()
    idx = torch.argsort(torch.rand((2, 290), generator=g, device="cuda"), dim=1)[:, :257].to(torch.int32).contiguous()
    ns, pl, seq = i32([257, 200]), i32([890, 290]), i32([893, 295])

    def run():
        v = vsd.vsd_verify_attn_collect_quant(q, *args, pl, P_max=896, scale=0.1, stream=stream,
                                              logits=lg, partial=ps)
        s = vsd.vsd_sparse_decode_attn_quant(q[:, 0].contiguous() if stream is None else q0, *args, idx, ns, pl, seq,
                                             scale=0.1, max_tail=8, stream=stream)
        return v[0], v[1], v[2], s
    q0 = q[:, 0].contiguous()
    lg = torch.zeros((2, 2, 8, 896), device="cuda")
    ps = torch.zeros((2, 2, 896), device="cuda")
    torch.cuda.synchronize()
    return run


def test_calls_repeat_bit_for_bit(vsd):
    run = _calls(vsd, 51)
    first = [x.clone() for x in run()]
    for _ in range(5):
        assert all(torch.equal(a, b) for a, b in zip(first, run()))
    assert vsd.vsd_read_device_status() == 0


def test_calls_on_two_streams_at_once(vsd):
    """Each call's scratch is its own: interleaved calls on two streams give what they give
    alone."""
    alone = [[x.clone() for x in _calls(vsd, s)()] for s in (52, 53)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    runs = [_calls(vsd, s, stream=st) for s, st in zip((52, 53), streams)]
    got = []
    for _ in range(20):
        got.append([run() for run in runs])
    torch.cuda.synchronize()
    for pair in got:
        for a, b in zip(alone, pair):
            assert torch.equal(a[0], b[0]) and torch.equal(a[3], b[3])
    assert vsd.vsd_read_device_status() == 0


def test_calls_of_growing_and_shrinking_sizes_on_two_streams(vsd):
    """Calls without a workspace of their own, small and large in turn and on two streams,
    give the bits of calls with one."""
    def sizes():
        for B, P in ((1, 300), (3, 2000), (1, 300), (2, 5000), (3, 2000)):
            cache = ref.Cache([P + 4] * B, 2, 64, seed=B * 31 + P)
            q = torch.randn((B, 4, 8, 64), generator=cache.gen).bfloat16().cuda()
            yield cache.cuda(), q, i32([P] * B), P

    own = [torch.empty(1 << 25, dtype=torch.uint8, device="cuda")]
    calls = list(sizes())

    def run(x, **kw):
        (kc, vc, ks, vs, bt), q, pl, P = x
        idx = torch.arange(0, P, 3, dtype=torch.int32, device="cuda").repeat(q.shape[0], 1)
        n = i32([idx.shape[1]] * q.shape[0])
        return (vsd.vsd_verify_attn_collect_quant(q, kc, vc, ks, vs, bt, pl, P_max=P, scale=0.125, **kw) +
                (vsd.vsd_sparse_decode_attn_quant(q[:, 0].contiguous(), kc, vc, ks, vs, bt, idx, n, pl, pl + 1,
                                                  scale=0.125, max_tail=1, **kw),))

    want = [run(x, workspace=own[0]) for x in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for x in calls + calls[::-1]:
        for s, g in zip(streams, got):
            with torch.cuda.stream(s):
                g.append(run(x))
    torch.cuda.synchronize()
    assert vsd.vsd_read_device_status() == 0
    for g in got:
        for a, b in zip(g, want + want[::-1]):
            assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_calls_from_several_threads(vsd):
    """Four host threads, two of them on one stream, call without workspaces of their own."""
    runs = [_calls(vsd, 90 + i) for i in range(4)]
    want = [[x.clone() for x in run()] for run in runs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    streams.append(streams[0])
    bad = []

    def work(i):
        try:
            with torch.cuda.stream(streams[i]):
                for _ in range(25):
                    got = [x.clone() for x in runs[i]()]
                    streams[i].synchronize()
                    if not all(torch.equal(a, b) for a, b in zip(got, want[i])):
                        bad.append(i)
        except Exception as e:  # noqa: BLE001 (reported below)
            bad.append(e)
    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    assert not bad
    assert vsd.vsd_read_device_status() == 0


def test_captured_graphs_replayed_together(vsd):
    alone = [[x.clone() for x in _calls(vsd, s)()] for s in (54, 55)]
    graphs, outs = [], []
    side = torch.cuda.Stream()
    for s in (54, 55):
        run = _calls(vsd, s, stream=side)
        with torch.cuda.stream(side):
            run()
        side.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            outs.append(run())
        graphs.append(g)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(10):
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    for a, o in zip(alone, outs):
        assert all(torch.equal(x, y) for x, y in zip(a, o))
    assert vsd.vsd_read_device_status() == 0


def test_append_and_read_on_a_stream_and_in_a_graph(vsd):
    cache = ref.Cache([64], 2, 64, seed=61)
    kc, vc, ks, vs, bt = cache.cuda()
    rows = torch.randn((1, 5, 2, 64), generator=cache.gen).bfloat16().cuda()
    pos = i32([30])
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    vsd.vsd_append_kv_quant(rows, rows, kc, vc, ks, vs, bt, pos, stream=st)
    st.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        pos.add_(5)
        vsd.vsd_append_kv_quant(rows, rows, kc, vc, ks, vs, bt, pos, stream=st)
        out = vsd.vsd_read_kv_quant(kc, vc, ks, vs, bt, i32_like(pos, 30), n=20, stream=st)
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    for c, s in zip(cache.codes, cache.scales):
        for p in (30, 35, 40):
            ref.append(c, s, rows.cpu().double(), cache.table, [p], [5])
    for got, want in zip(out, cache.kv(0, 30 + torch.arange(15))):
        assert torch.equal(got[0, :15].cpu(), want.float().bfloat16())
    assert vsd.vsd_read_device_status() == 0


def i32_like(t, value):
    return torch.full_like(t, value)


def test_nothing_to_do(vsd):
    cache = ref.Cache([20], 2, 64, seed=62)
    kc, vc, ks, vs, bt = cache.cuda()
    none = i32([])
    empty = torch.zeros((0, bt.shape[1]), dtype=torch.int32, device="cuda")
    rows = torch.zeros((0, 3, 2, 64), dtype=torch.bfloat16, device="cuda")
    vsd.vsd_append_kv_quant(rows, rows, kc, vc, ks, vs, empty, none)
    assert vsd.vsd_read_kv_quant(kc, vc, ks, vs, empty, none, n=3)[0].shape == (0, 3, 2, 64)
    assert vsd.vsd_read_kv_quant(kc, vc, ks, vs, bt, i32([0]), n=0)[0].shape == (1, 0, 2, 64)
    q = torch.zeros((0, 2, 4, 64), dtype=torch.bfloat16, device="cuda")
    assert vsd.vsd_verify_attn_collect_quant(q, kc, vc, ks, vs, empty, none, P_max=8, scale=1.0)[0].shape == q.shape
    q = torch.zeros((0, 4, 64), dtype=torch.bfloat16, device="cuda")
    assert vsd.vsd_sparse_decode_attn_quant(q, kc, vc, ks, vs, empty, None, None, none, none, scale=1.0,
                                            max_tail=1).shape == q.shape
    assert vsd.vsd_read_device_status() == 0


def test_binding_refuses_mismatched_tensors(vsd):
    cache = ref.Cache([40], 2, 64, seed=63)
    kc, vc, ks, vs, bt = cache.cuda()
    q = torch.zeros((1, 2, 4, 64), dtype=torch.bfloat16, device="cuda")
    pl = i32([20])
    call = vsd.vsd_verify_attn_collect_quant
    ok = dict(P_max=32, scale=0.1)
    call(q, kc, vc, ks, vs, bt, pl, **ok)
    bad = [
        ((q, kc, vc, ks, vs.cpu(), bt, pl), ok),
        ((q, kc, vc, ks[:-1], vs, bt, pl), ok),
        ((q, kc, vc[:-1], ks, vs, bt, pl), ok),
        ((q, kc, vc, ks.t().contiguous(), vs, bt, pl), ok),
        ((q, kc, vc, ks, vs.t(), bt, pl), ok),
        ((q, kc.view(torch.uint8), vc, ks, vs, bt, pl), ok),
        ((q.transpose(1, 2), kc, vc, ks, vs, bt, pl), ok),
        ((q, kc, vc, ks, vs, bt, pl.long()), ok),
        ((q, kc, vc, ks, vs, bt, i32([20, 20])), ok),
        ((q, kc, vc, ks, vs, bt, pl), dict(ok, out=torch.zeros_like(q).float())),
        ((q, kc, vc, ks, vs, bt, pl), dict(ok, logits=torch.zeros((1, 2, 4, 31), device="cuda"))),
        ((torch.zeros((1, 2, 4, 128), dtype=torch.bfloat16, device="cuda"), kc, vc, ks, vs, bt, pl), ok),
    ]
    for args, kw in bad:
        with pytest.raises((TypeError, ValueError)):
            call(*args, **kw)
    with pytest.raises(vsd.VsdError):
        call(q, kc, vc, ks, vs, bt, pl, workspace=torch.zeros(256, dtype=torch.uint8, device="cuda"), **ok)
    # rows of another layout, and a view whose storage is not contiguous
    rows = torch.zeros((1, 3, 2, 64), dtype=torch.bfloat16, device="cuda")
    for bad_rows in (rows[..., :32], rows.transpose(1, 2), rows[0]):
        with pytest.raises((TypeError, ValueError)):
            vsd.vsd_append_kv_quant(bad_rows, bad_rows, kc, vc, ks, vs, bt, pl)
    assert vsd.vsd_read_device_status() == 0


def test_caches_past_2_31_bytes(vsd):
    """Pages whose codes lie past 2^31 bytes (and, with head_dim 128 and 8 heads, at every
    block above 131072)."""
    Hkv, d, NB = 8, 128, 133000
    small = ref.Cache([200], Hkv, d, seed=71)
    nblk = -(-200 // 16)
    high = [NB - 1 - 3 * i for i in range(nblk)]
    big = []
    for kv in range(2):
        codes = torch.zeros((NB, Hkv, 16, d), dtype=torch.uint8, device="cuda")
        scales = torch.ones((NB, Hkv), device="cuda")
        for lp in range(nblk):
            blk = int(small.table[0, lp])
            codes[high[lp]] = small.codes[kv][blk].cuda()
            scales[high[lp]] = small.scales[kv][blk].cuda()
        big.append((codes.view(torch.float8_e4m3fn), scales))
    bt = torch.full_like(small.table, -1)
    bt[0, :nblk] = torch.tensor(high, dtype=torch.int32)
    bt = bt.cuda()
    args = (big[0][0], big[1][0], big[0][1], big[1][1], bt)
    rows = torch.randn((1, 3, Hkv, d), generator=small.gen).bfloat16()
    for c, s in zip(small.codes, small.scales):
        ref.append(c, s, rows.double(), small.table, [190], [3])
    vsd.vsd_append_kv_quant(rows.cuda(), rows.cuda(), *args, i32([190]))
    got = vsd.vsd_read_kv_quant(*args, i32([0]), n=193)
    for x, want in zip(got, small.kv(0, torch.arange(193))):
        assert torch.equal(x[0].cpu(), want.float().bfloat16())
    q = torch.randn((1, 1, Hkv, d), generator=small.gen).bfloat16()
    k, v = small.kv(0, torch.arange(193))
    scale = 1 / math.sqrt(d)
    out = vsd.vsd_verify_attn_collect_quant(q.cuda(), *args, i32([192]), P_max=192, scale=scale)[0].cpu().double()
    idx = torch.arange(192, dtype=torch.int32, device="cuda")[None]
    drf = vsd.vsd_sparse_decode_attn_quant(q[:, 0].cuda(), *args, idx, i32([192]), i32([192]), i32([193]),
                                           scale=scale, max_tail=1).cpu().double()
    assert vsd.vsd_read_device_status() == 0
    for h in range(Hkv):
        want, mag = ref.softmax_av(scale * (k[:, h] @ q[0, 0, h].double()), v[:, h])
        for o in (out[0, 0, h], drf[0, h]):
            assert torch.all((o - want).abs() <= ref.out_bound(want, mag))


@pytest.fixture(scope="module")
def short_wait_lib(tmp_path_factory):
    """A copy of the library in which one wait of each waiting kernel waits for a barrier
    that nothing completes before the kernel's end, with a 200 us limit."""
    from sparse_attention_speculative_gb300 import build
    build.build()
    d = tmp_path_factory.mktemp("short_wait_quant")
    path = build.build(extra_flags=("-DVSD_TEST_STALLED_WAIT", "-DVSD_WAIT_LIMIT_NS=200000ull"),
                       out=str(d / "libvsd_stall.so"), objdir=str(d / "obj"))
    lib = ctypes.CDLL(path)
    lib.vsd_read_device_status.argtypes = [ctypes.c_void_p, ctypes.POINTER(ctypes.c_uint)]
    return lib


def test_waits_that_run_out_end_the_kernels_cleanly(vsd, short_wait_lib):
    """Each call returns within a second and raises VSD_DEV_TIMEOUT and nothing else; the
    regular library gives the same results after them as before."""
    run = _calls(vsd, 81)
    before = [x.clone() for x in run()]
    cache = ref.Cache([900, 300], 2, 128, seed=81)
    kc, vc, ks, vs, bt = cache.cuda()
    geom = vsd.Geom(2, 8, 2, 128, 16, bt.shape[1], kc.shape[0])
    p = lambda t: ctypes.c_void_p(t.data_ptr())  # noqa: E731
    q = torch.randn((2, 3, 8, 128), generator=cache.gen).bfloat16().cuda()
    out, pl, seq = torch.zeros_like(q), i32([890, 290]), i32([893, 295])
    idx = torch.arange(257, dtype=torch.int32, device="cuda").repeat(2, 1).contiguous()
    ns = i32([257, 200])
    ws = torch.zeros(32 << 20, dtype=torch.uint8, device="cuda")

    def status():
        flags = ctypes.c_uint(0)
        assert short_wait_lib.vsd_read_device_status(None, ctypes.byref(flags)) == 0
        return int(flags.value)

    def verify():
        return short_wait_lib.vsd_verify_attn_collect_quant(
            ctypes.byref(geom), 3, p(q), p(kc), p(vc), p(ks), p(vs), p(bt), p(pl), 0, 2, 896, ctypes.c_float(0.1),
            None, None, None, None, 0, 0, p(out), p(ws), ctypes.c_size_t(ws.numel()), None)

    def draft():
        return short_wait_lib.vsd_sparse_decode_attn_quant(
            ctypes.byref(geom), p(q), p(kc), p(vc), p(ks), p(vs), p(bt), p(idx), p(ns), 257, p(pl), p(seq), 8,
            ctypes.c_float(0.1), p(out), p(ws), ctypes.c_size_t(ws.numel()), None)
    for call in (verify, draft):
        torch.cuda.synchronize()
        t0 = time.perf_counter()
        assert call() == 0
        torch.cuda.synchronize()
        assert time.perf_counter() - t0 < 1.0
        assert status() == vsd.DEV_TIMEOUT
    assert all(torch.equal(a, b) for a, b in zip(before, run()))
    assert vsd.vsd_read_device_status() == 0
