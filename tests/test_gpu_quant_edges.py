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
    module.attach(vsd.VsdError, addr(lib.vsd_append_kv_quant), addr(lib.vsd_read_kv_quant_zeroed),
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


# ------------------------------------------------------------------ NaN and infinities
def attend(cache, prefix, q, Hkv, scale):
    """The verification's outputs in 64 bits: [B, R, Hq, d].  Nothing of a key that a row does
    not see enters it; a NaN in what it sees does."""
    B, R, Hq, d = q.shape
    out = torch.zeros((B, R, Hq, d), dtype=torch.float64)
    mag = torch.zeros_like(out)
    for b in range(B):
        k, v = cache.kv(b, torch.arange(prefix[b] + R))
        for h in range(Hq):
            g = h // (Hq // Hkv)
            for t in range(R):
                n = prefix[b] + t + 1
                out[b, t, h], mag[b, t, h] = ref.softmax_av(scale * (k[:n, g] @ q[b, t, h].double()), v[:n, g])
    return out, mag


def assert_outputs(got, want, mag):
    """NaN exactly where the definition has it, the others within the bound."""
    got = got.cpu().double()
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    fin = ~torch.isnan(want)
    assert torch.all((got - want).abs()[fin] <= ref.out_bound(want, mag)[fin])


@pytest.mark.parametrize("B,Hkv,d,longest", [(64, 8, 64, 120), (64, 8, 128, 120), (70, 8, 64, 300), (300, 2, 64, 100),
                                             (3, 2, 64, 500)])
def test_verify_nan_values_reach_the_rows_that_see_them(vsd, B, Hkv, d, longest):
    """NaN codes in the values of every third pair's verify block, in another row and
    dimension each, and of a few pairs' prefixes: the outputs are NaN in the rows and
    dimensions that see one, and nowhere else.  Most sequences are one or two tiles, so that a
    CTA walks several pairs."""
    R, G = 3, 2
    g = torch.Generator().manual_seed(B + d)
    prefix = torch.randint(0, longest - R, (B,), generator=g).tolist()
    cache = ref.Cache([p + R for p in prefix], Hkv, d, seed=B * 3 + d)
    for pair in range(0, B * Hkv, 3):
        b, h = pair // Hkv, pair % Hkv
        j = prefix[b] + pair % R
        cache.codes[1][int(cache.table[b, j // 16]), h, j % 16, (pair * 7) % d] = ref.NAN_CODE + 128 * (pair & 1)
    for pair in range(1, B * Hkv, 50):
        b, h = pair // Hkv, pair % Hkv
        if prefix[b]:
            j = (pair * 5) % prefix[b]
            cache.codes[1][int(cache.table[b, j // 16]), h, j % 16, pair % d] = ref.NAN_CODE
    q = torch.randn((B, R, Hkv * G, d), generator=g).bfloat16()
    args, pl, qc = cache.cuda(), i32(prefix), q.cuda()
    out = [vsd.vsd_verify_attn_collect_quant(qc, *args, pl, P_max=longest, scale=0.125, collect=False)[0]
           for _ in range(20)]
    assert vsd.vsd_read_device_status() == 0
    want, mag = attend(cache, prefix, q, Hkv, 0.125)
    assert torch.isnan(want).any() and not torch.isnan(want).all()
    assert_outputs(out[0], want, mag)
    for o in out[1:]:
        assert torch.equal(o.view(torch.int16), out[0].view(torch.int16))


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("others", ["zeros", "ordinary", "largest"])
@pytest.mark.parametrize("d", [64, 128])
def test_a_nan_or_an_infinity_in_a_query_row_stays_in_it(vsd, bad, others, d):
    """The row that holds it becomes NaN, outputs and logits; the rows beside it do not, be they
    zeros (they average the values), ordinary or within a few binades of the largest."""
    R, Hq, Hkv, P = 3, 4, 2, 150
    cache = ref.Cache([P + R], Hkv, d, seed=d)
    q = torch.zeros((1, R, Hq, d))
    if others != "zeros":
        q = torch.randn((1, R, Hq, d), generator=cache.gen)
        if others == "largest":
            q = q.sign() * 2.0 ** 127
            for s in cache.scales[0]:
                s *= 2.0 ** -118
    q = q.bfloat16()
    q[0, 1, 2, 17] = bad
    logits = torch.zeros((1, 2, Hq, P), device="cuda")
    out, lg, _ = vsd.vsd_verify_attn_collect_quant(q.cuda(), *cache.cuda(), i32([P]), P_max=P, scale=2.0 ** -12,
                                                   row0=0, row1=1, logits=logits)
    drafts = vsd.vsd_sparse_decode_attn_quant(q[:, 1].contiguous().cuda(), *cache.cuda(), None, None, i32([0]),
                                              i32([P + 2]), scale=2.0 ** -12, max_tail=P + 2)
    assert vsd.vsd_read_device_status() == 0
    mine = torch.zeros((1, R, Hq), dtype=torch.bool)
    mine[0, 1, 2] = True
    want, mag = attend(cache, [P], torch.where(mine[..., None], torch.zeros_like(q), q), Hkv, 2.0 ** -12)
    want[mine] = float("nan")
    assert_outputs(out, want, mag)
    assert_outputs(drafts, want[:, 1], mag[:, 1])
    nan = torch.isnan(lg.cpu())
    assert nan[0, 1, 2].all() and nan.sum() == P
    if others == "zeros":
        assert torch.all(lg.cpu()[~nan] == 0)


# ------------------------------------------------------------------ ends of the ranges
@pytest.mark.parametrize("d", [64, 128])
def test_large_queries_meet_small_key_scales(vsd, d):
    """Query rows from 2^-60 to bf16's last binade in one group, key scales near 2^-125: the
    logits are of order one, and no factor of theirs overflows on the way."""
    R, Hq, Hkv, P = 3, 4, 2, 300
    cache = ref.Cache([P + R], Hkv, d, seed=d + 5)
    for s in cache.scales[0]:
        s *= 2.0 ** -118
    q = torch.randn((1, R, Hq, d), generator=cache.gen)
    q = q.sign() * 2.0 ** 127
    q[0, 1, 1] *= 2.0 ** -127
    q[0, 2] *= 2.0 ** -100
    q[0, 0, 3] *= 2.0 ** -187
    q = q.bfloat16()
    for rows in (q, q[:, :, ::3].repeat_interleave(2, dim=2), q[:, :1].expand(1, R, Hq, d).contiguous()):
        logits = torch.zeros((1, 2, Hq, P), device="cuda")
        out = vsd.vsd_verify_attn_collect_quant(rows.cuda(), *cache.cuda(), i32([P]), P_max=P, scale=2.0 ** -12,
                                                logits=logits)[0]
        drafts = vsd.vsd_sparse_decode_attn_quant(rows[:, R - 1].contiguous().cuda(), *cache.cuda(), None, None,
                                                  i32([0]), i32([P + R]), scale=2.0 ** -12, max_tail=P + R)
        assert vsd.vsd_read_device_status() == 0
        want, mag = attend(cache, [P], rows, Hkv, 2.0 ** -12)
        assert_outputs(out, want, mag)
        assert_outputs(drafts, want[:, R - 1], mag[:, R - 1])
        k = cache.kv(0, torch.arange(P))[0]
        for c, t in ((0, 0), (1, R - 1)):
            for h in range(Hq):
                x = rows[0, t, h].double()
                err = (logits[0, c, h].cpu().double() - 2.0 ** -12 * (k[:, h // 2] @ x)).abs()
                assert torch.all(err <= ref.logit_bound(x, k[:, h // 2], 2.0 ** -12))


# ------------------------------------------------------------------ rows that are skipped
@pytest.mark.parametrize("given", [None, "k", "v"])
@pytest.mark.parametrize("with_valid", [False, True])
@pytest.mark.parametrize("d", [64, 128])
def test_read_returns_zeros_for_rows_it_skips(vsd, with_valid, given, d):
    """Outputs that the call allocates hold nothing of what their memory held before, neither
    for a page whose block is bad nor for a sequence whose range leaves the table at either
    end; an output that is given keeps those rows."""
    B, n, Hkv = 5, 40, 2
    cache = ref.Cache([64] * B, Hkv, d, seed=9)
    cache.table[0, 1] = 9999
    width = cache.table.shape[1] * 16
    args, pos = cache.cuda(), i32([10, 5000, 8, -7, width - n + 1])
    nv = i32([n, n, n - 7, n, n]) if with_valid else None
    torch.cuda.synchronize()
    old = [torch.full((B, n, Hkv, d), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(8)]
    mine = torch.full((B, n, Hkv, d), 7.0, dtype=torch.bfloat16, device="cuda")
    torch.cuda.synchronize()
    del old
    got = vsd.vsd_read_kv_quant(*args, pos, n=n, n_valid=nv, **({} if given is None else {given + "_out": mine}))
    assert vsd.vsd_read_device_status() == vsd.DEV_BAD_BLOCK | vsd.DEV_BAD_LENGTH
    for kv, name in enumerate("kv"):
        want = torch.full((B, n, Hkv, d), 7.0 if given == name else 0.0, dtype=torch.bfloat16)
        for b, t0, t1 in ((0, 0, 6), (0, 22, n), (2, 0, n - 7 if with_valid else n)):
            j = int(pos[b]) + torch.arange(t0, t1)
            want[b, t0:t1] = cache.kv(b, j)[kv].float().bfloat16()
        assert torch.equal(got[kv].cpu(), want)


@pytest.mark.parametrize("n", [1, 15, 16, 17, 18, 31, 33, 50])
def test_read_zeros_every_skipped_row_and_no_other_memory(vsd, n):
    """Ranges that begin at every slot of a page, below 0 and past the table, all of them
    skipped: n rows of zeros each, and what lies around the outputs stays."""
    Hkv, d, B = 1, 64, 40
    starts = list(range(-20, 0)) + list(range(5000, 5000 + B - 20))
    cache = ref.Cache([64] * B, Hkv, d, seed=10)
    kc, vc, ks, vs, bt = cache.cuda()
    from sparse_attention_speculative_gb300._lib import Geom, load
    geom = Geom(B, Hkv, Hkv, d, 16, bt.shape[1], kc.shape[0])
    size, pad = B * n * Hkv * d, 1024
    outs = [torch.full((size + 2 * pad,), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    pos = i32(starts)
    p = lambda t: ctypes.c_void_p(t.data_ptr())  # noqa: E731
    for zeroed in (0, 1, 2, 3):
        for o in outs:
            o.fill_(7.0)
        torch.cuda.synchronize()
        assert load().vsd_read_kv_quant_zeroed(ctypes.addressof(geom), n, p(kc), p(vc), p(ks), p(vs), p(bt), p(pos), 0,
                                               None, p(outs[0][pad:]), p(outs[1][pad:]), zeroed, None) == 0
        torch.cuda.synchronize()
        assert vsd.vsd_read_device_status() == vsd.DEV_BAD_LENGTH
        for i, o in enumerate(outs):
            assert torch.all(o[:pad] == 7.0) and torch.all(o[pad + size:] == 7.0)
            assert torch.all(o[pad:pad + size] == (0.0 if zeroed >> i & 1 else 7.0))


# ------------------------------------------------------------------ value scales far apart
@pytest.mark.parametrize("gap", [0, 4, 10, 14, 20])
@pytest.mark.parametrize("at", ["first", "middle", "last"])
@pytest.mark.parametrize("call", ["verify", "draft"])
def test_value_scales_far_apart(vsd, call, at, gap):
    """One page of loud values with half of the probability, its codes zero in every other
    dimension, among 8192 equal keys of value scales 2^gap smaller: every dimension is within
    the bound of products x = p vs that are held to 2^-27 (draft step: 2^-28) of the largest.
    Where the scales are within 2^4 of each other that adds nothing that counts."""
    d, P = 64, 8192
    cache = ref.Cache([P + 1], 1, d, seed=gap + 77)
    loud = {"first": 0, "middle": P // 32, "last": P // 16 - 1}[at]
    one = ref.encode(torch.tensor([1.0], dtype=torch.float64))[0]
    for lp in range(P // 16 + 1):
        blk = int(cache.table[0, lp])
        n = min(16, P + 1 - lp * 16)
        cache.codes[0][blk, :, :n] = 0
        cache.scales[0][blk] = 1.0
        cache.scales[1][blk] = 2.0 ** -gap
    blk = int(cache.table[0, loud])
    cache.codes[0][blk, 0, :, 0] = one
    cache.scales[1][blk] = 1.0
    cache.codes[1][blk, 0, :, ::2] = 0
    q = torch.zeros((1, 1, 1, d)).bfloat16()
    q[..., 0] = 6.25                                    # 16 e^6.25 = 8288
    args = cache.cuda()
    if call == "verify":
        out = vsd.vsd_verify_attn_collect_quant(q.cuda(), *args, i32([P]), P_max=P, scale=1.0, collect=False)[0]
    else:
        idx = torch.arange(P, dtype=torch.int32, device="cuda")[None]
        out = vsd.vsd_sparse_decode_attn_quant(q[:, 0].cuda(), *args, idx, i32([P]), i32([P]), i32([P + 1]),
                                               scale=1.0, max_tail=1)
    assert vsd.vsd_read_device_status() == 0
    j = torch.arange(P + 1)
    k, v = (x[:, 0] for x in cache.kv(0, j))
    z = k @ q[0, 0, 0].double()
    want, mag = ref.softmax_av(z, v)
    vs = cache.scales[1][cache.table[0].long()[j // 16], 0].double()
    top = float((torch.softmax(z, 0) * vs).max())
    floor = 2.0 ** (-27 if call == "verify" else -28) * top * (v / vs[:, None]).abs().sum(0)
    bound = ref.out_bound(want, mag)
    assert torch.all((out.cpu().double().reshape(d) - want).abs() <= bound + floor)
    if gap <= 4:
        assert torch.all(floor <= bound / 8)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("down", [0, 1, 2, 4, 5])
def test_logits_of_rows_that_share_a_factor(vsd, d, down):
    """Rows whose largest magnitudes lie 2^down apart, their other dimensions far below and all
    of one sign against keys of one sign, so that what the queries' parts cannot hold adds up:
    each logit is within the stated 2^-18 of its row's largest (2^-22 where the rows have
    factors of their own, or the same one) times the keys' magnitudes, and fp32's sums."""
    R, Hq, P = 2, 4, 40
    cache = ref.Cache([P + R], 1, d, seed=d + down)
    for blk in cache.table[0, :3].tolist():
        for code in cache.codes[0][blk:blk + 1]:
            code &= 0x7F
            code[code == 0x7F] = 0x7E
    n = torch.arange(d)
    # 1.9921875 * 2^-k, every significant bit set, k from 8 to 23
    low = (2.0 - 2.0 ** -7) * 2.0 ** -(8.0 + n % 16)
    q = low.expand(1, R, Hq, d).clone()
    q[..., 0] = 1.5
    q[0, 1] *= 2.0 ** -down
    q = q.bfloat16()
    logits = torch.zeros((1, 2, Hq, P), device="cuda")
    vsd.vsd_verify_attn_collect_quant(q.cuda(), *cache.cuda(), i32([P]), P_max=P, scale=1.0, logits=logits)
    assert vsd.vsd_read_device_status() == 0
    k = cache.kv(0, torch.arange(P))[0][:, 0]
    for t in range(R):
        x = q[0, t, 0].double()
        held = 2.0 ** -22 if t == 0 or down in (0, 5) else 2.0 ** (-22 + down)
        bound = 2.0 ** -16 * (k.abs() @ x.abs()) + held * x.abs().max() * k.abs().sum(-1)
        err = (logits[0, t].cpu().double() - k @ x).abs()
        assert torch.all(err <= bound)


# ------------------------------------------------------------------ splits of 16 heads a group
@pytest.mark.parametrize("B,k", [(4, 1781), (4, 1800), (8, 7000), (8, 7300)])
def test_draft_of_sixteen_heads_around_its_waves(vsd, B, k):
    """Lists on both sides of the borders where a split takes one, two and four batches with 16
    heads a group (456 and 3648 CTAs)."""
    Hkv, d, G = 8, 64, 16
    tail = 5
    cache = ref.Cache([k + 50] * B, Hkv, d, seed=k)
    g = torch.Generator().manual_seed(k)
    n = [k] + [int(x) for x in torch.randint(0, k, (B - 1,), generator=g)]
    idx = torch.full((B, k), -1, dtype=torch.int32)
    for b in range(B):
        idx[b, :n[b]] = torch.randperm(k + 40, generator=g)[:n[b]].sort().values.to(torch.int32)
    q = torch.randn((B, Hkv * G, d), generator=g).bfloat16()
    out = vsd.vsd_sparse_decode_attn_quant(q.cuda(), *cache.cuda(), idx.cuda(), i32(n), i32([k + 40] * B),
                                           i32([k + 40 + tail] * B), scale=0.125, max_tail=tail).cpu().double()
    assert vsd.vsd_read_device_status() == 0
    for b in range(B):
        j = torch.cat([idx[b, :n[b]].long(), torch.arange(k + 40, k + 40 + tail)])
        kk, vv = cache.kv(b, j)
        for h in range(0, Hkv * G, 5):
            want, mag = ref.softmax_av(0.125 * (kk[:, h // G] @ q[b, h].double()), vv[:, h // G])
            assert torch.all((out[b, h] - want).abs() <= ref.out_bound(want, mag))
