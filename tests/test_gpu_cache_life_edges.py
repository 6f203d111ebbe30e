"""Calls of the rows, weights and eviction at the ends of what they allow: caches and logits past
2^31 elements, many sequences, host threads at once, many heads."""
import threading

import pytest
import torch

from tests import cache_life_ref as life
from tests import quant_ref as ref

pytestmark = pytest.mark.gpu
PAGE = 16


@pytest.fixture(scope="module")
def vsd():
    import sparse_attention_speculative_gb300 as m
    m.load()
    m.vsd_read_device_status()
    return m


@pytest.fixture(autouse=True)
def clean_status(vsd):
    yield
    vsd.vsd_read_device_status()
    torch.cuda.empty_cache()


def int32(x):
    return torch.as_tensor(x, dtype=torch.int32).cuda()


@pytest.mark.parametrize("quant", [False, True])
def test_caches_past_31_bits(vsd, quant):
    """Rows stored, weighed and moved in blocks whose elements 32 bits do not count."""
    Hkv, d, n = 8, 128, 40
    NB = 2 ** 31 // (Hkv * PAGE * d) + 8
    kind = torch.uint8 if quant else torch.bfloat16
    cache = [torch.zeros((NB, Hkv, PAGE, d), dtype=kind, device="cuda") for _ in range(2)]
    cache = [c.view(torch.float8_e4m3fn) for c in cache] if quant else cache
    scales = [torch.ones((NB, Hkv), device="cuda") for _ in range(2)] if quant else []
    top = NB - 1
    table = int32([[top, top - 1, top - 2, 0]])
    other = int32([[top - 3, top - 4]])
    g = torch.Generator().manual_seed(1)
    x = torch.randn((1, n, 3 * Hkv, d), generator=g).to(torch.bfloat16).cuda()
    q, k, v = x[:, :, :Hkv], x[:, :, Hkv:2 * Hkv], x[:, :, 2 * Hkv:]
    call = vsd.vsd_norm_rope_append_kv_quant if quant else vsd.vsd_norm_rope_append_kv
    call(q, k, v, *cache, *scales, table, int32([0]), None)

    def rows(i, blocks):
        got = cache[i][torch.as_tensor(blocks, device="cuda")]
        s = scales[i][torch.as_tensor(blocks, device="cuda")][:, :, None, None] if quant else 1.0
        return (got.float() * s).transpose(1, 2).reshape(-1, Hkv, d)

    for i, src in ((0, k), (1, v)):
        have, want = rows(i, [top, top - 1, top - 2])[:n], src[0].float()
        assert torch.all((have - want).abs() <= (2.0 ** -4 * want.abs() + 2.0 ** -8 if quant else 0))
        assert torch.all(rows(i, [0, 1]) == 0)
    # weights beside a verify block there
    w = torch.zeros((1, Hkv, 38), device="cuda")
    lg = torch.randn((1, 2, Hkv, 38), generator=g).cuda()
    qv = q[:, 38:40].contiguous()
    if quant:
        vsd.vsd_accumulate_weights_quant(lg, qv, cache[0], scales[0], table, int32([38]), w, scale=0.1)
    else:
        vsd.vsd_accumulate_weights(lg, qv, cache[0], table, int32([38]), w, scale=0.1)
    key = rows(0, [top, top - 1, top - 2])[38:40].double()
    want = torch.zeros((Hkv, 38), dtype=torch.float64, device="cuda")
    for c in range(2):
        z = torch.einsum("hd,uhd->hu", qv[0, c].double(), key[:c + 1]) * 0.1
        want += torch.softmax(torch.cat([lg[0, c].double(), z], 1), 1)[:, :38]
    assert torch.all((w[0].double() - want).abs() <= 2.0 ** -17 * want + 1e-30)
    # moved down to other blocks
    idx = torch.arange(0, 38, 2)
    before = [rows(i, [top, top - 1, top - 2])[idx.cuda()] for i in range(2)]
    call = vsd.vsd_compact_kv_quant if quant else vsd.vsd_compact_kv
    out = call(*cache, *scales, table, other, int32([38]), idx[None].int().cuda(), int32([19]), weights=w)
    for i in range(2):
        got = rows(i, [top - 3, top - 4])[:19]
        assert torch.all((got - before[i]).abs() <= (2.0 ** -4 * before[i].abs() + 2.0 ** -8 if quant else 0))
    assert torch.equal(out[0], w[0][:, idx.cuda()])
    assert vsd.vsd_read_device_status() == 0


def test_logits_past_31_bits(vsd):
    B, Hq, Hkv, d, P_max = 9, 64, 8, 64, 2 ** 21 + 4
    logits = torch.zeros((B, 2, Hq, P_max), device="cuda")
    assert logits.numel() > 2 ** 31
    g = torch.Generator().manual_seed(2)
    part = torch.randn((2, Hq, 900), generator=g)
    logits[-1, :, :, :900] = part.cuda()
    q = torch.zeros((B, 2, Hq, d), dtype=torch.bfloat16, device="cuda")
    kc = torch.zeros((60, Hkv, PAGE, d), dtype=torch.bfloat16, device="cuda")
    table = torch.arange(60, dtype=torch.int32, device="cuda").repeat(B, 1)
    w = torch.zeros((B, Hkv, P_max), device="cuda")
    vsd.vsd_accumulate_weights(logits, q, kc, table, int32([0] * (B - 1) + [900]), w, scale=1.0)
    want, bound = life.accumulated(torch.zeros((1, Hkv, 900), dtype=torch.float64), part[None], [[torch.zeros((Hq, 1)), torch.zeros((Hq, 2))]],
                                   (0, 1), [900], Hq // Hkv)
    assert torch.all((w[-1, :, :900].cpu().double() - want[0]).abs() <= bound[0])
    assert torch.all(w[:-1].amax() == 0) and torch.all(w[-1, :, 900:].amax() == 0)
    assert vsd.vsd_read_device_status() == 0


def test_the_longest_prefix_of_one_head(vsd):
    """A million positions: slices of many steps."""
    P = 2 ** 20 - 3
    g = torch.Generator(device="cuda").manual_seed(3)
    lg = torch.randn((1, 1, 1, P), generator=g, device="cuda") * 3
    q = torch.zeros((1, 1, 1, 64), dtype=torch.bfloat16, device="cuda")
    kc = torch.zeros((1, 1, PAGE, 64), dtype=torch.bfloat16, device="cuda")
    table = torch.zeros((1, 2 ** 16), dtype=torch.int32, device="cuda")
    w = torch.zeros((1, 1, P), device="cuda")
    vsd.vsd_accumulate_weights(lg, q, kc, table, int32([P]), w, scale=1.0)
    want = torch.softmax(torch.cat([lg[0, 0, 0].double(), torch.zeros(1, device="cuda", dtype=torch.float64)]), 0)[:P]
    # (the sum of a million terms, in a tree over threads: 2^-18)
    assert torch.all((w[0, 0].double() - want).abs() <= 2.0 ** -18 * want + 2.0 ** -120)


@pytest.mark.parametrize("B", [300, 5000])
def test_many_short_sequences(vsd, B):
    """More sequences than the GPU holds clusters, each of a few rows."""
    Hq, Hkv, d, R = 4, 2, 64, 2
    g = torch.Generator().manual_seed(B)
    prefix = torch.randint(0, 30, (B,), generator=g)
    table = torch.arange(B * 2, dtype=torch.int32).view(B, 2)
    bits = torch.randn((2 * B, Hkv, PAGE, d), generator=g).to(torch.bfloat16)
    q = torch.randn((B, R, Hq, d), generator=g).to(torch.bfloat16)
    lg = torch.randn((B, 2, Hq, 30), generator=g)
    w = torch.zeros((B, Hkv, 30), device="cuda")
    vsd.vsd_accumulate_weights(lg.cuda(), q.cuda(), bits.cuda(), table.cuda(), int32(prefix), w, scale=0.2)
    j = prefix[:, None] + torch.arange(R)
    key = bits[table.long().gather(1, j // PAGE), :, j % PAGE].double().repeat_interleave(2, 2)        # [B, R, Hq, d]
    z = torch.einsum("bchd,buhd->bchu", q.double(), key) * 0.2
    z = torch.where(torch.arange(R) <= torch.arange(R)[:, None, None], z, -torch.inf)
    past = torch.where(torch.arange(30) < prefix[:, None, None, None], lg.double(), -torch.inf)
    want = torch.softmax(torch.cat([past, z], 3), 3)[..., :30].view(B, 2, Hkv, 2, 30).sum((1, 3))
    assert torch.all((w.cpu().double() - want).abs() <= 2.0 ** -17 * want + 1e-30)
    # every second row kept, in place
    n = (prefix + 1) // 2
    idx = torch.where(torch.arange(15) < n[:, None], 2 * torch.arange(15), -1).int()
    kc, vc = bits.cuda(), (-bits).cuda()
    out = vsd.vsd_compact_kv(kc, vc, table.cuda(), table.cuda(), int32(prefix), idx.cuda(), int32(n), weights=w)
    at = torch.arange(15)
    src = bits[table.long().gather(1, (idx.clamp(min=0) // PAGE).long()), :, idx.clamp(min=0).long() % PAGE]   # [B, 15, Hkv, d]
    keep = (at < n[:, None])
    got = kc.cpu()[table[:, 0].long(), :, :15].transpose(1, 2)
    assert torch.equal(got[keep], src[keep])
    assert torch.equal(vc.cpu()[table[:, 0].long(), :, :15].transpose(1, 2)[keep], -src[keep])
    ww = w.cpu().gather(2, idx.clamp(min=0).long()[:, None].expand(B, Hkv, 15))
    assert torch.equal(out.cpu(), torch.where(keep[:, None], ww, 0.0))
    # one token each, 8 bit
    codes = [torch.zeros((2 * B, Hkv, PAGE, d), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn) for _ in range(2)]
    scales = [torch.zeros((2 * B, Hkv), device="cuda") for _ in range(2)]
    rows = q[:, :1, :Hkv].contiguous().cuda()
    vsd.vsd_norm_rope_append_kv_quant(q[:, :1].cuda(), rows, rows, *codes, *scales, table.cuda(), int32(prefix), None)
    k2 = [torch.zeros_like(c.view(torch.uint8)).view(torch.float8_e4m3fn) for c in codes]
    s2 = [torch.zeros_like(s) for s in scales]
    vsd.vsd_append_kv_quant(rows, rows, *k2, *s2, table.cuda(), int32(prefix))
    for a, b in zip(codes + scales, k2 + s2):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    assert vsd.vsd_read_device_status() == 0


def test_many_heads_a_token(vsd):
    """Query heads by the hundred, groups of 16 and KV heads that blocks of four do not divide."""
    for Hq, Hkv, d in ((128, 8, 128), (80, 5, 64), (7, 7, 128)):
        g = torch.Generator().manual_seed(Hq)
        x = torch.randn((2, 20, Hq + 2 * Hkv, d), generator=g).to(torch.bfloat16)
        y = x.cuda()
        freq = life.inv_freq(d)
        turns = vsd.vsd_rope_turns(freq)
        parts = (y[:, :, :Hq], y[:, :, Hq:Hq + Hkv], y[:, :, Hq + Hkv:])
        table = int32([[0, 1, 2], [5, 4, 3]])
        kc, vc = (torch.zeros((6, Hkv, PAGE, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
        q = vsd.vsd_norm_rope_append_kv(*parts, kc, vc, table, int32([3, 28]), turns)
        codes = [torch.zeros((6, Hkv, PAGE, d), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn) for _ in range(2)]
        scales = [torch.ones((6, Hkv), device="cuda") for _ in range(2)]
        q8 = vsd.vsd_norm_rope_append_kv_quant(*parts, *codes, *scales, table, int32([3, 28]), turns)
        assert torch.equal(q, q8)
        for b, p in ((0, 3), (1, 28)):
            want, off = life.turned(x[b, :, :Hq].double(), None, 0, range(p, p + 20), freq, False)
            assert torch.all((q[b].cpu().double() - want).abs() <= life.bf16_bound(want, off))
            want, off = life.turned(x[b, :, Hq:Hq + Hkv].double(), None, 0, range(p, p + 20), freq, False)
            j = p + torch.arange(20)
            blk = table[b].cpu().long()[j // PAGE]
            assert torch.all((kc.cpu()[blk, :, j % PAGE].double() - want).abs() <= life.bf16_bound(want, off))
            s = scales[0].cpu()[blk].double()[:, :, None]
            have = ref.decode(codes[0].view(torch.uint8).cpu()[blk, :, j % PAGE]) * s
            assert torch.all((have - want).abs() <= 2.0 ** -4 * want.abs() + 2.0 ** -10 * s + 1.1 * off)
    assert vsd.vsd_read_device_status() == 0


def test_host_threads_at_once(vsd):
    """The calls from several host threads, each on a stream of its own: the results of one alone."""
    B, Hq, Hkv, d, n = 2, 8, 2, 64, 33
    turns = vsd.vsd_rope_turns(life.inv_freq(d))
    table = int32([[0, 1, 2, 3], [7, 6, 5, 4]])
    pos = int32([1, 20])

    def work(seed, stream=None):
        g = torch.Generator(device="cuda").manual_seed(seed)
        with torch.cuda.stream(stream or torch.cuda.current_stream()):
            x = torch.randn((B, n, Hq + 2 * Hkv, d), generator=g, device="cuda").to(torch.bfloat16)
            codes = [torch.zeros((8, Hkv, PAGE, d), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn) for _ in range(2)]
            scales = [torch.ones((8, Hkv), device="cuda") for _ in range(2)]
            out = []
            for _ in range(20):
                q = vsd.vsd_norm_rope_append_kv_quant(x[:, :, :Hq], x[:, :, Hq:Hq + Hkv], x[:, :, Hq + Hkv:], *codes,
                                                      *scales, table, pos, turns)
                lg = torch.randn((B, 2, Hq, 40), generator=g, device="cuda")
                w = torch.zeros((B, Hkv, 40), device="cuda")
                vsd.vsd_accumulate_weights_quant(lg, q[:, :2].contiguous(), codes[0], scales[0], table, int32([30, 40]), w,
                                                 scale=0.1)
                idx, ns, _ = vsd.vsd_select_topk(w, int32([30, 40]), k=24, n_sink=2, n_recent=4)
                w = vsd.vsd_compact_kv_quant(*codes, *scales, table, table, int32([30, 40]), idx, ns, weights=w)
                out += [q, w, idx]
            torch.cuda.current_stream().synchronize()
            return out + [c.view(torch.uint8) for c in codes] + scales

    want = [work(s) for s in range(4)]
    got = [None] * 4

    def run(s):
        got[s] = work(s, torch.cuda.Stream())
    threads = [threading.Thread(target=run, args=(s,)) for s in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for a, b in zip(want, got):
        assert b is not None and all(torch.equal(x, y) for x, y in zip(a, b))
