"""Normed and rotated rows, alone and stored in either cache, against the definition in 64 bits."""
import math

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


def bf16(x):
    return x.to(torch.bfloat16)


def weights_of(g, d, norm):
    if not norm:
        return None, None
    return tuple(bf16(1 + 0.3 * torch.randn(d, generator=g)) for _ in range(2))


def projection(g, B, n, Hq, Hkv, d, fused):
    """q, k, v on the CPU, and on the GPU as views of one product (or tensors of their own)."""
    x = bf16(torch.randn((B, n, Hq + 2 * Hkv, d), generator=g) * torch.exp(torch.randn((B, n, 1, 1), generator=g)))
    cpu = x[:, :, :Hq], x[:, :, Hq:Hq + Hkv], x[:, :, Hq + Hkv:]
    y = x.cuda()
    gpu = (y[:, :, :Hq], y[:, :, Hq:Hq + Hkv], y[:, :, Hq + Hkv:]) if fused else [z.cuda().contiguous() for z in cpu]
    return cpu, gpu


def cuda(x):
    return None if x is None else x.cuda()


def int32(x):
    return torch.as_tensor(x, dtype=torch.int32).cuda()


def check_rows(got, x, weight, pos, freq, inter, amp=1.0, eps=1e-6):
    want, off = life.turned(x.double(), weight, eps, pos, freq, inter, amp)
    assert torch.all((got.double() - want).abs() <= life.bf16_bound(want, off))


SHAPES = [  # B, n, Hq, Hkv, d, rot, interleaved, norm, fused
    (1, 1, 1, 1, 128, 128, False, True, True),
    (1, 1, 1, 1, 64, 64, True, False, False),
    (3, 5, 8, 2, 128, 128, False, True, True),
    (2, 7, 8, 1, 64, 64, False, True, False),
    (2, 3, 4, 4, 128, 64, False, False, True),
    (2, 3, 4, 4, 128, 32, True, True, True),
    (1, 33, 16, 2, 64, 16, True, True, False),
    (1, 2, 64, 8, 128, 8, False, True, True),
    (4, 1, 32, 8, 128, 0, False, True, True),
    (1, 301, 32, 8, 128, 128, True, True, True),
    (1, 2500, 8, 4, 64, 64, False, True, True),    # a warp takes a whole token
]


@pytest.mark.parametrize("B,n,Hq,Hkv,d,rot,inter,norm,fused", SHAPES)
def test_rows(vsd, B, n, Hq, Hkv, d, rot, inter, norm, fused):
    g = torch.Generator().manual_seed(B * n + d + rot)
    cpu, gpu = projection(g, B, n, Hq, Hkv, d, fused)
    wq, wk = weights_of(g, d, norm)
    freq = life.inv_freq(rot)
    base = [17 + 1000 * b for b in range(B)]
    q, k = vsd.vsd_norm_rope(gpu[0], gpu[1], vsd.vsd_rope_turns(freq) if rot else None, int32(base), pos_offset=3,
                             q_weight=cuda(wq), k_weight=cuda(wk), interleaved=inter)
    for b in range(B):
        pos = [base[b] + 3 + t for t in range(n)]
        check_rows(q[b].cpu(), cpu[0][b], wq, pos, freq, inter)
        check_rows(k[b].cpu(), cpu[1][b], wk, pos, freq, inter)
    assert vsd.vsd_read_device_status() == 0


@pytest.mark.parametrize("only", ["q", "k"])
def test_one_weight_alone(vsd, only):
    g = torch.Generator().manual_seed(5)
    cpu, gpu = projection(g, 2, 3, 4, 2, 128, True)
    w = weights_of(g, 128, True)[0]
    freq = life.inv_freq(128)
    q, k = vsd.vsd_norm_rope(gpu[0], gpu[1], vsd.vsd_rope_turns(freq), int32([0, 9]), eps=1e-3,
                             q_weight=cuda(w) if only == "q" else None, k_weight=cuda(w) if only == "k" else None)
    for b, p in ((0, 0), (1, 9)):
        check_rows(q[b].cpu(), cpu[0][b], w if only == "q" else None, range(p, p + 3), freq, False, eps=1e-3)
        check_rows(k[b].cpu(), cpu[1][b], w if only == "k" else None, range(p, p + 3), freq, False, eps=1e-3)


@pytest.mark.parametrize("base,offset", [(131072, 0), (2 ** 31 - 10, 2 ** 31 - 1), (-7, 0), (0, -(2 ** 31))])
@pytest.mark.parametrize("amp", [1.0, 1.25, -0.5])
def test_far_positions(vsd, base, offset, amp):
    """Angles stay exact at any position that the arguments can name."""
    g = torch.Generator().manual_seed(6)
    cpu, gpu = projection(g, 1, 9, 2, 2, 128, True)
    freq = life.inv_freq(128, 10000.0)
    q, k = vsd.vsd_norm_rope(gpu[0], gpu[1], vsd.vsd_rope_turns(freq), int32([base]), pos_offset=offset, amplitude=amp)
    pos = [base + offset + t for t in range(9)]
    # (the reference's own angle: a product of 32 and 53 bits, 2^-21 of a radian at 2^32)
    want, off = life.turned(cpu[0][0].double(), None, 0, pos, freq, False, amp)
    far = abs(amp) * 2.0 ** -20 * cpu[0][0].double().abs().amax(-1, keepdim=True) * (abs(base + offset) > 2 ** 30)
    assert torch.all((q[0].cpu().double() - want).abs() <= life.bf16_bound(want, off) + 2 * far)


def test_queries_alone_and_in_place(vsd):
    g = torch.Generator().manual_seed(7)
    cpu, gpu = projection(g, 2, 4, 8, 2, 64, False)
    freq = life.inv_freq(64)
    turns = vsd.vsd_rope_turns(freq)
    alone, none = vsd.vsd_norm_rope(gpu[0], None, turns, int32([3, 4]))
    assert none is None
    both = vsd.vsd_norm_rope(gpu[0], gpu[1], turns, int32([3, 4]))
    assert torch.equal(both[0], alone)
    q, k = vsd.vsd_norm_rope(gpu[0], gpu[1], turns, int32([3, 4]), q_out=gpu[0], k_out=gpu[1])
    assert q.data_ptr() == gpu[0].data_ptr() and torch.equal(q, both[0]) and torch.equal(k, both[1])
    # one token's projection: its parts are contiguous, and may be turned where they are
    x = torch.randn((1, 1, 12, 64), generator=g).to(torch.bfloat16)
    y = x.cuda()
    want = vsd.vsd_norm_rope(y[:, :, :8], y[:, :, 8:10], turns, int32([9]))
    vsd.vsd_norm_rope(y[:, :, :8], y[:, :, 8:10], turns, int32([9]), q_out=y[:, :, :8], k_out=y[:, :, 8:10])
    assert torch.equal(y[:, :, :8], want[0]) and torch.equal(y[:, :, 8:10], want[1]) and torch.equal(y[:, :, 10:].cpu(), x[:, :, 10:])
    # other memory of the rows is refused
    y = torch.zeros((2, 4, 12, 64), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(vsd.VsdError):
        vsd.vsd_norm_rope(y[:, :, :8], None, turns, int32([3, 4]), q_out=y.view(-1)[:2 * 4 * 8 * 64].view(2, 4, 8, 64))
    with pytest.raises(vsd.VsdError):
        vsd.vsd_norm_rope(y.view(-1)[:2 * 4 * 4 * 64].view(2, 4, 4, 64), None, turns, int32([3, 4]),
                          q_out=y.view(-1)[64:2 * 4 * 4 * 64 + 64].view(2, 4, 4, 64))
    # one row for all: strides of 0
    one = cpu[0][:1, :1].cuda().expand(2, 4, 8, 64)
    many = vsd.vsd_norm_rope(one, None, turns, int32([3, 4]))[0]
    assert torch.equal(many, vsd.vsd_norm_rope(one.contiguous(), None, turns, int32([3, 4]))[0])


def test_counts(vsd):
    """Rows behind n_valid: left in given outputs, zeros in new ones; a bad count is 0 and flagged."""
    g = torch.Generator().manual_seed(8)
    cpu, gpu = projection(g, 4, 6, 4, 2, 128, True)
    freq = life.inv_freq(128)
    turns = vsd.vsd_rope_turns(freq)
    valid = [6, 0, 4, 7]
    full = vsd.vsd_norm_rope(gpu[0], gpu[1], turns, int32([0] * 4))
    given = [torch.full_like(x, 7.0) for x in full]
    vsd.vsd_read_device_status()
    new = vsd.vsd_norm_rope(gpu[0], gpu[1], turns, int32([0] * 4), n_valid=int32(valid))
    kept = vsd.vsd_norm_rope(gpu[0], gpu[1], turns, int32([0] * 4), n_valid=int32(valid), q_out=given[0], k_out=given[1])
    assert vsd.vsd_read_device_status() == vsd.DEV_BAD_LENGTH
    for whole, a, b in zip(full, new, kept):
        for i, v in enumerate(valid):
            v = v if v <= 6 else 0
            assert torch.equal(a[i, :v], whole[i, :v]) and torch.equal(b[i, :v], whole[i, :v])
            assert torch.all(a[i, v:] == 0) and torch.all(b[i, v:] == 7)
    # one output given, the other new
    mixed = vsd.vsd_norm_rope(gpu[0], gpu[1], turns, int32([0] * 4), n_valid=int32(valid), q_out=torch.full_like(full[0], 7.0))
    assert torch.equal(mixed[0], kept[0]) and torch.equal(mixed[1], new[1])


@pytest.mark.parametrize("inter", [False, True])
def test_values_that_are_not_finite(vsd, inter):
    """An infinity or a NaN stays in its pair where nothing is normed, and never leaves the
    dimensions behind rot_dim; a row of them becomes NaN where it is."""
    x = torch.ones((1, 1, 3, 64), dtype=torch.bfloat16)
    x[0, 0, 0, 5] = math.inf
    x[0, 0, 1, 40] = math.nan
    x[0, 0, 1, 50] = -math.inf
    freq = life.inv_freq(32)
    turns = vsd.vsd_rope_turns(freq)
    y = vsd.vsd_norm_rope(x.cuda(), None, turns, int32([3]), interleaved=inter)[0].cpu()[0, 0]
    pair = {4, 5} if inter else {5, 21}
    assert set(torch.nonzero(~torch.isfinite(y[0])).flatten().tolist()) == pair
    assert torch.isnan(y[1, 40]) and y[1, 50] == -math.inf and torch.isfinite(y[1]).sum() == 62
    w = bf16(torch.ones(64)).cuda()
    y = vsd.vsd_norm_rope(x.cuda(), None, turns, int32([3]), q_weight=w, interleaved=inter)[0].cpu()[0, 0]
    assert torch.isnan(y[0, 5 if inter else 21]) and torch.all(torch.isnan(y[1, 33:48]) | (y[1, 33:48] == 0))
    assert torch.all(torch.isfinite(y[2]))
    # zeros: the norm's eps carries the row; squares beyond fp32: zeros
    z = torch.zeros((1, 1, 2, 64), dtype=torch.bfloat16)
    z[0, 0, 1] = 1e30
    y = vsd.vsd_norm_rope(z.cuda(), None, turns, int32([3]), q_weight=w, interleaved=inter)[0]
    assert torch.all(y == 0)


def bf16_cache(g, NB, Hkv, d):
    return [bf16(torch.randn((NB, Hkv, PAGE, d), generator=g)) for _ in range(2)]


CACHED = [  # B, n, Hq, Hkv, d, rot, inter, norm, start
    (1, 1, 4, 1, 128, 128, False, True, 0),
    (5, 1, 8, 2, 64, 64, False, True, 15),
    (3, 6, 16, 2, 128, 128, True, False, 30),
    (2, 40, 4, 4, 64, 32, False, True, 9),
    (1, 700, 8, 8, 128, 128, False, True, 0),
]


@pytest.mark.parametrize("B,n,Hq,Hkv,d,rot,inter,norm,start", CACHED)
def test_bf16_cache(vsd, B, n, Hq, Hkv, d, rot, inter, norm, start):
    """Keys and values at their places, nothing else touched, positions of the rotation apart
    from those in the cache."""
    g = torch.Generator().manual_seed(n + d)
    cpu, gpu = projection(g, B, n, Hq, Hkv, d, True)
    wq, wk = weights_of(g, d, norm)
    freq = life.inv_freq(rot)
    valid = [max(0, n - 3 * b) for b in range(B)]
    pos = [start + 5 * b for b in range(B)]
    turn_at = [100000 + 7 * b for b in range(B)]
    table, spare = life.tables([p + n for p in pos], g)
    NB = int(table.max()) + 1 if not len(spare) else max(int(table.max()), int(spare.max())) + 1
    caches = bf16_cache(g, NB, Hkv, d)
    dev = [c.cuda() for c in caches]
    q = vsd.vsd_norm_rope_append_kv(*gpu, *dev, table.cuda(), int32([p - 2 for p in pos]), vsd.vsd_rope_turns(freq),
                                    pos_offset=2, rope_base=int32(turn_at), n_valid=int32(valid), q_weight=cuda(wq),
                                    k_weight=cuda(wk), interleaved=inter)
    assert vsd.vsd_read_device_status() == 0
    got = [c.cpu() for c in dev]
    for b in range(B):
        at = [turn_at[b] + 2 + t for t in range(valid[b])]
        check_rows(q[b, :valid[b]].cpu(), cpu[0][b, :valid[b]], wq, at, freq, inter)
        assert torch.all(q[b, valid[b]:] == 0)
        j = pos[b] + torch.arange(valid[b])
        blk = table[b].long()[j // PAGE]
        check_rows(got[0][blk, :, j % PAGE], cpu[1][b, :valid[b]], wk, at, freq, inter)
        assert torch.equal(got[1][blk, :, j % PAGE], cpu[2][b, :valid[b]])
        for c, o in zip(got, caches):
            c[blk, :, j % PAGE] = o[blk, :, j % PAGE]
    assert all(torch.equal(c, o) for c, o in zip(got, caches))
    # the same as the two calls that it joins
    two = [c.cuda() for c in caches]
    if B == 1:
        q2, k2 = vsd.vsd_norm_rope(gpu[0], gpu[1], vsd.vsd_rope_turns(freq), int32(turn_at), pos_offset=2,
                                   q_weight=cuda(wq), k_weight=cuda(wk), interleaved=inter)
        vsd.vsd_append_kv(k2, gpu[2].contiguous(), *two, table.cuda(), int32(pos))
        assert torch.equal(q, q2) and all(torch.equal(x, y) for x, y in zip(dev, two))


def test_values_keep_their_bits(vsd):
    """v passes as it is, NaN payloads and infinities among it."""
    bits = torch.randint(-2 ** 15, 2 ** 15, (1, 17, 2, 64), generator=torch.Generator().manual_seed(1)).to(torch.int16)
    v = bits.view(torch.bfloat16).cuda()
    z = torch.zeros((1, 17, 2, 64), dtype=torch.bfloat16, device="cuda")
    kc, vc = (torch.zeros((2, 2, PAGE, 64), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    vsd.vsd_norm_rope_append_kv(z, z, v, kc, vc, int32([[1, 0]]), int32([0]), vsd.vsd_rope_turns(life.inv_freq(64)))
    got = torch.cat([vc[1], vc[0]], 1)[:, :17].transpose(0, 1)
    assert torch.equal(got.view(torch.int16).cpu(), bits[0])


def test_bf16_cache_bad_places(vsd):
    """Rows outside the table and pages outside the cache are skipped and flagged, the others
    stored; queries come out all the same."""
    g = torch.Generator().manual_seed(3)
    cpu, gpu = projection(g, 3, 4, 4, 2, 64, True)
    turns = vsd.vsd_rope_turns(life.inv_freq(64))
    table = int32([[0, 1], [5, 2], [3, -1]])
    want_q = vsd.vsd_norm_rope(gpu[0], gpu[1], turns, int32([30, 14, 14]))[0]
    kc, vc = (torch.zeros((5, 2, PAGE, 64), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    q = vsd.vsd_norm_rope_append_kv(*gpu, kc, vc, table, int32([30, 14, 14]), turns)
    assert vsd.vsd_read_device_status() == vsd.DEV_BAD_BLOCK | vsd.DEV_BAD_LENGTH
    assert torch.equal(q, want_q)
    assert torch.equal(vc[1, :, 14:].transpose(0, 1), gpu[2][0, :2])       # rows 30, 31; 32, 33 have no page
    assert torch.equal(vc[2, :, :2].transpose(0, 1), gpu[2][1, 2:])        # rows 16, 17; 14, 15 in block 5 of 5
    assert torch.equal(vc[3, :, 14:].transpose(0, 1), gpu[2][2, :2])
    vc[1, :, 14:] = vc[2, :, :2] = vc[3, :, 14:] = 0
    assert torch.all(vc == 0)
    # below zero
    q = vsd.vsd_norm_rope_append_kv(*gpu, kc, vc, table, int32([-4, -4, -4]), turns)
    assert vsd.vsd_read_device_status() == vsd.DEV_BAD_LENGTH and torch.all(vc == 0)


@pytest.mark.parametrize("B,n,Hq,Hkv,d,rot,inter,norm,start", CACHED + [(2, 9, 8, 2, 128, 64, False, False, 7)])
@pytest.mark.parametrize("power", [True, False])
def test_8bit_cache(vsd, B, n, Hq, Hkv, d, rot, inter, norm, start, power):
    """The scale of a page from its turned rows, codes within half a step of them, earlier rows
    kept or requantised; the values' pages bit for bit as vsd_append_kv_quant stores them."""
    g = torch.Generator().manual_seed(n + d + power)
    cpu, gpu = projection(g, B, n, Hq, Hkv, d, True)
    wq, wk = weights_of(g, d, norm)
    freq = life.inv_freq(rot)
    valid = [max(0, n - 3 * b) for b in range(B)]
    pos = [start + 5 * b for b in range(B)]
    turn_at = [100000 + 7 * b for b in range(B)]
    cache = ref.Cache([p + n for p in pos], Hkv, d, seed=n, power_of_two=power)
    for s in cache.scales:      # (a scale of every page: earlier rows have one; some small, so that it must grow)
        s.copy_(torch.where(torch.isnan(s), torch.ones(()), s))
        s[::3] *= 2.0 ** -10
    turns = vsd.vsd_rope_turns(freq)
    dev, two = cache.cuda(), cache.cuda()
    dev = [x.clone() for x in dev]
    q = vsd.vsd_norm_rope_append_kv_quant(*gpu, *dev, int32(pos), turns, rope_base=int32(turn_at),
                                          n_valid=int32(valid), q_weight=cuda(wq), k_weight=cuda(wk),
                                          interleaved=inter)
    assert vsd.vsd_read_device_status() == 0
    for b in range(B):
        at = [turn_at[b] + t for t in range(valid[b])]
        check_rows(q[b, :valid[b]].cpu(), cpu[0][b, :valid[b]], wq, at, freq, inter)
    # values: the existing call's
    vsd.vsd_append_kv_quant(gpu[1].contiguous(), gpu[2].contiguous(), *two, int32(pos), n_valid=int32(valid))
    assert torch.equal(dev[1].view(torch.uint8), two[1].view(torch.uint8)) and torch.equal(dev[3], two[3])
    codes, scales = dev[0].view(torch.uint8).cpu(), dev[2].cpu()
    was_codes, was_scales = cache.codes[0].clone(), cache.scales[0].clone()
    for b in range(B):
        if not valid[b]:
            continue
        at = [turn_at[b] + t for t in range(valid[b])]
        want, off = life.turned(cpu[1][b, :valid[b]].double(), wk, 1e-6, at, freq, inter)
        t = 0
        while t < valid[b]:
            p = pos[b] + t
            s0, s1 = p % PAGE, min(PAGE, p % PAGE + valid[b] - t)
            blk = int(cache.table[b, p // PAGE])
            for h in range(Hkv):
                x, o = want[t:t + s1 - s0, h], off[t:t + s1 - s0, h]
                top = float(x.abs().max())
                now, was = float(scales[blk, h]), float(was_scales[blk, h])
                err = float(o.max()) + 2.0 ** -40 * top
                may = {ref.page_scale(top - err), ref.page_scale(top), ref.page_scale(top + err)}
                if s0 and was and top + err <= was * 448:
                    may = {was}
                elif s0 and was and top - err <= was * 448:
                    may.add(was)
                assert now in may
                have = ref.decode(codes[blk, h, s0:s1]) * now
                # half a step of e4m3: 2^-4 of the value, 2^-10 of the scale below the smallest normal
                assert torch.all((have - x).abs() <= 2.0 ** -4 * x.abs() + 2.0 ** -10 * now + 1.1 * o)
                if s0:
                    old = was_codes[blk, h, :s0]
                    if now != was:
                        ratio = (torch.tensor(was) / torch.tensor(now))        # (fp32, as the product)
                        old = ref.encode((ref.decode(old).float() * ratio).double())
                    assert torch.equal(ref.decode(codes[blk, h, :s0]), ref.decode(old))
                was_codes[blk, h, :s1], was_scales[blk, h] = codes[blk, h, :s1], scales[blk, h]
            t += s1 - s0
    assert torch.equal(codes, was_codes) and torch.equal(scales, was_scales)      # nothing else was written


def test_8bit_cache_odd_values(vsd):
    """NaN and infinities become NaN and do not set the scale; rows of zeros; a page of scale 0."""
    n, d = 4, 64
    k = torch.zeros((1, n, 1, d), dtype=torch.bfloat16)
    k[0, 0, 0, 0], k[0, 0, 0, 7], k[0, 1, 0, 3], k[0, 2, 0, 1] = math.inf, 5.0, math.nan, -3.0
    q = k.cuda()
    codes = [torch.zeros((1, 1, PAGE, d), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn) for _ in range(2)]
    scales = [torch.zeros((1, 1), device="cuda") for _ in range(2)]
    vsd.vsd_norm_rope_append_kv_quant(q, q, q, *codes, *scales, int32([[0]]), int32([1]), None)
    for c, s in zip(codes, scales):
        assert s.item() == ref.page_scale(5.0)
        x = ref.decode(c.view(torch.uint8).cpu()[0, 0]) * s.item()
        assert torch.isnan(x[1, 0]) and torch.isnan(x[2, 3]) and x[1, 7] == 5 and x[3, 1] == -3
        assert torch.isnan(x).sum() == 2 and torch.all(x[4] == 0)
    vsd.vsd_norm_rope_append_kv_quant(q[:, 3:], q[:, 3:], q[:, 3:], *codes, *scales, int32([[0]]), int32([0]), None)
    assert all(s.item() == 2.0 ** -126 for s in scales)
    assert torch.all(torch.stack(codes).float()[:, :, :, 0] == 0)


def test_8bit_cache_refused_ranges(vsd):
    g = torch.Generator().manual_seed(4)
    cpu, gpu = projection(g, 3, 4, 4, 2, 64, True)
    turns = vsd.vsd_rope_turns(life.inv_freq(64))
    codes = [torch.zeros((4, 2, PAGE, 64), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn) for _ in range(2)]
    scales = [torch.ones((4, 2), device="cuda") for _ in range(2)]
    want_q = vsd.vsd_norm_rope(gpu[0], None, turns, int32([30, 14, 3]))[0]
    q = vsd.vsd_norm_rope_append_kv_quant(*gpu, *codes, *scales, int32([[0, 1], [9, 2], [3, -1]]), int32([30, 14, 3]),
                                          turns)
    assert vsd.vsd_read_device_status() == vsd.DEV_BAD_BLOCK | vsd.DEV_BAD_LENGTH
    assert torch.equal(q, want_q)
    raw = [c.view(torch.uint8) for c in codes]
    assert all(torch.all(r[:2] == 0) and torch.any(r[2, :, :2] != 0) and torch.any(r[3, :, 3:7] != 0) for r in raw)
    assert all(torch.all(r[2, :, 2:] == 0) and torch.all(r[3, :, 7:] == 0) for r in raw)


def test_another_stream_and_a_captured_graph(vsd):
    """One graph, replayed on other inputs, beside eager calls on another stream."""
    B, n, Hq, Hkv, d = 2, 3, 8, 2, 128
    g = torch.Generator().manual_seed(11)
    turns = vsd.vsd_rope_turns(life.inv_freq(d))
    table, _ = life.tables([40, 40], g)
    NB = 8
    sets = [[x.contiguous() for x in projection(g, B, n, Hq, Hkv, d, False)[1]] for _ in range(3)]
    pos = int32([5, 9])
    want = []
    for s in sets:
        c = [torch.zeros((NB, Hkv, PAGE, d), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        want.append([vsd.vsd_norm_rope_append_kv(*s, *c, table.cuda(), pos, turns), *c])
    cache = [torch.zeros((NB, Hkv, PAGE, d), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    ins = [torch.zeros_like(x) for x in sets[0]]
    tab = table.cuda()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = vsd.vsd_norm_rope_append_kv(*ins, *cache, tab, pos, turns)
    side = torch.cuda.Stream()
    for s, w in zip(sets, want):
        for x, y in zip(ins, s):
            x.copy_(y)
        for c in cache:
            c.zero_()
        graph.replay()
        side.wait_stream(torch.cuda.current_stream())
        mine = [torch.zeros_like(c) for c in cache]
        side.wait_stream(torch.cuda.current_stream())
        eager = vsd.vsd_norm_rope_append_kv(*s, *mine, tab, pos, turns, stream=side)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip([out, *cache], w))
        assert all(torch.equal(a, b) for a, b in zip([eager, *mine], w))


def test_empty_calls(vsd):
    turns = vsd.vsd_rope_turns(life.inv_freq(64))
    q = torch.zeros((0, 3, 4, 64), dtype=torch.bfloat16, device="cuda")
    assert vsd.vsd_norm_rope(q, q, turns, int32([]))[0].shape == q.shape
    q = torch.zeros((2, 0, 4, 64), dtype=torch.bfloat16, device="cuda")
    assert vsd.vsd_norm_rope(q, q, turns, int32([0, 0]))[1].shape == q.shape
    c = torch.zeros((1, 4, PAGE, 64), dtype=torch.bfloat16, device="cuda")
    assert vsd.vsd_norm_rope_append_kv(q, q, q, c, c.clone(), int32([[0], [0]]), int32([0, 0]), turns).shape == q.shape


def test_mismatched_tensors(vsd):
    q = torch.zeros((2, 3, 4, 64), dtype=torch.bfloat16, device="cuda")
    k = q[:, :, :2].contiguous()
    turns = vsd.vsd_rope_turns(life.inv_freq(64))
    c = torch.zeros((4, 2, PAGE, 64), dtype=torch.bfloat16, device="cuda")
    bt, pos = int32([[0, 1], [2, 3]]), int32([0, 0])
    w = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError):
        vsd.vsd_norm_rope(q, k[:, :2], turns, pos)
    with pytest.raises(ValueError):
        vsd.vsd_norm_rope(q, k[:1], turns, pos)
    with pytest.raises(ValueError):
        vsd.vsd_norm_rope(q, k, turns, pos[:1])
    with pytest.raises(ValueError, match="strides"):
        vsd.vsd_norm_rope(torch.zeros((2, 3, 4, 68), dtype=torch.bfloat16, device="cuda")[..., :64], None, turns, pos)
    with pytest.raises(ValueError, match="contiguous"):
        vsd.vsd_norm_rope(torch.zeros((2, 3, 64, 64), dtype=torch.bfloat16, device="cuda").transpose(2, 3)[:, :, :4],
                          None, turns, pos)
    with pytest.raises(TypeError):
        vsd.vsd_norm_rope(q, k, turns.int(), pos)
    with pytest.raises(TypeError):
        vsd.vsd_norm_rope(q, k, turns, pos, q_weight=w.float())
    with pytest.raises(ValueError):
        vsd.vsd_norm_rope(q, k, turns, pos, k_weight=w[:32])
    with pytest.raises(vsd.VsdError):
        vsd.vsd_norm_rope(q, k, vsd.vsd_rope_turns(life.inv_freq(128)), pos)      # rot_dim above head_dim
    with pytest.raises(vsd.VsdError):
        vsd.vsd_norm_rope(q, k, turns[:6].contiguous(), pos)                      # 12
    with pytest.raises(ValueError):
        vsd.vsd_norm_rope(q, k, turns, pos, q_out=k)
    with pytest.raises(ValueError):
        vsd.vsd_norm_rope_append_kv(q, q, k, c, c.clone(), bt, pos, turns)
    with pytest.raises(ValueError):
        vsd.vsd_norm_rope_append_kv(q, k, k, c, c.clone(), bt[:1], pos, turns)
    with pytest.raises(ValueError):
        vsd.vsd_norm_rope_append_kv(q, k, k, c, c[:3], bt, pos, turns)
    with pytest.raises(TypeError):
        vsd.vsd_norm_rope_append_kv(q, None, k, c, c.clone(), bt, pos, turns)
    with pytest.raises(TypeError):
        vsd.vsd_norm_rope_append_kv(q, k, k, c.float(), c.float(), bt, pos, turns)


@pytest.mark.parametrize("d,inter", [(128, False), (64, True)])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (3, 3), (4, 1), (10, 5), (28, 7), (96, 12)])
@pytest.mark.parametrize("B,n", [(1, 1), (3, 2), (5, 97), (1, 1531), (2, 1700)])
def test_numbers_of_heads_and_tokens(vsd, B, n, Hq, Hkv, d, inter):
    """Parts of a token, tokens and several tokens a block, the last block not full, counts that end
    inside a block: the rows of the formula, and the same bits by each of the calls."""
    g = torch.Generator().manual_seed(B * n + Hq)
    cpu, gpu = projection(g, B, n, Hq, Hkv, d, True)
    wq, wk = weights_of(g, d, True)
    freq = life.inv_freq(d)
    turns = vsd.vsd_rope_turns(freq)
    valid = [max(0, n - 1 - 5 * b) if n > 1 else n for b in range(B)]
    base = [1 + 40 * b for b in range(B)]
    how = dict(n_valid=int32(valid), q_weight=cuda(wq), k_weight=cuda(wk), interleaved=inter)
    q, k = vsd.vsd_norm_rope(gpu[0], gpu[1], turns, int32(base), **how)
    for b in range(B):
        t = valid[b]
        pos = [base[b] + j for j in range(t)]
        check_rows(q[b, :t].cpu(), cpu[0][b, :t], wq, pos, freq, inter)
        check_rows(k[b, :t].cpu(), cpu[1][b, :t], wk, pos, freq, inter)
        assert torch.all(q[b, t:] == 0) and torch.all(k[b, t:] == 0)
    pages = (max(base) + n + PAGE - 1) // PAGE
    table = torch.arange(B * pages, dtype=torch.int32).reshape(B, pages).cuda()
    cache = [torch.zeros((B * pages, Hkv, PAGE, d), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    assert torch.equal(vsd.vsd_norm_rope_append_kv(*gpu, *cache, table, int32(base), turns, **how), q)
    for b in range(B):
        at = slice(base[b], base[b] + valid[b])
        for c, x in zip(cache, (k, gpu[2])):
            rows = c[b * pages:(b + 1) * pages].transpose(1, 2).reshape(pages * PAGE, Hkv, d)
            assert torch.equal(rows[at], x[b, :valid[b]])
            rows = rows.clone()
            rows[at] = 0
            assert torch.all(rows == 0)
    codes = [torch.zeros_like(c).to(torch.float8_e4m3fn) for c in cache]
    scales = [torch.zeros((B * pages, Hkv), device="cuda") for _ in range(2)]
    assert torch.equal(vsd.vsd_norm_rope_append_kv_quant(*gpu, *codes, *scales, table, int32(base), turns, **how), q)
    for b in range(B):
        rows = codes[0][b * pages:(b + 1) * pages].float() * scales[0][b * pages:(b + 1) * pages, :, None, None]
        rows = rows.transpose(1, 2).reshape(pages * PAGE, Hkv, d)[base[b]:base[b] + valid[b]]
        have, want = rows, k[b, :valid[b]].float()
        # half a step of e4m3 and one of bf16; below its normals 2^-10 of the page's scale, the largest of the page's
        # values (at most the largest of all) over 448 and less than twice that
        top = float(want.abs().max()) if valid[b] else 0.0
        assert torch.all((have - want).abs() <= (2.0 ** -4 + 2.0 ** -7) * want.abs() + 2.0 ** -9 * top / 224)
    assert vsd.vsd_read_device_status() == 0
