"""The 8-bit cache's calls on the GPU against their definition in 64 bits."""
import math

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


def codes_of(t):
    return t.view(torch.uint8).cpu()


def same_codes(got, want):
    """Equal codes, any NaN code for a NaN, any sign of zero kept as it is."""
    nan = (want & 0x7F) == 0x7F
    assert torch.equal((got & 0x7F) == 0x7F, nan)
    assert torch.equal(got[~nan], want[~nan])


# ------------------------------------------------------------------ storing
def _check_append(vsd, cache, rows, pos, valid, n, pos_offset=0, pass_valid=True):
    kc, vc, ks, vs, bt = cache.cuda()
    want = [(c.clone(), s.clone()) for c, s in zip(cache.codes, cache.scales)]
    for (c, s), x in zip(want, rows):
        ref.append(c, s, x.double(), cache.table, pos, valid)
    base = torch.tensor([p - pos_offset for p in pos], dtype=torch.int32, device="cuda")
    nv = torch.tensor(valid, dtype=torch.int32, device="cuda") if pass_valid else None
    vsd.vsd_append_kv_quant(rows[0].cuda(), rows[1].cuda(), kc, vc, ks, vs, bt, base,
                            pos_offset=pos_offset, n_valid=nv)
    assert vsd.vsd_read_device_status() == 0
    for (c, s), gc, gs in zip(want, (kc, vc), (ks, vs)):
        same_codes(codes_of(gc), c)
        assert torch.equal(torch.nan_to_num(gs.cpu(), nan=-1.0), torch.nan_to_num(s, nan=-1.0))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hkv", [1, 3, 8])
@pytest.mark.parametrize("pos,valid,n", [
    ([0], [1], 1), ([0], [16], 16), ([0, 5], [40, 40], 40), ([15, 16, 17], [1, 1, 1], 1),
    ([0, 7, 31, 33, 64], [0, 3, 37, 1, 20], 37), ([250], [6], 6), ([3], [300], 300),
])
def test_append_stores_the_definitions_codes(vsd, d, Hkv, pos, valid, n):
    caps = [p + n + 5 for p in pos]
    cache = ref.Cache(caps, Hkv, d, seed=n * 7 + d)
    g = torch.Generator().manual_seed(5)
    rows = [(torch.randn((len(pos), n, Hkv, d), generator=g) *
             torch.exp(2 * torch.randn((len(pos), n, 1, 1), generator=g))).bfloat16() for _ in range(2)]
    _check_append(vsd, cache, rows, pos, valid, n)


def test_append_over_scales_that_are_no_powers_of_two(vsd):
    cache = ref.Cache([100, 100], 2, 128, seed=3, power_of_two=False)
    g = torch.Generator().manual_seed(6)
    for mag in (0.01, 1.0, 30.0):
        rows = [(torch.randn((2, 5, 2, 128), generator=g) * mag).bfloat16() for _ in range(2)]
        _check_append(vsd, cache, rows, [50, 61], [5, 5], 5, pos_offset=-1, pass_valid=False)


@pytest.mark.parametrize("scale", [2.0 ** 127, 1.37, 2.0 ** -126, 2.0 ** -130])
def test_append_keeps_a_callers_scale(vsd, scale):
    """Scales at the ends of the range and between powers of two, rows that they hold (some
    values below the smallest code), NaN and infinities among them."""
    cache = ref.Cache([40], 3, 128, seed=13)
    blk = int(cache.table[0, 1])
    for kv in range(2):
        cache.scales[kv][blk] = scale
    g = torch.Generator().manual_seed(8)
    rows = [(torch.randn((1, 7, 3, 128), generator=g) * 50.0 * min(scale, 2.0 ** 118)).bfloat16() for _ in range(2)]
    for x in rows:
        x[0, 1, 0, 5], x[0, 2, 1, 127], x[0, 6, 2, 0] = math.nan, math.inf, -math.inf
    _check_append(vsd, cache, rows, [21], [7], 7)


@pytest.mark.parametrize("mag", [0.0, 0.3])
def test_append_into_a_page_of_scale_zero(vsd, mag):
    """Earlier rows with scale 0 (a caller's own page of zeros): a scale of 0 cannot hold
    the new rows, zeros among them; the earlier rows stay zeros."""
    cache = ref.Cache([40, 40], 2, 64, seed=12)
    for b in range(2):
        blk = int(cache.table[b, 1])
        cache.scales[0][blk] = 0.0
        cache.scales[1][blk] = 0.0
    g = torch.Generator().manual_seed(7)
    rows = [(torch.randn((2, 3, 2, 64), generator=g) * mag).bfloat16() for _ in range(2)]
    _check_append(vsd, cache, rows, [20, 31], [3, 1], 3)


def test_append_extreme_values(vsd):
    """Zero rows, subnormal and largest bf16 values, values at the border of a scale,
    NaN and infinities (which do not set the scale)."""
    d = 64
    cache = ref.Cache([64], 1, d, seed=4)
    vals = torch.tensor([0.0, -0.0, 2.0 ** -133, 3.38e38, -3.38e38, 448.0, 450.0, -449.0, 1.75, 1.7578125,
                         math.nan, math.inf, -math.inf, 2.0 ** -126, 1e-30, -7.0]).bfloat16()
    for i in range(len(vals)):
        for j in (0, 5, 10, 11):
            row = torch.zeros((1, 2, 1, d)).bfloat16()
            row[0, 0, 0, 3] = vals[i]
            row[0, 1, 0, 60] = vals[j]
            for pos in (16, 20):
                _check_append(vsd, cache, [row, -row], [pos], [2], 2)


def test_append_token_by_token_equals_its_definition(vsd):
    """One token at a time over three pages, the loudness rising and falling: every step
    matches the definition's cache after the same steps."""
    Hkv, d = 2, 128
    cache = ref.Cache([60], Hkv, d, seed=9)
    kc, vc, ks, vs, bt = cache.cuda()
    g = torch.Generator().manual_seed(8)
    for p in range(10, 50):
        rows = [(torch.randn((1, 1, Hkv, d), generator=g) * 2.0 ** ((p * 7) % 11 - 4)).bfloat16() for _ in range(2)]
        for c, s, x in zip(cache.codes, cache.scales, rows):
            ref.append(c, s, x.double(), cache.table, [p], [1])
        vsd.vsd_append_kv_quant(rows[0].cuda(), rows[1].cuda(), kc, vc, ks, vs, bt,
                                torch.tensor([p], dtype=torch.int32, device="cuda"))
    assert vsd.vsd_read_device_status() == 0
    for c, s, gc, gs in zip(cache.codes, cache.scales, (kc, vc), (ks, vs)):
        same_codes(codes_of(gc), c)
        assert torch.equal(torch.nan_to_num(gs.cpu(), nan=-1.0), torch.nan_to_num(s, nan=-1.0))


def test_append_flags_and_skips_what_does_not_fit(vsd):
    cache = ref.Cache([40, 40, 40, 40], 2, 64, seed=2)
    cache.table[3, 1] = 9999
    kc, vc, ks, vs, bt = cache.cuda()
    rows = torch.ones((4, 8, 2, 64)).bfloat16().cuda()
    width = cache.table.shape[1] * 16
    before = codes_of(kc).clone()

    def call(base, valid):
        vsd.vsd_append_kv_quant(rows, rows, kc, vc, ks, vs, bt,
                                torch.tensor(base, dtype=torch.int32, device="cuda"),
                                n_valid=torch.tensor(valid, dtype=torch.int32, device="cuda"))
        return vsd.vsd_read_device_status()
    assert call([-1, width - 7, 0, 0], [8, 8, 0, 0]) == vsd.DEV_BAD_LENGTH
    assert call([0, 0, 0, 0], [9, -1, 0, 0]) == vsd.DEV_BAD_LENGTH
    assert torch.equal(codes_of(kc), before)
    assert call([0, 0, 0, 16], [0, 0, 0, 8]) == vsd.DEV_BAD_BLOCK
    assert torch.equal(codes_of(kc), before)


# ------------------------------------------------------------------ reading
@pytest.mark.parametrize("d,Hkv,pos,valid,n", [
    (64, 1, [0], [1], 1), (128, 8, [3, 40], [50, 11], 50), (64, 3, [16, 0, 31], [0, 17, 200], 200),
])
def test_read_returns_code_times_scale(vsd, d, Hkv, pos, valid, n):
    cache = ref.Cache([p + n for p in pos], Hkv, d, seed=n, power_of_two=False)
    args = cache.cuda()
    base = torch.tensor(pos, dtype=torch.int32, device="cuda")
    nv = torch.tensor(valid, dtype=torch.int32, device="cuda")
    k_out = torch.full((len(pos), n, Hkv, d), 7.0, dtype=torch.bfloat16, device="cuda")
    got = vsd.vsd_read_kv_quant(*args, base, n=n, n_valid=nv, k_out=k_out)
    assert got[0] is k_out and vsd.vsd_read_device_status() == 0
    for kv in range(2):
        want = torch.full((len(pos), n, Hkv, d), 7.0 if kv == 0 else 0.0, dtype=torch.bfloat16)
        for b in range(len(pos)):
            j = pos[b] + torch.arange(valid[b])
            # code (4 bits) * scale (24 bits): below 2^28 apart, one rounding to fp32 and
            # one to bf16; the kernel's two roundings are these two
            want[b, :valid[b]] = cache.kv(b, j)[kv].float().bfloat16()
        assert torch.equal(got[kv].cpu(), want)


def test_read_skips_bad_blocks_and_ranges(vsd):
    cache = ref.Cache([40, 40], 2, 64, seed=2)
    cache.table[0, 1] = -1
    args = cache.cuda()
    out = torch.full((2, 20, 2, 64), 3.0, dtype=torch.bfloat16, device="cuda")
    vsd.vsd_read_kv_quant(*args, torch.tensor([10, 1000], dtype=torch.int32, device="cuda"), n=20,
                          k_out=out, v_out=out.clone())
    assert vsd.vsd_read_device_status() == vsd.DEV_BAD_BLOCK | vsd.DEV_BAD_LENGTH
    assert torch.all(out[0, 6:] == 3.0) and torch.all(out[1] == 3.0)
    assert torch.equal(out[0, :6].cpu(), cache.kv(0, 10 + torch.arange(6))[0].float().bfloat16())


# ------------------------------------------------------------------ verification
def check_verify(vsd, cache, prefix, Hq, d, R, P_max, rows=None, q=None, scale=None, **kw):
    B, Hkv = len(prefix), cache.codes[0].shape[1]
    G = Hq // Hkv
    row0, row1 = rows or (0, R - 1)
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    if q is None:
        q = torch.randn((B, R, Hq, d), generator=cache.gen).bfloat16()
    logits = torch.full((B, 2, Hq, P_max), 5.0, device="cuda")
    partial = torch.full((B, Hkv, P_max), 5.0, device="cuda")
    out, lg, ps = vsd.vsd_verify_attn_collect_quant(
        q.cuda(), *cache.cuda(), torch.tensor(prefix, dtype=torch.int32, device="cuda"), P_max=P_max,
        scale=scale, row0=row0, row1=row1, logits=logits, partial=partial, **kw)
    assert vsd.vsd_read_device_status() == 0
    out, lg, ps = out.cpu().double(), lg.cpu().double(), ps.cpu().double()
    q = q.double()
    for b in range(B):
        P = prefix[b]
        assert torch.all(lg[b, :, :, P:] == 5.0) and torch.all(ps[b, :, P:] == 5.0)
        k, v = cache.kv(b, torch.arange(P + R))
        for h in range(Hq):
            g = h // G
            for t in range(R):
                z = scale * (k[:, g] @ q[b, t, h])
                want, mag = ref.softmax_av(z[:P + t + 1], v[:P + t + 1, g])
                err = (out[b, t, h] - want).abs()
                assert torch.all(err <= ref.out_bound(want, mag)), (b, t, h, float(err.max()))
            for c, t in ((0, row0), (1, row1)):
                z = scale * (k[:P, g] @ q[b, t, h])
                err = (lg[b, c, h, :P] - z).abs()
                assert torch.all(err <= ref.logit_bound(q[b, t, h], k[:P, g], scale)), (b, c, h)
        for g in range(Hkv):
            want = torch.zeros(P, dtype=torch.float64)
            bound = torch.zeros(P, dtype=torch.float64)
            for t in (row0, row1):
                for h in range(g * G, (g + 1) * G):
                    z = scale * (k[:P, g] @ q[b, t, h])
                    want += z
                    # the term's own error, and 2 G roundings of sums of at most these
                    bound += ref.logit_bound(q[b, t, h], k[:P, g], scale) + 2 * G * 2.0 ** -24 * z.abs()
            assert torch.all((ps[b, g, :P] - want).abs() <= bound), (b, g)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hq,Hkv,R", [(1, 1, 1), (2, 2, 5), (4, 2, 3), (8, 2, 6), (8, 1, 6), (16, 2, 8), (16, 1, 4), (6, 3, 16), (4, 1, 16)])
def test_verify_matches_its_definition(vsd, d, Hq, Hkv, R):
    prefix = [0, 1, 127, 300, 129]
    cache = ref.Cache([p + R for p in prefix], Hkv, d, seed=d + R)
    check_verify(vsd, cache, prefix, Hq, d, R, P_max=320)


@pytest.mark.parametrize("prefix", [[0], [15], [16], [17], [111], [112], [113], [128], [1000], [4095]])
def test_verify_lengths(vsd, prefix):
    cache = ref.Cache([p + 3 for p in prefix], 2, 128, seed=prefix[0] + 1, power_of_two=False)
    check_verify(vsd, cache, prefix, 4, 128, 3, P_max=prefix[0], rows=(2, 1))


def test_verify_many_sequences_share_sms(vsd):
    g = torch.Generator().manual_seed(1)
    prefix = torch.randint(0, 400, (50,), generator=g).tolist()
    cache = ref.Cache([p + 2 for p in prefix], 4, 64, seed=17)
    check_verify(vsd, cache, prefix, 8, 64, 2, P_max=400, rows=(1, 1))


@pytest.mark.parametrize("B,P", [(1, 380), (1, 381), (1, 508), (1, 509), (19, 600), (19, 1300), (40, 1500), (76, 200)])
def test_verify_short_sequences(vsd, B, P):
    """Pairs that take one CTA each and pairs that share them, lengths from none to the longest."""
    g = torch.Generator().manual_seed(B * 7 + P)
    prefix = [P] + torch.randint(0, P + 1, (B - 1,), generator=g).tolist()
    if B > 2:
        prefix[1] = 0
    cache = ref.Cache([p + 4 for p in prefix], 2, 64, seed=B + P)
    check_verify(vsd, cache, prefix, 4, 64, 4, P_max=P)


def test_verify_more_sequences_than_a_cta_holds_lengths_of(vsd):
    g = torch.Generator().manual_seed(2)
    prefix = torch.randint(0, 150, (300,), generator=g).tolist()
    cache = ref.Cache([p + 1 for p in prefix], 1, 64, seed=18)
    check_verify(vsd, cache, prefix, 1, 64, 1, P_max=150)


def test_verify_one_long_sequence_among_short_ones(vsd):
    prefix = [3, 0, 9000, 40, 1, 700]
    cache = ref.Cache([p + 2 for p in prefix], 2, 128, seed=19)
    check_verify(vsd, cache, prefix, 4, 128, 2, P_max=9100)


def test_verify_peaked_rows_and_rising_maxima(vsd):
    """Logits up to a few hundred whose maximum keeps rising along the sequence, and pages
    whose value scales differ by 2^12: running maxima and value references move."""
    d, R, P = 128, 2, 700
    cache = ref.Cache([P + R], 1, d, seed=5)
    for lp in range(cache.table.shape[1]):
        blk = int(cache.table[0, lp])
        if blk >= 0:
            cache.scales[0][blk] = 2.0 ** (-9 + lp / 9)
            cache.scales[1][blk] = 2.0 ** (-9 + (lp * 5) % 13)
    check_verify(vsd, cache, [P], 2, d, R, P_max=P)


def test_verify_one_loud_key_over_many_quiet_ones(vsd):
    """Half of the probability on one key, the rest spread over thousands of equal keys:
    probabilities far below the largest one still count."""
    d, P = 64, 8000
    cache = ref.Cache([P + 1], 1, d, seed=6)
    one = ref.encode(torch.tensor([1.0], dtype=torch.float64))[0]
    for lp in range(-(-(P + 1) // 16)):
        blk = int(cache.table[0, lp])
        n = min(16, P + 1 - lp * 16)
        cache.codes[0][blk, :, :n] = 0
        cache.scales[0][blk] = 1.0
        cache.scales[1][blk] = 1.0
        cache.codes[1][blk, :, :n] = one
    loud = 4321
    blk = int(cache.table[0, loud // 16])
    cache.codes[0][blk, 0, loud % 16, 0] = one
    cache.codes[1][blk, 0, loud % 16] = one | 0x80
    for z in (math.log(8000.0), 1.0, 15.0):
        q = torch.zeros((1, 1, 1, d)).bfloat16()
        q[..., 0] = z
        check_verify(vsd, cache, [P], 1, d, 1, P_max=P, q=q, scale=1.0)


def test_verify_zero_values_with_tiny_scales_before_ordinary_ones(vsd):
    """3.2 million keys whose values are zeros with the smallest scale that storing rows
    writes, their logits 9 above the first ones', then a thousand ordinary keys: the sums
    of the former's probabilities stay finite in every part of the sequence."""
    d, P, tail = 64, 3200000, 1000
    one = ref.encode(torch.tensor([1.0], dtype=torch.float64))[0]
    codes = torch.zeros((2, 3, 1, 16, d), dtype=torch.uint8)  # K and V of three pages
    codes[0, 1:, 0, :, 0] = one
    codes[1, 2] = one
    scales = torch.tensor([[1.0, 1.0, 1.0], [2.0 ** -126, 2.0 ** -126, 1.0]])[..., None].contiguous()
    table = torch.ones((1, P // 16 + 1), dtype=torch.int32)
    table[0, :8] = 0
    table[0, (P - tail) // 16:] = 2
    n = P + 1 - (P - tail) // 16 * 16  # keys of the last page
    q = torch.zeros((1, 1, 1, d)).bfloat16()
    q[..., 0] = 9.0
    kc, vc = (codes[i].cuda().view(torch.float8_e4m3fn) for i in range(2))
    out = vsd.vsd_verify_attn_collect_quant(
        q.cuda(), kc, vc, scales[0].cuda(), scales[1].cuda(), table.cuda(),
        torch.tensor([P], dtype=torch.int32, device="cuda"), P_max=P, scale=1.0, collect=False)[0]
    assert vsd.vsd_read_device_status() == 0
    want = torch.tensor(n / (P + 1 - 128 + 128 * math.exp(-9.0)), dtype=torch.float64)
    assert torch.all((out.cpu().double() - want).abs() <= ref.out_bound(want, want))


def test_verify_query_ranges(vsd):
    """Queries whose dimensions differ by 2^14, zero queries and the largest bf16 values'
    binade: the two parts a query is split into hold it."""
    d, R, P = 128, 3, 150
    cache = ref.Cache([P + R], 2, d, seed=11)
    q = torch.randn((1, R, 4, d), generator=cache.gen)
    q[0, 0, 0] *= torch.exp2(-torch.arange(d) / 9.0)
    q[0, 0, 1] = 0.0
    q[0, 1, 2] *= 2.0 ** 100
    q[0, 1, 3] *= 2.0 ** -120
    check_verify(vsd, cache, [P], 4, d, R, P_max=P, q=q.bfloat16())


def test_verify_without_collection_and_outputs_given(vsd):
    cache = ref.Cache([70], 2, 64, seed=12)
    q = torch.randn((1, 1, 4, 64), generator=cache.gen).bfloat16().cuda()
    pl = torch.tensor([69], dtype=torch.int32, device="cuda")
    a, lg, ps = vsd.vsd_verify_attn_collect_quant(q, *cache.cuda(), pl, P_max=69, scale=0.1, collect=False)
    assert lg is None and ps is None
    out = torch.empty_like(a)
    b = vsd.vsd_verify_attn_collect_quant(q, *cache.cuda(), pl, P_max=69, scale=0.1, out=out)[0]
    assert b is out and torch.equal(a, b)


def test_verify_flags_bad_blocks_and_lengths(vsd):
    d, R = 64, 2
    cache = ref.Cache([100, 60, 50], 2, d, seed=13)
    good = [c.clone() for c in cache.codes]
    cache.table[0, 2] = 10 ** 6     # keys 32 .. 47 of sequence 0 drop out
    q = torch.randn((3, R, 4, d), generator=cache.gen).bfloat16()
    prefix = [98, 500, 48]
    out = vsd.vsd_verify_attn_collect_quant(
        q.cuda(), *cache.cuda(), torch.tensor(prefix, dtype=torch.int32, device="cuda"), P_max=100, scale=0.125)[0]
    assert vsd.vsd_read_device_status() == vsd.DEV_BAD_BLOCK | vsd.DEV_BAD_LENGTH
    out = out.cpu().double()
    assert torch.all(out[1] == 0)
    for b in (0, 2):
        for t in range(R):
            j = torch.tensor([x for x in range(prefix[b] + t + 1) if b != 0 or not 32 <= x < 48])
            k, v = cache.kv(b, j)
            for h in range(4):
                want, mag = ref.softmax_av(0.125 * (k[:, h // 2] @ q[b, t, h].double()), v[:, h // 2])
                assert torch.all((out[b, t, h] - want).abs() <= ref.out_bound(want, mag))
    assert all(torch.equal(a, b) for a, b in zip(good, cache.codes))


def test_verify_nan_of_a_visible_key_reaches_only_its_rows(vsd):
    """A NaN code in a key of the verify block: rows before it do not see it."""
    d, R, P = 64, 3, 20
    cache = ref.Cache([P + R], 1, d, seed=14)
    blk = int(cache.table[0, (P + 2) // 16])
    cache.codes[0][blk, 0, (P + 2) % 16, 5] = ref.NAN_CODE
    q = torch.randn((1, R, 2, d), generator=cache.gen).bfloat16().cuda()
    out = vsd.vsd_verify_attn_collect_quant(q, *cache.cuda(), torch.tensor([P], dtype=torch.int32, device="cuda"),
                                            P_max=P, scale=0.125)[0]
    assert torch.all(torch.isfinite(out[:, :2])) and torch.all(torch.isnan(out[:, 2]))


# ------------------------------------------------------------------ draft step
def check_draft(vsd, cache, idx, t0, t1, Hq, d, max_tail, status=0, keep=None, k_max=None):
    B, Hkv = len(t0), cache.codes[0].shape[1]
    G = Hq // Hkv
    k_max = max([len(x) for x in idx] + [0]) if k_max is None else k_max
    it = torch.full((B, k_max), -1, dtype=torch.int32)
    for b, x in enumerate(idx):
        it[b, :len(x)] = torch.tensor(x, dtype=torch.int32)
    ns = torch.tensor([len(x) for x in idx], dtype=torch.int32)
    q = torch.randn((B, Hq, d), generator=cache.gen).bfloat16()
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    out = vsd.vsd_sparse_decode_attn_quant(
        q.cuda(), *cache.cuda(), it.cuda() if k_max else None, ns.cuda() if k_max else None, i32(t0), i32(t1),
        scale=1.0 / math.sqrt(d), max_tail=max_tail).cpu().double()
    assert vsd.vsd_read_device_status() == status
    for b in range(B):
        lst = list(idx[b]) + list(range(t0[b], t1[b]))
        j = torch.tensor([x for x in lst if keep is None or keep(b, x)], dtype=torch.int64)
        if j.numel() == 0:
            assert torch.all(out[b] == 0)
            continue
        k, v = cache.kv(b, j)
        for h in range(Hq):
            z = (k[:, h // G] @ q[b, h].double()) / math.sqrt(d)
            want, mag = ref.softmax_av(z, v[:, h // G])
            err = (out[b, h] - want).abs()
            assert torch.all(err <= ref.out_bound(want, mag)), (b, h, float(err.max()))
    return out


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (4, 2), (8, 2), (16, 2), (16, 1), (3, 3)])
def test_draft_matches_its_definition(vsd, d, Hq, Hkv):
    lens = [1, 130, 400, 17, 600]
    cache = ref.Cache([x + 6 for x in lens], Hkv, d, seed=d + Hq, power_of_two=False)
    g = torch.Generator().manual_seed(3)
    idx = [sorted(torch.randperm(x, generator=g)[:k].tolist()) for x, k in zip(lens, (0, 128, 257, 16, 100))]
    check_draft(vsd, cache, idx, lens, [x + t for x, t in zip(lens, (0, 6, 1, 0, 3))], Hq, d, max_tail=6)


@pytest.mark.parametrize("k", [0, 1, 127, 128, 129, 2000])
def test_draft_list_lengths(vsd, k):
    cache = ref.Cache([2100], 2, 128, seed=k + 1)
    g = torch.Generator().manual_seed(k)
    check_draft(vsd, cache, [sorted(torch.randperm(2090, generator=g)[:k].tolist())], [2090], [2091], 8, 128, 4,
                k_max=k + 3)


def test_draft_repeated_and_unordered_positions(vsd):
    cache = ref.Cache([300], 1, 64, seed=21)
    g = torch.Generator().manual_seed(2)
    check_draft(vsd, cache, [torch.randint(0, 290, (500,), generator=g).tolist()], [290], [300], 4, 64, 10)


def test_draft_dense_tail_only_and_empty(vsd):
    cache = ref.Cache([40, 300], 2, 64, seed=22)
    check_draft(vsd, cache, [[], []], [10, 0], [10, 300], 4, 64, 300)


def test_draft_skips_what_it_cannot_read(vsd):
    cache = ref.Cache([300, 300], 2, 64, seed=23)
    cache.table[1, 4] = -5
    check_draft(vsd, cache, [[3, -7, 250, 4000], [10, 65, 80]], [290, 290], [292, 292], 4, 64, 2,
                status=vsd.DEV_BAD_INDEX | vsd.DEV_BAD_BLOCK,
                keep=lambda b, x: 0 <= x < 292 and not (b == 1 and 64 <= x < 80))
    cache = ref.Cache([300], 2, 64, seed=24)
    check_draft(vsd, cache, [[1, 2]], [290], [299], 4, 64, 5, status=vsd.DEV_BAD_LENGTH, keep=lambda b, x: False)


# ------------------------------------------------------------------ together
def test_a_decode_run_on_the_8_bit_cache(vsd):
    """Prompt rows stored, verification, selection, draft steps that store their token
    first, verification again over the grown cache: every output against the definition on
    the definition's own cache, and the rows read back."""
    B, Hq, Hkv, d, R, k = 2, 8, 2, 64, 3, 64
    P = [150, 97]
    cache = ref.Cache([200, 200], Hkv, d, seed=31)
    kc, vc, ks, vs, bt = cache.cuda()
    g = torch.Generator().manual_seed(32)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731

    def store(pos, n, valid):
        rows = [(torch.randn((B, n, Hkv, d), generator=g) * (1 + pos[0] % 3)).bfloat16() for _ in range(2)]
        for c, s, x in zip(cache.codes, cache.scales, rows):
            ref.append(c, s, x.double(), cache.table, pos, valid)
        vsd.vsd_append_kv_quant(rows[0].cuda(), rows[1].cuda(), kc, vc, ks, vs, bt, i32(pos), n_valid=i32(valid))

    def verify():
        q = torch.randn((B, R, Hq, d), generator=g).bfloat16()
        out, _, partial = vsd.vsd_verify_attn_collect_quant(q.cuda(), kc, vc, ks, vs, bt, i32(P), P_max=200,
                                                            scale=0.125)
        for b in range(B):
            kk, vv = cache.kv(b, torch.arange(P[b] + R))
            for t in range(R):
                for h in range(Hq):
                    n = P[b] + t + 1
                    want, mag = ref.softmax_av(0.125 * (kk[:n, h // 4] @ q[b, t, h].double()), vv[:n, h // 4])
                    assert torch.all((out[b, t, h].cpu().double() - want).abs() <= ref.out_bound(want, mag))
        return partial
    store([0, 0], 150, P)
    store(P, R, [R, R])
    partial = verify()
    idx, n_sel, _ = vsd.vsd_select_topk(partial, i32(P), k=k, n_sink=4, n_recent=16)
    P = [P[0] + 2, P[1] + 1]                     # accepted counts
    for i in range(R):
        store([p + i for p in P], 1, [1, 1])
        q = torch.randn((B, Hq, d), generator=g).bfloat16()
        tail = [150, 97]
        seq = [p + i + 1 for p in P]
        out = vsd.vsd_sparse_decode_attn_quant(q.cuda(), kc, vc, ks, vs, bt, idx, n_sel, i32(tail), i32(seq),
                                               scale=0.125, max_tail=8).cpu().double()
        for b in range(B):
            j = torch.cat([idx[b, :int(n_sel[b])].cpu().long(), torch.arange(tail[b], seq[b])])
            kk, vv = cache.kv(b, j)
            for h in range(Hq):
                want, mag = ref.softmax_av(0.125 * (kk[:, h // 4] @ q[b, h].double()), vv[:, h // 4])
                assert torch.all((out[b, h] - want).abs() <= ref.out_bound(want, mag))
    store(P, R, [R, R])
    verify()
    rows = vsd.vsd_read_kv_quant(kc, vc, ks, vs, bt, i32([0, 0]), n=98)
    assert vsd.vsd_read_device_status() == 0
    for b in range(B):
        for got, want in zip(rows, cache.kv(b, torch.arange(98))):
            assert torch.equal(got[b].cpu(), want.float().bfloat16())
