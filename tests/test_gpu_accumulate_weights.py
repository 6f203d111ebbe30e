"""Attention weight accumulated from collected logits, against the definition in 64 bits."""
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


def int32(x):
    return torch.as_tensor(x, dtype=torch.int32).cuda()


class Case:
    """Random logits over prefixes of these lengths; the cache holds the verify block's keys (and
    NaN everywhere else)."""

    def __init__(self, prefix, P_max, R, C, G, Hkv, d, quant, seed, spread=1.0, stride=None):
        g = torch.Generator().manual_seed(seed)
        B, self.prefix, self.G, self.R, self.C = len(prefix), list(prefix), G, R, C
        self.scale = 1 / math.sqrt(d)
        self.logits = spread * torch.randn((B, C, Hkv * G, P_max), generator=g)
        self.q = torch.randn((B, R, Hkv * G, d), generator=g).to(torch.bfloat16)
        stride = P_max if stride is None else stride
        self.weights = torch.rand((B, Hkv, stride), generator=g)
        self.table, spare = life.tables([p + R for p in prefix], g)
        NB = int(torch.cat([self.table.flatten(), spare.int()]).max()) + 1
        if quant:
            self.codes = torch.full((NB, Hkv, PAGE, d), ref.NAN_CODE, dtype=torch.uint8)
            self.scales = 2.0 ** torch.randint(-8, -4, (NB, Hkv), generator=g).float() * 1.25
        self.keys = torch.full((NB, Hkv, PAGE, d), math.nan, dtype=torch.bfloat16)
        for b, p in enumerate(prefix):
            for u in range(R):
                blk = int(self.table[b, (p + u) // PAGE])
                k = torch.randn((Hkv, d), generator=g, dtype=torch.float64)
                self.keys[blk, :, (p + u) % PAGE] = k.to(torch.bfloat16)
                if quant:
                    self.codes[blk, :, (p + u) % PAGE] = ref.encode((k / self.scales[blk].double()[:, None]).clamp(-448, 448))
        self.quant = quant

    def key(self, b, j):
        blk = self.table[b].long()[j // PAGE]
        if self.quant:
            return ref.decode(self.codes[blk, :, j % PAGE]) * self.scales[blk].double()[:, :, None]
        return self.keys[blk, :, j % PAGE].double()

    def block_logits(self, rows, seen=None):
        """[b][c]: the logits of row c against the verify block, [Hq, r + 1]."""
        out = []
        for b, p in enumerate(self.prefix):
            k = self.key(b, p + torch.arange(self.R))                                   # [R, Hkv, d]
            out.append([None if r < 0 else self.scale * torch.einsum(
                "hd,uhd->hu", self.q[b, r].double(), k[:r + 1].repeat_interleave(self.G, 1)) for r in rows])
        return out

    def call(self, vsd, rows=None, logits=None, weights=None, prefix=None, table=None, stream=None):
        w = self.weights.cuda() if weights is None else weights
        lg = self.logits.cuda() if logits is None else logits
        pl = int32(self.prefix) if prefix is None else prefix
        bt = self.table.cuda() if table is None else table
        more = dict(scale=self.scale, rows=rows, stream=stream)
        if self.quant:
            got = vsd.vsd_accumulate_weights_quant(lg, self.q.cuda(), self.codes.cuda().view(torch.float8_e4m3fn),
                                                   self.scales.cuda(), bt, pl, w, **more)
        else:
            got = vsd.vsd_accumulate_weights(lg, self.q.cuda(), self.keys.cuda(), bt, pl, w, **more)
        assert got is w
        return w

    def check(self, got, rows, prefix=None):
        want, bound = life.accumulated(self.weights.double(), self.logits, self.block_logits(rows), rows,
                                       self.prefix if prefix is None else prefix, self.G)
        got = got.cpu()
        assert torch.all((got.double() - want).abs() <= bound)
        for b, P in enumerate(self.prefix):
            assert torch.equal(got[b, :, P:], self.weights[b, :, P:])                    # bit for bit


LENGTHS = [  # prefix lengths, P_max, stride
    ([1], 1, 1), ([0, 1, 2, 3], 5, 7), ([31, 32, 33, 16], 33, 40), ([512], 512, 512), ([2047, 2048, 0], 2048, 2052),
    ([2049, 17], 2049, 2049), ([4096, 4095], 4096, 4096), ([5000, 1, 4999], 5003, 5003), ([16500, 32769], 32772, 32772),
]


@pytest.mark.parametrize("quant", [False, True])
@pytest.mark.parametrize("prefix,P_max,stride", LENGTHS)
def test_lengths(vsd, prefix, P_max, stride, quant):
    c = Case(prefix, P_max, R=4, C=2, G=2, Hkv=2, d=64, quant=quant, seed=P_max, stride=stride, spread=2.0)
    c.check(c.call(vsd), (0, 3))
    assert vsd.vsd_read_device_status() == 0


@pytest.mark.parametrize("R,C,G,Hkv,d", [
    (1, 1, 1, 1, 64), (1, 2, 4, 2, 128), (2, 2, 4, 2, 128), (5, 2, 8, 2, 128), (6, 2, 1, 3, 64), (3, 3, 4, 2, 128),
    (16, 2, 4, 1, 128), (16, 16, 4, 1, 64), (6, 6, 8, 2, 128), (4, 4, 16, 1, 64), (12, 12, 1, 2, 128), (3, 2, 16, 1, 64),
])
@pytest.mark.parametrize("quant", [False, True])
def test_rows_and_heads(vsd, R, C, G, Hkv, d, quant):
    """Every count of columns' groups: held in registers (up to 8, up to 16) and read again."""
    rows = tuple(range(R)) if C == R else (0, R - 1) if R > 1 else (0, -1)
    c = Case([1500, 77, 0], 1500, R, C, G, Hkv, d, quant, seed=R * 100 + G)
    c.check(c.call(vsd), rows)
    assert vsd.vsd_read_device_status() == 0


@pytest.mark.parametrize("P_max,prefix", [(40000, [39999, 123]), (70001, [70001])])
def test_long_slices(vsd, P_max, prefix):
    """Slices of several steps, which are read again."""
    c = Case(prefix, P_max, R=3, C=2, G=4, Hkv=1, d=64, quant=False, seed=9)
    c.check(c.call(vsd), (0, 2))
    c = Case(prefix, P_max, R=2, C=2, G=16, Hkv=1, d=64, quant=True, seed=9)
    c.check(c.call(vsd), (0, 1))


@pytest.mark.parametrize("P_max,stride", [(32, 35), (700, 701), (40000, 40001)])
def test_strides_and_addresses_that_vectors_do_not_fit(vsd, P_max, stride):
    """Row strides or bases off 16 bytes: values one by one, the same sums."""
    c = Case([P_max - 1, 5], P_max, R=2, C=2, G=2, Hkv=2, d=64, quant=False, seed=2, stride=stride)
    c.check(c.call(vsd), (0, 1))
    c = Case([P_max - 1, 5], P_max, R=2, C=2, G=2, Hkv=2, d=64, quant=False, seed=2, stride=P_max)
    c.check(c.call(vsd), (0, 1))
    for off in (1, 2, 3):
        lg = torch.empty(c.logits.numel() + 4, device="cuda")[off:off + c.logits.numel()].view(c.logits.shape).copy_(c.logits)
        w = torch.empty(c.weights.numel() + 4, device="cuda")[off:off + c.weights.numel()].view(c.weights.shape).copy_(c.weights)
        c.check(c.call(vsd, logits=lg), (0, 1))
        c.check(c.call(vsd, weights=w), (0, 1))


def test_chosen_rows(vsd):
    c = Case([300, 40], 300, R=5, C=2, G=4, Hkv=2, d=64, quant=False, seed=3)
    for rows in ((0, 4), (3, 1), (-1, 2), (4, -1), (2, 2)):
        c.check(c.call(vsd, rows=rows), rows)
    assert torch.equal(c.call(vsd, rows=(-1, -1)).cpu(), c.weights)
    c.check(c.call(vsd, rows=[0, 4]), (0, 4))
    for bad in ((0,), (0, 5), (0, -2), (0, 1, 2)):
        with pytest.raises(ValueError):
            c.call(vsd, rows=bad)
    with pytest.raises(ValueError):
        c.call(vsd, logits=torch.zeros((2, 3, 8, 300), device="cuda"))                   # which rows?
    with pytest.raises(TypeError):
        c.call(vsd, rows=("a", 1))


def test_weights_of_a_row_add_up(vsd):
    """With the verify block's share left out, the added weights of a row and group sum to at
    most its heads; without a block key in sight (one far below), to all of it."""
    c = Case([1000], 1000, R=1, C=1, G=4, Hkv=2, d=64, quant=False, seed=4)
    c.weights.zero_()
    c.logits += 40.0                                          # the block's key: e^-40 beside the prefix
    got = c.call(vsd).cpu().double().sum(-1)
    assert torch.all((got - 4).abs() <= 4 * 2.0 ** -18)


def test_large_and_far_logits(vsd):
    """Spreads beyond fp32's exponentials, equal logits, logits of the type's lowest value."""
    c = Case([3000, 900], 3000, R=2, C=2, G=2, Hkv=1, d=64, quant=False, seed=5, spread=60.0)
    c.logits[0, 0, 0] = 3e4                                    # all equal, far from zero
    c.logits[0, 1, 1, :2999] = -3.4028234663852886e38
    c.logits[1, 0, 0] -= 1e6
    c.logits[1, 1, 1, 100:] = -math.inf
    c.check(c.call(vsd), (0, 1))


@pytest.mark.parametrize("P_max", [700, 5000, 40000])
def test_logits_that_are_not_finite(vsd, P_max):
    """A NaN or an infinity makes its row's weights NaN, and only those; all minus infinity beside
    a block key: nothing is added."""
    c = Case([P_max - 1], P_max, R=2, C=2, G=1, Hkv=4, d=64, quant=False, seed=6)
    c.logits[0, 0, 0, P_max // 3] = math.nan
    c.logits[0, 1, 1, P_max - 2] = math.inf
    c.logits[0, :, 2] = -math.inf
    c.logits[0, :, 3, P_max - 1] = math.nan                   # behind the prefix: not read
    got = c.call(vsd).cpu()[0, :, :P_max - 1]
    assert torch.all(torch.isnan(got[:2]))
    assert torch.equal(got[2], c.weights[0, 2, :P_max - 1])
    assert torch.all(torch.isfinite(got[3]))


@pytest.mark.parametrize("P_max", [700, 40000])
def test_the_largest_logits(vsd, P_max):
    """Up to 2^127 in magnitude a logit is one like others; beyond, it counts as infinite."""
    c = Case([P_max], P_max, R=1, C=1, G=1, Hkv=4, d=64, quant=False, seed=6)
    c.logits[0, 0, 0, 7] = 2.0 ** 127
    c.logits[0, 0, 1, :] = -(2.0 ** 127)
    c.logits[0, 0, 2, :] = -3.4028234663852886e38
    c.logits[0, 0, 3, 7] = 3.4028234663852886e38
    got = c.call(vsd).cpu()[0] - c.weights[0]
    assert abs(float(got[0, 7]) - 1) <= 2.0 ** -20 and float(got[0].sum()) <= 1 + 2.0 ** -18
    assert torch.all(got[1:3] == 0)          # the block's own key has it all
    assert torch.all(torch.isnan(got[3]))


@pytest.mark.parametrize("P_max", [700, 40000])
def test_every_value_nan(vsd, P_max):
    c = Case([P_max], P_max, R=1, C=1, G=1, Hkv=1, d=64, quant=False, seed=6)
    c.logits.fill_(math.nan)
    assert torch.all(torch.isnan(c.call(vsd)))


def test_bad_lengths_and_blocks(vsd):
    c = Case([100, 200, 300, 50], 300, R=4, C=2, G=2, Hkv=2, d=64, quant=False, seed=7)
    got = c.call(vsd, prefix=int32([100, -1, 301, 50]))
    assert vsd.vsd_read_device_status() == vsd.DEV_BAD_LENGTH
    c.check(torch.stack([got[0].cpu(), *c.weights[1:3], got[3].cpu()]), (0, 3), prefix=[100, 0, 0, 50])
    assert torch.equal(got[1:3].cpu(), c.weights[1:3])
    # a table too short for the verify block: 300 + 4 rows in 19 pages
    got = c.call(vsd, table=c.table[:, :18].contiguous().cuda())
    assert vsd.vsd_read_device_status() == vsd.DEV_BAD_LENGTH
    assert torch.equal(got[2].cpu(), c.weights[2]) and not torch.equal(got[1].cpu(), c.weights[1])
    # the verify block's page outside the cache: its keys are left out
    table = c.table.clone()
    table[0, 6] = -1                                          # positions 96 .. 111
    got = c.call(vsd, table=table.cuda()).cpu()
    assert vsd.vsd_read_device_status() == vsd.DEV_BAD_BLOCK
    none = torch.full((4, 1), -math.inf, dtype=torch.float64)
    blocks = c.block_logits((0, 3))
    blocks[0] = [none, none]
    want, bound = life.accumulated(c.weights.double(), c.logits, blocks, (0, 3), c.prefix, 2)
    assert torch.all((got.double() - want).abs() <= bound)


def test_repeated_and_captured(vsd):
    """Bit-identical runs; a captured call replays on what its buffers hold then, beside another
    stream's."""
    c = Case([9000, 500], 9000, R=3, C=2, G=4, Hkv=2, d=128, quant=True, seed=8)
    a, b = c.call(vsd), c.call(vsd)
    assert torch.equal(a, b)
    w, lg, pl, bt = c.weights.cuda(), c.logits.cuda(), int32(c.prefix), c.table.cuda()
    q, kc, ks = c.q.cuda(), c.codes.cuda().view(torch.float8_e4m3fn), c.scales.cuda()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        vsd.vsd_accumulate_weights_quant(lg, q, kc, ks, bt, pl, w, scale=c.scale)
    w.copy_(c.weights)
    graph.replay()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = c.call(vsd, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(w, a) and torch.equal(other, a)
    pl.copy_(int32([20, 0]))
    w.copy_(c.weights)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(w[1].cpu(), c.weights[1]) and torch.equal(w[0, :, 20:].cpu(), c.weights[0, :, 20:])


def test_after_a_verification(vsd):
    """On the logits that a verification of the same cache collected: the weights are those of
    its attention."""
    B, R, G, Hkv, d, P = 2, 4, 4, 2, 64, 700
    g = torch.Generator().manual_seed(12)
    prefix = [P, 333]
    table, spare = life.tables([p + R for p in prefix], g)
    NB = int(table.max()) + 1
    kc, vc = (torch.randn((NB, Hkv, PAGE, d), generator=g).to(torch.bfloat16) for _ in range(2))
    q = torch.randn((B, R, Hkv * G, d), generator=g).to(torch.bfloat16)
    args = (q.cuda(), kc.cuda(), vc.cuda(), table.cuda(), int32(prefix))
    for every in (False, True):
        call = vsd.vsd_verify_attn_collect_all if every else vsd.vsd_verify_attn_collect
        _, logits, _ = call(*args, P_max=P, scale=d ** -0.5)
        w = torch.zeros((B, Hkv, P), device="cuda")
        vsd.vsd_accumulate_weights(logits, args[0], args[1], args[3], args[4], w, scale=d ** -0.5)
        rows = range(R) if every else (0, R - 1)
        for b, p in enumerate(prefix):
            j = torch.arange(p + R)
            k = kc[table[b].long()[j // PAGE], :, j % PAGE].double().repeat_interleave(G, 1)
            want = torch.zeros((Hkv, p), dtype=torch.float64)
            for r in rows:
                z = torch.einsum("hd,jhd->hj", q[b, r].double(), k[:p + r + 1]) * d ** -0.5
                want += torch.softmax(z, 1)[:, :p].view(Hkv, G, p).sum(1)
            # the logits' own error (their products in fp32: below 2^-13 of order-one logits)
            assert torch.all((w[b, :, :p].cpu().double() - want).abs() <= 2.0 ** -11 * want)


def test_mismatched_tensors(vsd):
    c = Case([30], 32, R=2, C=2, G=2, Hkv=2, d=64, quant=False, seed=1)
    lg, q, kc, bt, pl, w = c.logits.cuda(), c.q.cuda(), c.keys.cuda(), c.table.cuda(), int32([30]), c.weights.cuda()

    def call(lg=lg, q=q, kc=kc, bt=bt, pl=pl, w=w):
        vsd.vsd_accumulate_weights(lg, q, kc, bt, pl, w, scale=1.0)
    call()
    for kw in (dict(lg=lg[:, :, :2]), dict(lg=lg.transpose(2, 3)), dict(w=w[..., :31].contiguous()), dict(w=w[:, :1].contiguous()),
               dict(pl=int32([30, 1])), dict(bt=bt.repeat(2, 1)), dict(q=q[..., :32].contiguous()), dict(w=w.cpu()),
               dict(w=torch.zeros((1, 2, 64), device="cuda")[..., ::2])):
        with pytest.raises(ValueError):
            call(**kw)
    for kw in (dict(lg=lg.double()), dict(w=w.half()), dict(pl=pl.long()), dict(kc=kc.float())):
        with pytest.raises(TypeError):
            call(**kw)
