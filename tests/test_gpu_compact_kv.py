"""Eviction: kept rows moved together in either cache, in place and into other pages, exactly."""
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
    def __init__(self, lengths, k, Hkv, d, quant, heads, seed, where="same", power=True, keep=None, P_max=None):
        g = torch.Generator().manual_seed(seed)
        B = len(lengths)
        self.lengths, self.k, self.Hkv, self.quant, self.heads = list(lengths), k, Hkv, quant, heads
        kept = [min(x, k) if keep is None else min(x, k, keep[b]) for b, x in enumerate(lengths)]
        pages = -(-max(1, k) // PAGE)
        # blocks of the sequences, of the other pages, and some that nothing uses
        self.table, rest = life.tables(lengths, g, spare=B * pages + 3)
        NB = sum(-(-x // PAGE) for x in lengths) + B * pages + 3
        if where == "same":
            self.dst = self.table
        elif where == "copy":
            self.dst = self.table[:, :max(pages, 1)].clone()
        else:
            self.dst = rest[:B * pages].view(B, pages).int()
            if where == "mixed":                  # every other page in place
                even = torch.arange(pages) % 2 == 0
                here = torch.zeros_like(self.dst)
                here[:, :min(pages, self.table.shape[1])] = self.table[:, :pages]
                self.dst = torch.where(even & (here >= 0) & (torch.arange(pages) < self.table.shape[1]), here, self.dst)
        Hi = Hkv if heads else 1
        self.idx = torch.full((B, Hi, k), -1, dtype=torch.int32)
        self.n = torch.zeros((B, Hi), dtype=torch.int32)
        for b in range(B):
            for h in range(Hi):
                n = kept[b]
                self.idx[b, h, :n] = torch.randperm(lengths[b], generator=g)[:n].sort().values.int()
                self.n[b, h] = n
        P_max = P_max or max(1, max(lengths))
        self.weights = torch.rand((B, Hkv, P_max), generator=g)
        if quant:
            self.caches = [ref.encode(100 * torch.randn((NB, Hkv, PAGE, d), generator=g).double().clamp(-4, 4)) for _ in range(2)]
            e = 2.0 ** torch.randint(-8, 8, (2, NB, Hkv), generator=g).float()
            e *= 1 if power else 1 + torch.rand((2, NB, Hkv), generator=g)
            self.scales = [e[0], e[1]]
            self.caches[0][0, 0, 0, 0] = ref.NAN_CODE
        else:
            bits = torch.randint(-2 ** 15, 2 ** 15, (2, NB, Hkv, PAGE, d), generator=g).to(torch.int16)
            self.caches, self.scales = [bits[0], bits[1]], []

    def lists(self):
        return (self.idx.cuda(), self.n.cuda()) if self.heads else (self.idx[:, 0].contiguous().cuda(), self.n[:, 0].contiguous().cuda())

    def run(self, vsd, weights="new", stride=None, **kw):
        """(caches, scales, weights_out) after the call, on the CPU."""
        as_type = torch.float8_e4m3fn if self.quant else torch.bfloat16
        dev = [c.cuda().view(as_type) for c in self.caches]
        sc = [s.cuda() for s in self.scales]
        tab = self.table.cuda()
        dst = tab if self.dst is self.table else self.dst.cuda()
        w = None if weights == "none" else self.weights.cuda()
        out = {"none": None, "new": None, "place": w}.get(weights, None)
        if weights == "given":
            out = torch.full((w.shape[0], w.shape[1], stride), 9.0, device="cuda")
        call = vsd.vsd_compact_kv_quant if self.quant else vsd.vsd_compact_kv
        idx, n = kw.pop("lists", None) or self.lists()
        prefix = kw.pop("prefix", None)
        got = call(*dev, *sc, kw.pop("table", tab), kw.pop("dst", dst), int32(self.lengths) if prefix is None else prefix,
                   idx, n, weights=w, weights_out=out, **kw)
        assert out is None or got is out
        raw = torch.uint8 if self.quant else torch.int16
        return [c.view(raw).cpu() for c in dev], [s.cpu() for s in sc], None if got is None else got.cpu()

    def want(self):
        caches, scales = [c.clone() for c in self.caches], [s.clone() for s in self.scales]
        out = torch.zeros((len(self.lengths), self.Hkv, self.k))
        for b in range(len(self.lengths)):
            for g in range(self.Hkv):
                h = g if self.heads else 0
                n = int(self.n[b, h])
                j = self.idx[b, h, :n].long()
                src = self.table[b].long()[j // PAGE]
                out[b, g, :n] = self.weights[b, g, j]
                for kv in range(2):
                    rows = self.caches[kv][src, g, j % PAGE]
                    for p in range(0, n, PAGE):
                        blk, m = int(self.dst[b, p // PAGE]), min(PAGE, n - p)
                        x = rows[p:p + m]
                        if self.quant:
                            s = self.scales[kv][src, g][p:p + m]
                            ratio = s / s.max()
                            y = ref.encode((ref.decode(x).float() * ratio[:, None]).double())
                            x = torch.where((ratio == 1)[:, None], x, y)
                            scales[kv][blk, g] = s.max()
                        caches[kv][blk, g, :m] = x
        return caches, scales, out

    def check(self, got):
        want = self.want()
        for a, b in zip(got[0], want[0]):
            if self.quant:                        # (a NaN's sign says nothing)
                a, b = (torch.where((x & 0x7F) == 0x7F, torch.tensor(0x7F, dtype=torch.uint8), x) for x in (a, b))
            assert torch.equal(a, b)
        assert all(torch.equal(a, b) for a, b in zip(got[1], want[1]))
        if got[2] is not None:
            k = self.k
            assert torch.equal(got[2][..., :k], want[2])
            assert torch.all(got[2][..., k:] == 0)


@pytest.mark.parametrize("quant", [False, True])
@pytest.mark.parametrize("heads", [False, True])
@pytest.mark.parametrize("where", ["same", "copy", "other", "mixed"])
@pytest.mark.parametrize("lengths,k,Hkv,d", [
    ([1], 1, 1, 64), ([0, 5, 16, 17, 40], 16, 2, 64), ([100, 33, 7], 33, 3, 128), ([300, 299], 250, 2, 128),
    ([1000, 64, 1], 129, 2, 64), ([3000], 1500, 4, 128),
])
def test_moves(vsd, lengths, k, Hkv, d, where, heads, quant):
    c = Case(lengths, k, Hkv, d, quant, heads, seed=k + d, where=where)
    c.check(c.run(vsd))
    assert vsd.vsd_read_device_status() == 0


@pytest.mark.parametrize("quant", [False, True])
def test_long_lists_in_place(vsd, quant):
    """Several steps of the widest clusters, most rows kept (sources just ahead of places)."""
    c = Case([20000, 12345], 16000, 1, 64, quant, True, seed=1)
    c.check(c.run(vsd))
    c = Case([3000] * 12, 1500, 8, 64, quant, False, seed=2)
    c.check(c.run(vsd))


def test_nothing_evicted(vsd):
    """Every row kept: an in-place call changes nothing; neither does a second one."""
    for quant in (False, True):
        c = Case([50, 16, 0], 64, 2, 64, quant, False, seed=3)
        got = c.run(vsd, weights="place") if c.weights.shape[2] >= 64 else c.run(vsd, weights="given", stride=70)
        assert all(torch.equal(a, b) for a, b in zip(got[0], c.caches))
        for a, b, t in zip(got[1], c.scales, (0, 1)):
            assert torch.equal(a, b)
        for b, n in enumerate(c.lengths):
            assert torch.equal(got[2][b, :, :n], c.weights[b, :, :n]) and torch.all(got[2][b, :, n:] == 0)


@pytest.mark.parametrize("quant", [False, True])
def test_weights_in_place_and_given(vsd, quant):
    c = Case([500, 200, 0], 130, 2, 64, quant, True, seed=4)
    c.check(c.run(vsd, weights="place"))
    c.check(c.run(vsd, weights="given", stride=333))
    c.check(c.run(vsd, weights="given", stride=130))
    c.check(c.run(vsd, weights="none"))


def test_scales_of_no_power(vsd):
    c = Case([700, 90], 300, 2, 128, True, True, seed=5, power=False)
    c.check(c.run(vsd))


def test_scales_of_zero(vsd):
    """Pages of scale 0 (rows of zeros) beside others, and alone."""
    c = Case([64, 64], 40, 1, 64, True, False, seed=6, where="other")
    for s in c.scales:
        s[c.table[0, :2].long()] = 0.0
        s[c.table[1].long()] = 0.0
    got = c.run(vsd)
    want = c.want()
    n = 40
    for kv in range(2):
        for b in range(2):
            for p in range(0, n, PAGE):
                blk, m = int(c.dst[b, p // PAGE]), min(PAGE, n - p)
                assert torch.equal(got[1][kv][blk], want[1][kv][blk])
                value = ref.decode(got[0][kv][blk, 0, :m]) * got[1][kv][blk].double()
                j = c.idx[b, 0, p:p + m].long()
                src = c.table[b].long()[j // PAGE]
                was = ref.decode(c.caches[kv][src, 0, j % PAGE]) * c.scales[kv][src, 0].double()[:, None]
                # (requantised to the largest scale: half a step, exact for scales that are equal)
                assert torch.all(((value - was).abs() <= 2.0 ** -4 * was.abs() + 2.0 ** -10 * float(got[1][kv][blk])) | torch.isnan(was))


def test_refused_lists_and_entries(vsd):
    c = Case([100, 100, 100, 100, 100], 40, 2, 64, False, False, seed=7, where="other")
    idx, n = c.lists()
    n[0], n[1] = -1, 41                                      # counts outside
    idx[2, 5], idx[2, 6], idx[2, 39] = 100, 3, -1             # beyond the prefix, below its place, none
    table, dst = c.table.clone(), c.dst.clone()
    j = int(c.idx[3, 0, 17])
    table[3, j // PAGE] = 10 ** 6
    dst[4, 1] = -1
    out = torch.full((5, 2, 40), 9.0, device="cuda")
    dev = [x.cuda().view(torch.bfloat16) for x in c.caches]
    vsd.vsd_compact_kv(*dev, table.cuda(), dst.cuda(), int32(c.lengths), idx, n, weights=c.weights.cuda(), weights_out=out)
    assert vsd.vsd_read_device_status() == vsd.DEV_BAD_LENGTH | vsd.DEV_BAD_INDEX | vsd.DEV_BAD_BLOCK
    got, w = [x.view(torch.int16).cpu() for x in dev], out.cpu()
    assert torch.all(w[:2] == 9)
    skipped = {2: {5, 6, 39}, 3: {i for i in range(40) if int(c.idx[3, 0, i]) // PAGE == j // PAGE}, 4: set(range(16, 32))}
    want, _, want_w = c.want()
    for b in range(5):
        for i in range(40):
            blk = int(c.dst[b, i // PAGE])
            moved = b >= 2 and i not in skipped[b]
            for kv in range(2):
                assert torch.equal(got[kv][blk, :, i % PAGE], (want if moved else c.caches)[kv][blk, :, i % PAGE])
            if b >= 2:
                assert torch.equal(w[b, :, i], want_w[b, :, i] if moved or b == 4 else torch.zeros(2))
    # prefix lengths that cannot be, and a destination of too few pages
    for kw in (dict(prefix=int32([-1, 10 ** 6, -5, -1, -1])), dict(dst=c.dst[:, :2].contiguous().cuda())):
        got = c.run(vsd, **kw)
        assert vsd.vsd_read_device_status() == vsd.DEV_BAD_LENGTH
        assert all(torch.equal(a, b) for a, b in zip(got[0], c.caches)) and torch.all(got[2] == 0)


def test_repeated_captured_and_on_another_stream(vsd):
    c = Case([600, 300], 200, 2, 128, True, False, seed=8, where="other")
    dev = [x.cuda().view(torch.float8_e4m3fn) for x in c.caches]
    sc, tab, dst, pl = [x.cuda() for x in c.scales], c.table.cuda(), c.dst.cuda(), int32(c.lengths)
    idx, n = c.lists()
    w, out = c.weights.cuda(), torch.zeros((2, 2, 200), device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        vsd.vsd_compact_kv_quant(*dev, *sc, tab, dst, pl, idx, n, weights=w, weights_out=out)
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    c.check(([x.view(torch.uint8).cpu() for x in dev], [x.cpu() for x in sc], out.cpu()))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        c.check(c.run(vsd))


def test_mismatched_tensors(vsd):
    c = Case([30], 16, 2, 64, False, False, seed=9)
    kc, vc = (x.cuda().view(torch.bfloat16) for x in c.caches)
    tab, pl, w = c.table.cuda(), int32([30]), c.weights.cuda()
    idx, n = c.lists()

    def call(kc=kc, vc=vc, tab=tab, dst=tab, pl=pl, idx=idx, n=n, **kw):
        return vsd.vsd_compact_kv(kc, vc, tab, dst, pl, idx, n, **kw)
    assert call() is None
    for kw in (dict(vc=vc[1:]), dict(dst=tab.repeat(2, 1)), dict(pl=int32([1, 2])), dict(n=n[:0]), dict(idx=idx.view(1, 1, 16)),
               dict(idx=idx[:, ::2]), dict(weights=w[:, :1].contiguous()), dict(weights_out=w), dict(weights=w, weights_out=w[..., :8].contiguous()),
               dict(weights=w.cpu())):
        with pytest.raises(ValueError):
            call(**kw)
    for kw in (dict(kc=kc.float()), dict(idx=idx.long()), dict(weights=w.double()), dict(dst=None)):
        with pytest.raises(TypeError):
            call(**kw)
    apart = torch.zeros(200, device="cuda")
    with pytest.raises(vsd.VsdError):                 # partly over each other
        call(weights=apart[:60].view(1, 2, 30), weights_out=apart[50:110].view(1, 2, 30))
    with pytest.raises(vsd.VsdError):                 # one buffer, two strides
        call(weights=w, weights_out=w.view(-1)[:2 * 16].view(1, 2, 16))
