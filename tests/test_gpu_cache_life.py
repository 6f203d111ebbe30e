"""The operators in a run, as a decode uses them: a prompt's rows enter, tokens attend and their
weights gather, the cache is cut, and decoding goes on with positions that count every token."""
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


def int32(x):
    return torch.as_tensor(x, dtype=torch.int32).cuda()


class Model:
    """One layer's attention in 64 bits: rows kept as lists, one for each sequence and KV head."""

    def __init__(self, B, Hkv):
        self.k = [[[] for _ in range(Hkv)] for _ in range(B)]
        self.v = [[[] for _ in range(Hkv)] for _ in range(B)]
        self.w = [[torch.zeros(0, dtype=torch.float64) for _ in range(Hkv)] for _ in range(B)]


@pytest.mark.parametrize("heads", [False, True])
@pytest.mark.parametrize("quant", [False, True])
@pytest.mark.parametrize("graphed", [False, True])
def test_decode_with_eviction(vsd, quant, heads, graphed):
    B, Hq, Hkv, d, P0, k, steps = 2, 8, 2, 64, [150, 90], 64, 5
    G, scale = Hq // Hkv, d ** -0.5
    g = torch.Generator().manual_seed(21 + quant)
    freq = life.inv_freq(d, 10000.0)
    turns = vsd.vsd_rope_turns(freq)
    wq, wk = ((1 + 0.2 * torch.randn(d, generator=g)).to(torch.bfloat16) for _ in range(2))
    width = 16
    table = torch.arange(B * width, dtype=torch.int32).view(B, width)[:, torch.randperm(width, generator=g)].contiguous()
    tab = table.cuda()
    NB = B * width
    cache = [torch.zeros((NB, Hkv, PAGE, d), dtype=torch.uint8 if quant else torch.bfloat16, device="cuda") for _ in range(2)]
    if quant:
        cache = [c.view(torch.float8_e4m3fn) for c in cache] + [torch.zeros((NB, Hkv), device="cuda") for _ in range(2)]
    W = 256
    weights = torch.zeros((B, Hkv, W), device="cuda")
    norm = dict(q_weight=wq.cuda(), k_weight=wk.cuda())
    append = vsd.vsd_norm_rope_append_kv_quant if quant else vsd.vsd_norm_rope_append_kv

    def rows(n):
        x = torch.randn((B, n, Hq + 2 * Hkv, d), generator=g).to(torch.bfloat16)
        y = x.cuda()
        return x, (y[:, :, :Hq], y[:, :, Hq:Hq + Hkv], y[:, :, Hq + Hkv:])

    # a padded prompt
    n0 = max(P0)
    x, parts = rows(n0)
    append(*parts, *cache, tab, int32([0, 0]), turns, n_valid=int32(P0), **norm)
    held, seen = int32(P0), int32(P0)        # rows in the cache, tokens of the sequence
    one = [torch.zeros((B, 1, h, d), dtype=torch.bfloat16, device="cuda") for h in (Hq, Hkv, Hkv)]

    def step():
        """One token of each sequence: its row, its attention, its weights."""
        q = append(*one, *cache, tab, held, turns, rope_base=seen, **norm)
        if quant:
            out, logits, _ = vsd.vsd_verify_attn_collect_quant(q, *cache, tab, held, P_max=W, scale=scale,
                                                               workspace=None)
            vsd.vsd_accumulate_weights_quant(logits, q, cache[0], cache[2], tab, held, weights, scale=scale)
        else:
            out, logits, _ = vsd.vsd_verify_attn_collect(q, *cache, tab, held, P_max=W, scale=scale)
            vsd.vsd_accumulate_weights(logits, q, cache[0], tab, held, weights, scale=scale)
        held.add_(1)
        seen.add_(1)
        return q, out

    def cut():
        if heads:
            idx, n, _ = vsd.vsd_select_topk(weights.view(B * Hkv, 1, W), held.repeat_interleave(Hkv), k=k, n_sink=4, n_recent=16)
            idx, n = idx.view(B, Hkv, k), n.view(B, Hkv)
        else:
            idx, n, _ = vsd.vsd_select_topk(weights, held, k=k, n_sink=4, n_recent=16)
        call = vsd.vsd_compact_kv_quant if quant else vsd.vsd_compact_kv
        call(*cache, tab, tab, held, idx, n, weights=weights, weights_out=weights)
        held.copy_(n[:, 0] if heads else n)
        return idx

    if graphed:
        vsd.vsd_verify_attn_collect(torch.zeros((B, 1, Hq, d), dtype=torch.bfloat16, device="cuda"),
                                    *[torch.zeros((NB, Hkv, PAGE, d), dtype=torch.bfloat16, device="cuda")] * 2, tab,
                                    int32([0, 0]), P_max=W, scale=scale)     # its workspace exists before the capture
        torch.cuda.synchronize()
        step_graph, cut_graph = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
        with torch.cuda.graph(step_graph):
            step_out = step()
        with torch.cuda.graph(cut_graph):
            cut_out = cut()

    # the model: positions of the kept rows, for each sequence and head
    at = [[list(range(P0[b])) for _ in range(Hkv)] for b in range(B)]

    def read(b, h, n):
        """The rows of the cache as it stands (their own rounding is other tests' matter)."""
        j = torch.arange(n)
        blk = table[b].long()[j // PAGE]
        c = [t.cpu() for t in cache]
        if quant:
            return [ref.decode(c[i].view(torch.uint8)[blk, h, j % PAGE]) * c[2 + i][blk, h].double()[:, None] for i in range(2)]
        return [c[i][blk, h, j % PAGE].double() for i in range(2)]

    def true_key(b, h, pos):
        return life.turned(hist[b][pos][Hq + h].double().view(1, 1, d), wk, 1e-6, [pos], freq, False)[0].view(d)

    hist = [[x[b, t] for t in range(P0[b])] for b in range(B)]
    total = torch.zeros((B, Hkv, W), dtype=torch.float64)
    for phase in range(3):
        for _ in range(steps):
            x, parts = rows(1)
            for dst, src in zip(one, parts):
                dst.copy_(src)
            if graphed:
                step_graph.replay()
                q, out = step_out
            else:
                q, out = step()
            torch.cuda.synchronize()
            for b in range(B):
                pos = len(hist[b])
                hist[b].append(x[b, 0])
                want_q, off = life.turned(x[b, 0, :Hq].double()[None], wq, 1e-6, [pos], freq, False)
                assert torch.all((q[b, 0].cpu().double() - want_q[0]).abs() <= life.bf16_bound(want_q, off)[0])
                for h in range(Hkv):
                    at[b][h].append(pos)
                    n = len(at[b][h])
                    kk, vv = read(b, h, n)
                    for i in (0, n // 2, n - 1):              # rows are those of the positions they should be
                        t = true_key(b, h, at[b][h][i])
                        assert torch.all((kk[i] - t).abs() <= (2.0 ** -3 if quant else 2.0 ** -7) * (t.abs() + 0.1 * t.abs().max()))
                    z = q[b, 0, h * G:(h + 1) * G].cpu().double() @ kk.T * scale
                    p = torch.softmax(z, 1)
                    want = p @ vv
                    # bf16 outputs, and probabilities held to 2^-8 (bf16) or 2^-11 of theirs
                    tol = 2.0 ** -8 * want.abs() + 2.0 ** -7 * (p @ vv.abs()) + 1e-6
                    assert torch.all((out[b, 0, h * G:(h + 1) * G].cpu().double() - want).abs() <= tol)
                    total[b, h, :n - 1] += p[:, :-1].sum(0)
        w = weights.cpu().double()
        # logits of order one in fp32, and the additions: 2^-11 of what is there
        assert torch.all((w - total).abs() <= 2.0 ** -11 * total)
        if graphed:
            cut_graph.replay()
            idx = cut_out
        else:
            idx = cut()
        torch.cuda.synchronize()
        idx = idx.cpu()
        new = torch.zeros_like(total)
        for b in range(B):
            for h in range(Hkv):
                n = min(k, len(at[b][h]))
                j = (idx[b, h] if heads else idx[b])[:n].long()
                assert set(range(4)) <= set(j.tolist()) and set(range(len(at[b][h]) - 16, len(at[b][h]))) <= set(j.tolist())
                new[b, h, :n] = w[b, h, j]
                at[b][h] = [at[b][h][i] for i in j.tolist()]
        total = new
        assert torch.equal(weights.cpu().double(), total)
        assert held.tolist() == [len(at[b][0]) for b in range(B)] and seen.tolist() == [len(x) for x in hist]
    assert vsd.vsd_read_device_status() == 0
