"""The operators around a cache's life, as measured cases.

Three operators share the paged KV cache (bf16 rows, or e4m3 codes with one fp32 scale for
each page and KV head): `rope` brings rows in (queries and keys normed per head and rotated by
their positions, keys and values stored in the same pass), `weights` adds the attention weight
of a verification's collected logits to each position's sum, `evict` keeps the positions of
the largest sums and moves their rows together.  `run` computes one of them, in plain torch
operations or (with `own`) by the framework's kernels; `exact` is the definition in 64 bits.
"""
import math

import torch

own = False

PAGE = 16
E4M3_MAX = 448.0
EPS = 1e-6


def listed():
    """The measured calls.  The geometries are those of the framework's workloads (Qwen3-8B
    and Qwen2.5-72B attention shapes, the tiny d = 64 case) and generic ones."""
    return [
        # a draft step of a served batch: one new token of each of 16 sequences, normed heads
        _rope("rope_one_token_b16", "bf16", 16, 1, 32, 8, 128, start=32771),
        # a prompt's rows from an empty cache
        _rope("rope_prompt_32k", "bf16", 1, 32768, 32, 8, 128),
        # a padded batch of prompt chunks that begin inside a page, a quarter-to-half rotation of
        # neighbouring pairs, no norms
        _rope("rope_chunks_ragged_d64", "bf16", 4, 1003, 16, 4, 64, rot=32, pairs=True, norm=False, start=205,
              ragged=True),
        # the verify blocks of a batch into an 8-bit cache, eight query heads a KV head, no norms
        _rope("rope_verify_block_8bit_b16", "8bit", 16, 6, 64, 8, 128, norm=False, start=8190),
        # a prompt chunk into an 8-bit cache that already holds some rows
        _rope("rope_chunk_4k_8bit", "8bit", 1, 4096, 32, 8, 128, start=205),
        # two rows of a short prefix, one KV head
        dict(name="weights_p512_d64", op="weights", store="bf16", B=1, P=512, Hq=4, Hkv=1, d=64, R=4, all=False,
             ragged=False),
        # the collected rows of a verification over one 32K sequence
        dict(name="weights_32k", op="weights", store="bf16", B=1, P=32768, Hq=32, Hkv=8, d=128, R=5, all=False,
             ragged=False),
        # every verify row of a batch of unequal sequences (a row stride that 4 does not divide)
        dict(name="weights_all_rows_ragged", op="weights", store="bf16", B=4, P=8203, Hq=32, Hkv=8, d=128, R=6,
             all=True, ragged=True),
        # the collected rows over a batch of 16 sequences of 32K, 8-bit cache
        dict(name="weights_batch16_32k", op="weights", store="8bit", B=16, P=32768, Hq=64, Hkv=8, d=128, R=6,
             all=False, ragged=False),
        # a padded batch of short sequences cut to 256 rows, a set for each KV head, 8-bit cache
        dict(name="evict_ragged_heads_d64_8bit", op="evict", store="8bit", B=5, P=1000, Hkv=4, d=64, k=256,
             heads=True, ragged=True),
        # one 32K sequence cut to 4096 rows, one set for all heads
        dict(name="evict_32k_to_4k", op="evict", store="bf16", B=1, P=32768, Hkv=8, d=128, k=4096, heads=False,
             ragged=False),
        # a batch of 16 sequences of 32K cut to 4096 rows each, 8-bit cache
        dict(name="evict_batch16_32k_8bit", op="evict", store="8bit", B=16, P=32768, Hkv=8, d=128, k=4096,
             heads=False, ragged=False),
    ]


def _rope(name, store, B, n, Hq, Hkv, d, rot=None, pairs=False, norm=True, start=0, ragged=False):
    c = dict(op="rope", store=store, B=B, n=n, Hq=Hq, Hkv=Hkv, d=d, rot=d if rot is None else rot, pairs=pairs,
             norm=norm, start=start, ragged=ragged)
    return dict(c, name=name) if name else c


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["rope", "rope", "weights", "evict"])
    B = _log_int(rng, 1, 16)
    d = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    G = rng.choice([1, 2, 4, 8])
    store = rng.choice(["bf16", "8bit"])
    ragged = rng.random() < 0.5
    if op == "rope":
        store = rng.choice(["bf16", "8bit", "rows"])      # rows: normed and rotated rows alone, no cache
        n = _log_int(rng, 1, (4096 if store == "8bit" else 32768 // G) // B)
        rot = rng.choice([d, d, d // 2, d // 4])
        return _rope("", store, B, n, Hkv * G, Hkv, d, rot, rng.random() < 0.3, rng.random() < 0.6,
                     rng.randrange(0, 100000), ragged)
    P = _log_int(rng, 1 if op == "weights" else 64, 131072 if B <= 4 else 32768)
    if op == "weights":
        R = rng.randint(1, min(16, 48 // G))
        whole = rng.random() < 0.25 and B * R * P * Hkv * G <= 32 << 20
        return dict(op=op, store=store, B=B, P=P, Hq=Hkv * G, Hkv=Hkv, d=d, R=R, all=whole, ragged=ragged)
    return dict(op=op, store=store, B=B, P=P, Hkv=Hkv, d=d, k=min(P, _log_int(rng, 16, 8192)),
                heads=rng.random() < 0.5, ragged=ragged)


# ------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 7919 + 23)
    return g


def _lengths(full, B, ragged, gen):
    """Per-sequence lengths: all `full`, or spread over [0, full] with a full one."""
    x = torch.full((B,), full, dtype=torch.int64, device="cuda")
    if ragged:
        u = torch.rand((B,), generator=gen, device="cuda", dtype=torch.float64)
        x = (u * full).long()
        x[0] = full
    return x


def _tables(caps, most, gen):
    """Shuffled block tables for several groups of sequences (caps: lengths [groups, B], at
    most most[group]) over one pool of blocks, -1 where unused; and the pool's size."""
    nblk = (caps + PAGE - 1) // PAGE
    NB = sum(-(-m // PAGE) for m in most) * caps.shape[1]
    perm = torch.randperm(NB, generator=gen, device="cuda")
    first = (torch.cumsum(nblk.view(-1), 0) - nblk.view(-1)).view(nblk.shape)
    tables = []
    for f, n in zip(first, nblk):
        at = torch.arange(max(1, int(n.max())), device="cuda")[None, :]
        slot = (f[:, None] + at).clamp_(max=NB - 1)
        tables.append(torch.where(at < n[:, None], perm[slot], -1).to(torch.int32))
    return tables, NB


def _rows(shape, gen):
    """Key / value rows: normal, with a channel profile and a few loud tokens."""
    *lead, H, d = shape
    x = torch.randn(shape, generator=gen, device="cuda")
    x *= torch.exp(0.4 * torch.randn((H, d), generator=gen, device="cuda"))
    x *= 1.0 + 3.0 * (torch.rand((*lead, 1, 1), generator=gen, device="cuda") < 0.01)
    return x


def _cache(NB, Hkv, d, store, gen):
    """A cache as it stands after its rows were stored: bf16 rows and None, or codes and
    power-of-two scales."""
    x = _rows((NB * PAGE, Hkv, d), gen).view(NB, PAGE, Hkv, d).transpose(1, 2)
    if store == "bf16":
        return x.to(torch.bfloat16).contiguous(), None
    s = torch.exp2(torch.ceil(torch.log2(x.abs().amax(dim=(2, 3)) / E4M3_MAX)))
    return (x / s[:, :, None, None]).to(torch.float8_e4m3fn).contiguous(), s


def prepare(case, seed):
    c, gen = case, _gen(seed)
    s = dict(case=case)
    B, Hkv, d = c["B"], c["Hkv"], c["d"]
    if c["op"] == "rope":
        n, Hq = c["n"], c["Hq"]
        # the three projections of a layer come as one product: q, k and v are views of it
        qkv = _rows((B, n, Hq + 2 * Hkv, d), gen).to(torch.bfloat16)
        s["q"], s["k_new"], s["v_new"] = qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hkv], qkv[:, :, Hq + Hkv:]
        for name in ("q_weight", "k_weight"):
            w = 1.0 + 0.2 * torch.randn((d,), generator=gen, device="cuda")
            s[name] = w.to(torch.bfloat16) if c["norm"] else None
        s["inv_freq"] = 1e6 ** (-torch.arange(0, c["rot"], 2, dtype=torch.float64, device="cuda") / c["rot"])
        start = torch.full((B,), c["start"], dtype=torch.int64, device="cuda")
        if c["start"]:       # every sequence begins at another place of a page
            start += torch.arange(B, device="cuda") * 5
        s["valid"] = _lengths(n, B, True, gen).to(torch.int32) if c["ragged"] else None
        s["q_out"] = torch.zeros((B, n, Hq, d), dtype=torch.bfloat16, device="cuda")
        s["pos"] = start.to(torch.int32)
        if c["store"] == "rows":
            s["k_out"] = torch.zeros((B, n, Hkv, d), dtype=torch.bfloat16, device="cuda")
        else:
            # rows long since evicted: the cache holds fewer rows than the sequence has had
            held = start.clamp(max=5000)
            s["at"] = held.to(torch.int32)
            (s["table"],), NB = _tables((held + n)[None], [int(held.max()) + n], gen)
            s["k"], s["ks"] = _cache(NB, Hkv, d, c["store"], gen)
            s["v"], s["vs"] = _cache(NB, Hkv, d, c["store"], gen)
        if own:              # the angles' table, made once for a model
            import sparse_attention_speculative_gb300 as vsd
            s["turns"] = vsd.vsd_rope_turns(s["inv_freq"])
        return s
    P = c["P"]
    prefix = _lengths(P, B, c["ragged"], gen)
    s["prefix"] = prefix.to(torch.int32)
    if c["op"] == "weights":
        Hq, R = c["Hq"], c["R"]
        (s["table"],), NB = _tables((prefix + R)[None], [P + R], gen)
        s["k"], s["ks"] = _cache(NB, Hkv, d, c["store"], gen)
        s["q"] = torch.randn((B, R, Hq, d), generator=gen, device="cuda").to(torch.bfloat16)
        s["scale"] = 1.0 / math.sqrt(d)
        C = R if c["all"] else 2
        # logits of the verify rows: a spread for each head, a loud first position
        z = torch.randn((B, C, Hq, P), generator=gen, device="cuda")
        z *= torch.exp(0.5 * torch.randn((B, 1, Hq, 1), generator=gen, device="cuda"))
        z[..., 0] += 6.0
        if not c["all"] and R == 1:
            z[:, 1] = z[:, 0]
        s["logits"] = z
        s["weights"] = 0.1 * torch.rand((B, Hkv, P), generator=gen, device="cuda") ** 4
        return s
    k = c["k"]
    s["n_sink"], s["n_recent"] = min(16, k // 8), min(256, k // 4)
    kept = prefix.clamp(max=k)
    (s["table"], s["dst"]), NB = _tables(torch.stack([prefix, kept]), [P, k], gen)
    s["k"], s["ks"] = _cache(NB, Hkv, d, c["store"], gen)
    s["v"], s["vs"] = _cache(NB, Hkv, d, c["store"], gen)
    # sums as they stand after a while: a few loud positions, many small ones, some exact zeros
    w = torch.exp(2.0 * torch.randn((B, Hkv, P), generator=gen, device="cuda") - 6.0)
    w *= torch.rand((B, Hkv, P), generator=gen, device="cuda") > 0.02
    s["weights"] = w.contiguous()
    s["weights_out"] = torch.zeros((B, Hkv, k), device="cuda")
    return s


# ------------------------------------------------------------------ one pass
def run(s):
    op = s["case"]["op"]
    if own:
        return {"rope": _own_rope, "weights": _own_weights, "evict": _own_evict}[op](s)
    return {"rope": _plain_rope, "weights": _plain_weights, "evict": _plain_evict}[op](s)


def _cache_of(s):
    r = dict(k=s["k"], v=s["v"])
    return r if s["ks"] is None else dict(r, k_scale=s["ks"], v_scale=s["vs"])


def _own_rope(s):
    import sparse_attention_speculative_gb300 as vsd
    c = s["case"]
    how = dict(n_valid=s["valid"], q_weight=s["q_weight"], k_weight=s["k_weight"], eps=EPS, interleaved=c["pairs"],
               q_out=s["q_out"])
    if c["store"] == "rows":
        q, k = vsd.vsd_norm_rope(s["q"], s["k_new"], s["turns"], s["pos"], k_out=s["k_out"], **how)
        return dict(q=q, k=k)
    if c["store"] == "bf16":
        q = vsd.vsd_norm_rope_append_kv(s["q"], s["k_new"], s["v_new"], s["k"], s["v"], s["table"], s["at"],
                                        s["turns"], rope_base=s["pos"], **how)
    else:
        q = vsd.vsd_norm_rope_append_kv_quant(s["q"], s["k_new"], s["v_new"], s["k"], s["v"], s["ks"], s["vs"],
                                              s["table"], s["at"], s["turns"], rope_base=s["pos"], **how)
    return dict(_cache_of(s), q=q)


def _own_weights(s):
    import sparse_attention_speculative_gb300 as vsd
    if s["ks"] is None:
        return vsd.vsd_accumulate_weights(s["logits"], s["q"], s["k"], s["table"], s["prefix"], s["weights"],
                                          scale=s["scale"])
    return vsd.vsd_accumulate_weights_quant(s["logits"], s["q"], s["k"], s["ks"], s["table"], s["prefix"],
                                            s["weights"], scale=s["scale"])


def _own_evict(s):
    import sparse_attention_speculative_gb300 as vsd
    c = s["case"]
    B, Hkv, k = c["B"], c["Hkv"], c["k"]
    w, prefix = s["weights"], s["prefix"]
    if c["heads"]:
        w, prefix = w.view(B * Hkv, 1, c["P"]), prefix.repeat_interleave(Hkv)
    idx, n_sel, _ = vsd.vsd_select_topk(w, prefix, k=k, n_sink=s["n_sink"], n_recent=s["n_recent"])
    if c["heads"]:
        idx, n_sel = idx.view(B, Hkv, k), n_sel.view(B, Hkv)
    args = (s["table"], s["dst"], s["prefix"], idx, n_sel)
    more = dict(weights=s["weights"], weights_out=s["weights_out"])
    if s["ks"] is None:
        vsd.vsd_compact_kv(s["k"], s["v"], *args, **more)
    else:
        vsd.vsd_compact_kv_quant(s["k"], s["v"], s["ks"], s["vs"], *args, **more)
    return dict(_cache_of(s), idx=idx, n_sel=n_sel, weights=s["weights_out"])


# ------------------------------------------------------------------ plain forms (32 bits)
def _normed(x, w):
    x = x.float()
    if w is None:
        return x
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w.float()


def _rotated(y, cos, sin, rot, pairs):
    """Rows y [B, n, H, d] turned by the angles of cos, sin [B, n, 1, rot / 2]."""
    if pairs:
        a, b = y[..., 0:rot:2], y[..., 1:rot:2]
        t = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = y[..., :rot // 2], y[..., rot // 2:rot]
        t = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([t, y[..., rot:]], -1)


def _plain_rope(s):
    c = s["case"]
    n = c["n"]
    t = torch.arange(n, device="cuda")[None, :]
    angle = (s["pos"].long()[:, None] + t).double()[:, :, None, None] * s["inv_freq"]     # [B, n, 1, rot / 2]
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    q = _rotated(_normed(s["q"], s["q_weight"]), cos, sin, c["rot"], c["pairs"]).to(torch.bfloat16)
    k = _rotated(_normed(s["k_new"], s["k_weight"]), cos, sin, c["rot"], c["pairs"])
    valid = s["valid"].long() if s["valid"] is not None else torch.full_like(s["pos"], n).long()
    keep = t < valid[:, None]
    if s["valid"] is not None:
        q = torch.where(keep[:, :, None, None], q, s["q_out"])
    if c["store"] == "rows":
        k = k.to(torch.bfloat16)
        return dict(q=q, k=k if s["valid"] is None else torch.where(keep[:, :, None, None], k, s["k_out"]))
    if c["store"] == "bf16":
        j = s["at"].long()[:, None] + t
        blk = torch.gather(s["table"].long(), 1, (j // PAGE).clamp(max=s["table"].shape[1] - 1))
        blk, row = blk[keep], (j % PAGE)[keep]
        s["k"][blk, :, row] = k.to(torch.bfloat16)[keep]
        s["v"][blk, :, row] = s["v_new"][keep]
    else:
        _store(s["k"], s["ks"], k, s["table"], s["at"].long(), valid)
        _store(s["v"], s["vs"], s["v_new"].float(), s["table"], s["at"].long(), valid)
    return dict(_cache_of(s), q=q)


def _store(codes, scales, new, table, pos, valid):
    """Rows new [B, n, Hkv, d] stored at pos .. pos + valid - 1 of each sequence.  A page's
    scale is the smallest power of two that keeps its rows within e4m3's range; a page that
    held earlier rows keeps its scale, or takes the larger one and has them requantised."""
    B, n, Hkv, d = new.shape
    pages = (n + PAGE - 2) // PAGE + 1
    off = pos % PAGE
    t = torch.arange(pages * PAGE, device=new.device)[None, :] - off[:, None]  # row of `new`
    stored = (t >= 0) & (t < valid[:, None])
    src = t.clamp(0, n - 1)
    x = torch.gather(new, 1, src[:, :, None, None].expand(B, pages * PAGE, Hkv, d))
    x = torch.where(stored[:, :, None, None], x, torch.zeros((), device=x.device))
    x = x.view(B, pages, PAGE, Hkv, d).transpose(2, 3)          # [B, pages, Hkv, 16, d]
    stored = stored.view(B, pages, PAGE)
    touched = stored.any(2)
    lp = (pos[:, None] // PAGE + torch.arange(pages, device=new.device)[None, :]).clamp(max=table.shape[1] - 1)
    blk = torch.gather(table.long(), 1, lp)
    blk, x, stored = blk[touched], x[touched], stored[touched]   # the pages that are written
    before = ~stored[:, 0]                                       # ... and held rows of the sequence
    first = torch.argmax(stored.to(torch.int32), dim=1)
    old = torch.arange(PAGE, device=new.device)[None, :] < first[:, None]
    was = scales[blk]
    amax = x.abs().amax(dim=(2, 3))
    m, e = torch.frexp(amax)                                     # amax = m 2^e, m in [0.5, 1)
    need = torch.where(amax > 0, e - 9 + (m > 0.875).to(e.dtype), torch.full_like(e, -126)).clamp(min=-126)
    now = torch.ldexp(torch.ones_like(amax), need)
    now = torch.where(before[:, None] & (amax <= was * E4M3_MAX), was, now)
    mine = (x / now[:, :, None, None]).to(torch.float8_e4m3fn)
    have = codes[blk]
    again = (have.float() * (was / now)[:, :, None, None]).to(torch.float8_e4m3fn)
    kept = torch.where(old[:, None, :, None], again.view(torch.uint8), have.view(torch.uint8))
    page = torch.where(stored[:, None, :, None], mine.view(torch.uint8), kept)
    codes.view(torch.uint8)[blk] = page
    scales[blk] = now


def _take(codes, scales, table, j):
    """Rows at positions j [B, n] of each sequence, in fp32: [B, n, Hkv, d]."""
    blk = torch.gather(table.long(), 1, (j // PAGE).clamp(max=table.shape[1] - 1)).clamp(min=0)
    x = codes[blk, :, j % PAGE].float()
    return x if scales is None else x * scales[blk][..., None]


def _plain_weights(s):
    c = s["case"]
    B, P, Hq, Hkv, R = c["B"], c["P"], c["Hq"], c["Hkv"], c["R"]
    rows = torch.arange(R, device="cuda") if c["all"] else torch.tensor([0, R - 1][:min(R, 2)], device="cuda")
    u = torch.arange(R, device="cuda")
    prefix = s["prefix"].long()
    key = _take(s["k"], s["ks"], s["table"], prefix[:, None] + u).repeat_interleave(Hq // Hkv, 2)  # [B, R, Hq, d]
    block = torch.einsum("bchd,buhd->bchu", s["q"][:, rows].float(), key) * s["scale"]
    block = torch.where(u <= rows[:, None, None], block, -torch.inf)
    seen = torch.arange(P, device="cuda") < prefix[:, None, None, None]
    z = torch.where(seen, s["logits"][:, :rows.numel()], -torch.inf)
    m = torch.maximum(z.amax(-1, keepdim=True), block.amax(-1, keepdim=True))
    e = torch.exp(z - m)
    total = e.sum(-1, keepdim=True) + torch.exp(block - m).sum(-1, keepdim=True)
    p = (e / total).view(B, rows.numel(), Hkv, Hq // Hkv, P).sum((1, 3))
    s["weights"] += p
    return s["weights"]


def _keep(s):
    """The kept positions of each sequence (and KV head, or 1): ascending, -1 behind them."""
    c = s["case"]
    B, Hkv, P, k = c["B"], c["Hkv"], c["P"], c["k"]
    if c["heads"]:
        w = s["weights"]
    else:                    # the heads' sums in their order: what the selection decides on
        w = torch.zeros((B, P), device="cuda")
        for g in range(Hkv):
            w = w + s["weights"][:, g]
        w = w[:, None]
    j, prefix = torch.arange(P, device="cuda"), s["prefix"].long()[:, None, None]
    kept = (j < s["n_sink"]) | (j >= prefix - s["n_recent"])
    w = torch.where(kept, torch.inf, w)
    w = torch.where(j < prefix, w, -torch.inf)
    order = w.sort(dim=-1, descending=True, stable=True).indices[..., :k]
    n = prefix.clamp(max=k)
    at = torch.arange(k, device="cuda")
    idx = torch.where(at < n, order, P).sort(dim=-1).values
    return torch.where(idx < P, idx, -1), n.expand(B, idx.shape[1], 1)[..., 0]


def _plain_evict(s):
    c = s["case"]
    B, Hkv, k = c["B"], c["Hkv"], c["k"]
    idx, n = _keep(s)
    j = idx.expand(B, Hkv, k).clamp(min=0)                       # [B, Hkv, k]
    there = torch.arange(k, device="cuda") < n[..., None].expand(B, Hkv, 1)
    g = torch.arange(Hkv, device="cuda")[None, :, None]
    b = torch.arange(B, device="cuda")[:, None, None]
    from_blk = s["table"].long()[b, j // PAGE].clamp(min=0)
    page = torch.arange(k, device="cuda") // PAGE
    to_blk = s["dst"].long()[:, page.clamp(max=s["dst"].shape[1] - 1)][:, None].expand(B, Hkv, k)
    to = (to_blk[there], g.expand(B, Hkv, k)[there], (torch.arange(k, device="cuda") % PAGE).expand(B, Hkv, k)[there])
    for name in ("k", "v"):
        cache, scales = s[name], s[name + "s"]
        if scales is None:
            cache[to] = cache[from_blk, g, j % PAGE][there]
            continue
        was = torch.where(there, scales[from_blk, g], 0.0)       # the rows' scales; a page takes their largest
        pages = -(-k // PAGE)
        top = torch.nn.functional.pad(was, (0, pages * PAGE - k)).view(B, Hkv, pages, PAGE).amax(-1)
        ratio = was / top.repeat_interleave(PAGE, -1)[..., :k].clamp(min=1e-38)
        rows = cache.view(torch.uint8)[from_blk, g, j % PAGE].view(torch.float8_e4m3fn).float() * ratio[..., None]
        cache.view(torch.uint8)[to] = rows.to(torch.float8_e4m3fn).view(torch.uint8)[there]
        first = there[..., ::PAGE]
        scales[to_blk[..., ::PAGE][first], g.expand(B, Hkv, pages)[first]] = top[first]
    s["weights_out"] = torch.where(there, torch.gather(s["weights"], 2, j), 0.0)
    n_sel = n if c["heads"] else n[:, 0]
    return dict(_cache_of(s), idx=(idx if c["heads"] else idx[:, 0]).to(torch.int32), n_sel=n_sel.to(torch.int32),
                weights=s["weights_out"])


# ------------------------------------------------------------------ definitions in 64 bits
def _nearest_e4m3(x):
    """The e4m3 value nearest to x (|x| <= 448), ties to the even code, in 64 bits."""
    e = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -9)))
    e = e - (torch.exp2(e) > x.abs()).double() + (torch.exp2(e + 1) <= x.abs()).double()
    step = torch.exp2(e.clamp(min=-6.0) - 3.0)
    return torch.round(x / step) * step


def _smallest_scale(top):
    """The smallest power of two s >= 2^-126 with top <= 448 s."""
    s = torch.exp2(torch.ceil(torch.log2(top.clamp(min=2.0 ** -118) / E4M3_MAX)).clamp(min=-126.0))
    return torch.where((top <= s / 2 * E4M3_MAX) & (s > 2.0 ** -126), s / 2, s)


def _exact_rope(s):
    c = s["case"]
    f64 = torch.float64
    B, n, rot = c["B"], c["n"], c["rot"]
    at = torch.arange(rot // 2, device="cuda")
    one, two = (2 * at, 2 * at + 1) if c["pairs"] else (at, at + rot // 2)

    def turned(x, w, b, rows):
        y = x[b, :rows].to(f64)
        if w is not None:
            y = y / torch.sqrt(y.square().sum(-1, keepdim=True) / c["d"] + EPS) * w.to(f64)
        pos = int(s["pos"][b]) + torch.arange(rows, dtype=f64, device="cuda")
        turn = torch.polar(torch.ones((rows, 1, rot // 2), dtype=f64, device="cuda"),
                           (pos[:, None] * s["inv_freq"]).remainder(2 * math.pi)[:, None])
        z = torch.complex(y[..., one], y[..., two]) * turn
        y[..., one], y[..., two] = z.real, z.imag
        return y

    rows_of = [n if s["valid"] is None else int(s["valid"][b]) for b in range(B)]
    res = dict(q=s["q_out"].to(f64))
    for b, rows in enumerate(rows_of):
        res["q"][b, :rows] = turned(s["q"], s["q_weight"], b, rows)
    if c["store"] == "rows":
        res["k"] = s["k_out"].to(f64)
        for b, rows in enumerate(rows_of):
            res["k"][b, :rows] = turned(s["k_new"], s["k_weight"], b, rows)
        return res
    table = s["table"].cpu()
    for name in ("k", "v"):
        res[name] = s[name].to(f64)
        if s[name + "s"] is not None:
            res[name + "_scale"] = s[name + "s"].to(f64)
        for b, rows in enumerate(rows_of):
            if not rows:
                continue
            x = turned(s["k_new"], s["k_weight"], b, rows) if name == "k" else s["v_new"][b, :rows].to(f64)
            lo = int(s["at"][b])
            j = torch.arange(lo, lo + rows, device="cuda")
            blk = table[b].cuda().long()
            if s[name + "s"] is None:
                res[name][blk[j // PAGE], :, j % PAGE] = x
                continue
            codes, scales = res[name], res[name + "_scale"]
            p0, p1 = lo // PAGE, (lo + rows + PAGE - 1) // PAGE
            held = torch.zeros(((p1 - p0) * PAGE, *x.shape[1:]), dtype=f64, device="cuda")
            held[lo - p0 * PAGE:lo - p0 * PAGE + rows] = x
            held = held.view(p1 - p0, PAGE, *x.shape[1:]).transpose(1, 2)
            sc = _smallest_scale(held.abs().amax((2, 3)))
            head = lo - p0 * PAGE                       # earlier rows of the first page
            if head:
                was = scales[blk[p0]].clone()
                sc[0] = torch.where(held[0].abs().amax((1, 2)) <= was * E4M3_MAX, was, sc[0])
                codes[blk[p0], :, :head] = _nearest_e4m3(codes[blk[p0], :, :head] * (was / sc[0])[:, None, None])
            q = _nearest_e4m3(held / sc[:, :, None, None]).transpose(1, 2).reshape(-1, *x.shape[1:])
            codes[blk[j // PAGE], :, j % PAGE] = q[head:head + rows]
            scales[blk[p0:p1]] = sc
    return res


def _exact_weights(s):
    c = s["case"]
    f64 = torch.float64
    R, G = c["R"], c["Hq"] // c["Hkv"]
    res = s["weights"].to(f64)
    rows = range(R) if c["all"] else sorted({0, R - 1})
    for b in range(c["B"]):
        P = int(s["prefix"][b])
        j = P + torch.arange(R, device="cuda")
        blk = s["table"][b].long()[j // PAGE]
        key = s["k"][blk, :, j % PAGE].to(f64)
        if s["ks"] is not None:
            key = key * s["ks"][blk].to(f64)[:, :, None]
        for slot, r in enumerate(rows):
            z = s["logits"][b, slot, :, :P].to(f64)
            mine = torch.stack([key[:r + 1, h // G] @ s["q"][b, r, h].to(f64) for h in range(c["Hq"])]) * s["scale"]
            p = torch.softmax(torch.cat([z, mine], 1), 1)[:, :P]
            res[b, :, :P] += p.view(c["Hkv"], G, P).sum(1)
    return res


def _exact_evict(s):
    c = s["case"]
    f64 = torch.float64
    B, Hkv, k = c["B"], c["Hkv"], c["k"]
    res = {name: s[name].to(f64) for name in ("k", "v")}
    if s["ks"] is not None:
        res.update(k_scale=s["ks"].to(f64), v_scale=s["vs"].to(f64))
    out = torch.zeros((B, Hkv, k), dtype=f64, device="cuda")
    for b in range(B):
        P = int(s["prefix"][b])
        n = min(P, k)
        if not n:
            continue
        w = s["weights"][b, :, :P].cpu()
        if not c["heads"]:
            total = torch.zeros(P)                      # (32 bits, head after head: what is decided on)
            for g in range(Hkv):
                total += w[g]
            w = total[None].expand(Hkv, P)
        j = torch.arange(P)
        safe = (j < s["n_sink"]) | (j >= P - s["n_recent"])
        cand = j[~safe]
        for g in range(Hkv):
            best = sorted(zip((-w[g][cand].double()).tolist(), cand.tolist()))[:n - int(safe.sum())]
            idx = torch.tensor(sorted(j[safe].tolist() + [x for _, x in best]), device="cuda")
            out[b, g, :n] = s["weights"][b, g, idx].to(f64)
            src = s["table"][b].long()[idx // PAGE]
            to = torch.arange(n, device="cuda")
            dst = s["dst"][b].long()[to // PAGE]
            for name in ("k", "v"):
                rows = s[name][src, g, idx % PAGE].to(f64)
                if s["ks"] is not None:
                    was = s[name + "s"][src, g].to(f64)
                    new = torch.stack([x.amax() for x in was.split(PAGE)])
                    rows = _nearest_e4m3(rows * (was / new[to // PAGE])[:, None])
                    res[name + "_scale"][dst[::PAGE], g] = new
                res[name][dst, g, to % PAGE] = rows
    return dict(res, idx=None, n_sel=None, weights=out)


def exact(case, seed):
    s = prepare(case, seed)
    return {"rope": _exact_rope, "weights": _exact_weights, "evict": _exact_evict}[case["op"]](s)


# ------------------------------------------------------------------ what a pass needs
def work(case):
    c = case
    B, Hkv, d = c["B"], c["Hkv"], c["d"]
    share = (1.0 + (0.5 if c["ragged"] else 1.0) * (B - 1)) / B   # mean length of a ragged batch: one is full
    held = d + 4 / PAGE if c["store"] == "8bit" else 2 * d        # a stored row of one head
    if c["op"] == "rope":
        rows = B * c["n"] * share
        kv = Hkv * 4 * d if c["store"] == "rows" else 2 * Hkv * (2 * d + held)
        return dict(bytes=rows * (c["Hq"] * 4 * d + kv), flops=rows * (c["Hq"] + Hkv) * d * (7 if c["norm"] else 3))
    keys = B * c["P"] * share
    if c["op"] == "weights":
        C = c["R"] if c["all"] else min(c["R"], 2)
        return dict(bytes=keys * (4 * C * c["Hq"] + 8 * Hkv) + B * (c["R"] * Hkv * held + C * c["Hq"] * 2 * d),
                    flops=keys * C * c["Hq"] * 4)
    kept = min(keys, B * c["k"])
    return dict(bytes=keys * Hkv * 4 + kept * Hkv * (4 * held + 8) + kept * 4 * (Hkv if c["heads"] else 1),
                flops=keys * Hkv)
