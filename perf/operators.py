"""The operators of the 8-bit paged KV cache, as measured cases.

Four operators share one cache (e4m3 codes [num_blocks][Hkv][16][d] with one fp32 scale
for each page and KV head, K and V apart): storing new rows (quantising them), reading
rows back, verification / decode attention with the collected logits, and the sparse
draft step.  `run` computes one of them, in plain torch operations or (with `own`) by
the framework's kernels; `exact` is the definition in 64 bits.
"""
import math

import torch

own = False

PAGE = 16
E4M3_MAX = 448.0


def listed():
    """The measured calls.  The geometries are those of the framework's workloads (Qwen3-8B
    and Qwen2.5-72B attention shapes, the tiny d = 64 case) and generic ones."""
    return [
        # a draft step of a served batch: one new token of each of 16 sequences
        dict(name="append_one_token_b16", op="append", B=16, n=1, Hkv=8, d=128, start=32771, ragged=False),
        # a prompt's rows after its prefill, from an empty cache
        dict(name="append_prompt_32k", op="append", B=1, n=32768, Hkv=8, d=128, start=0, ragged=False),
        # a padded batch of prompt chunks that begin inside a page, head_dim 64
        dict(name="append_chunks_ragged_d64", op="append", B=4, n=1003, Hkv=4, d=64, start=205, ragged=True),
        # a few rows of a padded batch read back
        dict(name="read_rows_ragged_d64", op="read", B=5, n=37, Hkv=4, d=64, start=130, ragged=True),
        # a long sequence handed to an operator that takes bf16
        dict(name="read_sequence_64k", op="read", B=1, n=65536, Hkv=8, d=128, start=0, ragged=False),
        # verification of four rows against a short prefix, one KV head
        dict(name="verify_p512_d64", op="verify", B=1, P=512, Hq=4, Hkv=1, d=64, R=4, ragged=False, collect=True),
        # single tokens of a batch of unequal sequences (no logits collected)
        dict(name="decode_one_row_ragged_b8", op="verify", B=8, P=8200, Hq=32, Hkv=8, d=128, R=1, ragged=True, collect=False),
        # verification over one 32K sequence, two rows' logits collected
        dict(name="verify_32k", op="verify", B=1, P=32768, Hq=32, Hkv=8, d=128, R=5, ragged=False, collect=True),
        # verification over a batch of 16 sequences of 32K, eight query heads a KV head
        dict(name="verify_batch16_32k", op="verify", B=16, P=32768, Hq=64, Hkv=8, d=128, R=6, ragged=False, collect=True),
        # the draft step of one 32K sequence over 2048 selected positions
        dict(name="draft_32k", op="draft", B=1, P=32768, Hq=32, Hkv=8, d=128, k=2048, tail=5, ragged=False),
        # the draft step of a batch of 16 over 512 selected positions each
        dict(name="draft_batch16_32k", op="draft", B=16, P=32768, Hq=64, Hkv=8, d=128, k=512, tail=7, ragged=False),
        # the draft step of four 64K sequences over 4096 selected positions, unequal lists
        dict(name="draft_64k_ragged", op="draft", B=4, P=65536, Hq=32, Hkv=8, d=128, k=4096, tail=11, ragged=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["append", "read", "verify", "draft"])
    B = _log_int(rng, 1, 16)
    d = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    ragged = rng.random() < 0.5
    if op in ("append", "read"):
        n = _log_int(rng, 1, (32768 if op == "append" else 65536) // B)
        return dict(op=op, B=B, n=n, Hkv=Hkv, d=d, start=rng.randrange(0, 4000), ragged=ragged)
    G = rng.choice([1, 2, 4, 8])
    if op == "verify":
        R = rng.randint(1, min(16, 48 // G))
        P = _log_int(rng, 1, 131072 if B <= 4 else 32768)
        return dict(op=op, B=B, P=P, Hq=Hkv * G, Hkv=Hkv, d=d, R=R, ragged=ragged, collect=rng.random() < 0.7)
    P = _log_int(rng, 64, 131072 if B <= 4 else 32768)
    k = min(P, _log_int(rng, 16, 8192))
    return dict(op=op, B=B, P=P, Hq=Hkv * G, Hkv=Hkv, d=d, k=k, tail=rng.randint(1, 15), ragged=ragged)


# ------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 7919 + 11)
    return g


def _lengths(full, B, ragged, gen):
    """Per-sequence lengths: all `full`, or spread over [0, full] with a full one."""
    x = torch.full((B,), full, dtype=torch.int64, device="cuda")
    if ragged:
        u = torch.rand((B,), generator=gen, device="cuda", dtype=torch.float64)
        x = (u * full).long()
        x[0] = full
    return x


def _table(caps, gen):
    """A shuffled block table for sequences of `caps` tokens (-1: unused entries), and the
    number of physical blocks."""
    nblk = (caps + PAGE - 1) // PAGE
    NB = int(nblk.sum())
    width = max(1, int(nblk.max()))
    perm = torch.randperm(NB, generator=gen, device="cuda")
    at = torch.arange(width, device="cuda")[None, :]
    first = torch.cumsum(nblk, 0) - nblk
    slot = (first[:, None] + at).clamp_(max=NB - 1)
    return torch.where(at < nblk[:, None], perm[slot], -1).to(torch.int32), NB


def _rows(shape, gen):
    """Key / value rows: normal, with a channel profile and a few loud tokens."""
    *lead, Hkv, d = shape
    x = torch.randn(shape, generator=gen, device="cuda")
    x *= torch.exp(0.4 * torch.randn((Hkv, d), generator=gen, device="cuda"))
    x *= 1.0 + 3.0 * (torch.rand((*lead, 1, 1), generator=gen, device="cuda") < 0.01)
    return x


def _filled_cache(NB, Hkv, d, gen):
    """A cache as it stands after its rows were stored: codes and power-of-two scales."""
    x = _rows((NB * PAGE, Hkv, d), gen).view(NB, PAGE, Hkv, d).transpose(1, 2)
    amax = x.abs().amax(dim=(2, 3))
    s = torch.exp2(torch.ceil(torch.log2(amax / E4M3_MAX)))
    codes = (x / s[:, :, None, None]).to(torch.float8_e4m3fn).contiguous()
    return codes, s


def prepare(case, seed):
    c, gen = case, _gen(seed)
    s = dict(case=case)
    B, Hkv, d = c["B"], c["Hkv"], c["d"]
    if c["op"] in ("append", "read"):
        n = c["n"]
        # every sequence begins at another place of a page when `start` is not 0
        start = torch.full((B,), c["start"], dtype=torch.int64, device="cuda")
        if c["start"]:
            start += torch.arange(B, device="cuda") * 5
        s["table"], NB = _table(start + n, gen)
        s["pos"] = start.to(torch.int32)
        s["valid"] = _lengths(n, B, True, gen).to(torch.int32) if c["ragged"] else None
        s["k"], s["ks"] = _filled_cache(NB, Hkv, d, gen)
        s["v"], s["vs"] = _filled_cache(NB, Hkv, d, gen)
        if c["op"] == "append":
            s["k_new"] = _rows((B, n, Hkv, d), gen).to(torch.bfloat16)
            s["v_new"] = _rows((B, n, Hkv, d), gen).to(torch.bfloat16)
        else:
            s["k_out"] = torch.zeros((B, n, Hkv, d), dtype=torch.bfloat16, device="cuda")
            s["v_out"] = torch.zeros_like(s["k_out"])
        return s
    Hq, P = c["Hq"], c["P"]
    prefix = _lengths(P, B, c["ragged"], gen)
    extra = c["R"] if c["op"] == "verify" else c["tail"]
    s["table"], NB = _table(prefix + extra, gen)
    s["k"], s["ks"] = _filled_cache(NB, Hkv, d, gen)
    s["v"], s["vs"] = _filled_cache(NB, Hkv, d, gen)
    s["prefix"] = prefix.to(torch.int32)
    s["scale"] = 1.0 / math.sqrt(d)
    if c["op"] == "verify":
        s["q"] = torch.randn((B, c["R"], Hq, d), generator=gen, device="cuda").to(torch.bfloat16)
        s["out"] = torch.zeros_like(s["q"])
        if c["collect"]:
            s["logits"] = torch.zeros((B, 2, Hq, P), dtype=torch.float32, device="cuda")
            s["partial"] = torch.zeros((B, Hkv, P), dtype=torch.float32, device="cuda")
        return s
    k = c["k"]
    s["q"] = torch.randn((B, Hq, d), generator=gen, device="cuda").to(torch.bfloat16)
    s["out"] = torch.zeros_like(s["q"])
    # k distinct positions of each prefix, ascending, -1 behind them
    key = torch.rand((B, P), generator=gen, device="cuda")
    key = torch.where(torch.arange(P, device="cuda")[None, :] < prefix[:, None], key, 2.0)
    idx = key.argsort(dim=1)[:, :k]
    n_sel = torch.minimum(prefix, torch.full_like(prefix, k))
    idx = torch.where(torch.arange(k, device="cuda")[None, :] < n_sel[:, None], idx, P).sort(dim=1).values
    s["idx"] = torch.where(idx < P, idx, -1).to(torch.int32).contiguous()
    s["n_sel"] = n_sel.to(torch.int32)
    s["seq"] = (prefix + c["tail"]).to(torch.int32)
    return s


# ------------------------------------------------------------------ one pass
def run(s):
    op = s["case"]["op"]
    if own:
        return _run_own(s)
    return {"append": _plain_append, "read": _plain_read, "verify": _plain_verify,
            "draft": _plain_draft}[op](s)


def _run_own(s):
    import sparse_attention_speculative_gb300 as vsd
    c = s["case"]
    if c["op"] == "append":
        vsd.vsd_append_kv_quant(s["k_new"], s["v_new"], s["k"], s["v"], s["ks"], s["vs"], s["table"],
                                s["pos"], n_valid=s["valid"])
        return dict(k=s["k"], v=s["v"], k_scale=s["ks"], v_scale=s["vs"])
    if c["op"] == "read":
        k, v = vsd.vsd_read_kv_quant(s["k"], s["v"], s["ks"], s["vs"], s["table"], s["pos"], n=c["n"],
                                     n_valid=s["valid"], k_out=s["k_out"], v_out=s["v_out"])
        return dict(k=k, v=v)
    if c["op"] == "verify":
        out, logits, partial = vsd.vsd_verify_attn_collect_quant(
            s["q"], s["k"], s["v"], s["ks"], s["vs"], s["table"], s["prefix"], P_max=c["P"],
            scale=s["scale"], logits=s.get("logits"), partial=s.get("partial"), out=s["out"],
            collect=c["collect"])
        return dict(out=out, logits=logits, partial=partial) if c["collect"] else dict(out=out)
    out = vsd.vsd_sparse_decode_attn_quant(
        s["q"], s["k"], s["v"], s["ks"], s["vs"], s["table"], s["idx"], s["n_sel"], s["prefix"], s["seq"],
        scale=s["scale"], max_tail=c["tail"], out=s["out"])
    return dict(out=out)


# ------------------------------------------------------------------ plain forms (32 bits)
def _store(codes, scales, new, table, pos, valid):
    """Rows new [B, n, Hkv, d] stored at pos .. pos + valid - 1 of each sequence.  A page's
    scale is the smallest power of two that keeps its rows within e4m3's range; a page that
    held earlier rows keeps its scale, or takes the larger one and has them requantised."""
    B, n, Hkv, d = new.shape
    pages = (n + PAGE - 2) // PAGE + 1
    x = torch.zeros((B, pages * PAGE, Hkv, d), device=new.device)
    off = pos % PAGE
    t = torch.arange(pages * PAGE, device=new.device)[None, :] - off[:, None]  # row of `new`
    stored = (t >= 0) & (t < valid[:, None])
    src = t.clamp(0, n - 1)
    x = torch.gather(new.float(), 1, src[:, :, None, None].expand(B, pages * PAGE, Hkv, d))
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


def _plain_append(s):
    c = s["case"]
    pos = s["pos"].long()
    valid = s["valid"].long() if s["valid"] is not None else torch.full_like(pos, c["n"])
    _store(s["k"], s["ks"], s["k_new"], s["table"], pos, valid)
    _store(s["v"], s["vs"], s["v_new"], s["table"], pos, valid)
    return dict(k=s["k"], v=s["v"], k_scale=s["ks"], v_scale=s["vs"])


def _take(codes, scales, table, j):
    """Rows at positions j [B, n] of each sequence, in fp32: [B, n, Hkv, d]."""
    blk = torch.gather(table.long(), 1, (j // PAGE).clamp(max=table.shape[1] - 1)).clamp(min=0)
    return codes[blk, :, j % PAGE].float() * scales[blk][..., None]


def _plain_read(s):
    n = s["case"]["n"]
    t = torch.arange(n, device="cuda")[None, :]
    j = s["pos"].long()[:, None] + t
    keep = None if s["valid"] is None else (t < s["valid"][:, None])[:, :, None, None]
    out = []
    for codes, scales, to in ((s["k"], s["ks"], s["k_out"]), (s["v"], s["vs"], s["v_out"])):
        x = _take(codes, scales, s["table"], j).to(torch.bfloat16)
        out.append(x if keep is None else torch.where(keep, x, to))
    return dict(k=out[0], v=out[1])


def _pages(codes, scales, table):
    """A batch's pages in fp32: [B, Hkv, pages * 16, d]."""
    blk = table.long().clamp(min=0)
    x = codes[blk].float() * scales[blk][..., None, None]        # [B, pages, Hkv, 16, d]
    B, pages, Hkv, _, d = x.shape
    return x.transpose(1, 2).reshape(B, Hkv, pages * PAGE, d)


def _softmax_av(z, seen, v):
    """softmax over the last axis of z where `seen` (rows that see nothing: 0), times v."""
    m = torch.where(seen, z, -torch.inf).amax(-1, keepdim=True)
    p = torch.where(seen, torch.exp(z - torch.where(m == -torch.inf, 0.0, m)), 0.0)
    total = p.sum(-1, keepdim=True)
    return p @ v / torch.where(total > 0, total, 1.0)


def _plain_verify(s):
    c = s["case"]
    B, R, Hq, Hkv, d, P = c["B"], c["R"], c["Hq"], c["Hkv"], c["d"], c["P"]
    G = Hq // Hkv
    kf, vf = _pages(s["k"], s["ks"], s["table"]), _pages(s["v"], s["vs"], s["table"])
    L = kf.shape[2]
    q = s["q"].float().view(B, R, Hkv, G, d).permute(0, 2, 1, 3, 4).reshape(B, Hkv, R * G, d)
    z = (q @ kf.transpose(2, 3)) * s["scale"]                    # [B, Hkv, R * G, L]
    j = torch.arange(L, device="cuda")
    last = s["prefix"].long()[:, None] + torch.arange(R, device="cuda")[None, :]
    last = last[:, None, :, None].expand(B, 1, R, G).reshape(B, 1, R * G, 1)
    o = _softmax_av(z, j <= last, vf)
    out = o.view(B, Hkv, R, G, d).permute(0, 2, 1, 3, 4).reshape(B, R, Hq, d).to(torch.bfloat16)
    if not c["collect"]:
        return dict(out=out)
    rows = z.view(B, Hkv, R, G, L)[:, :, [0, R - 1], :, :P]
    rows = torch.where(j[:P] < s["prefix"].long()[:, None, None, None, None], rows, 0.0)
    partial = rows.sum((2, 3))
    return dict(out=out, logits=rows.permute(0, 2, 1, 3, 4).reshape(B, 2, Hq, P), partial=partial)


def _plain_draft(s):
    c = s["case"]
    B, Hq, Hkv, d, k = c["B"], c["Hq"], c["Hkv"], c["d"], c["k"]
    tail = s["prefix"].long()[:, None] + torch.arange(c["tail"], device="cuda")[None, :]
    j = torch.cat([s["idx"].long().clamp(min=0), tail], 1)
    seen = torch.arange(k, device="cuda")[None, :] < s["n_sel"][:, None]
    seen = torch.cat([seen, tail < s["seq"][:, None]], 1)[:, None, None, :]
    kf = _take(s["k"], s["ks"], s["table"], j).transpose(1, 2)   # [B, Hkv, n, d]
    vf = _take(s["v"], s["vs"], s["table"], j).transpose(1, 2)
    q = s["q"].float().view(B, Hkv, Hq // Hkv, d)
    o = _softmax_av((q @ kf.transpose(2, 3)) * s["scale"], seen, vf)
    return dict(out=o.reshape(B, Hq, d).to(torch.bfloat16))


# ------------------------------------------------------------------ definitions in 64 bits
def _nearest_e4m3(x):
    """The e4m3 value nearest to x (|x| <= 448), ties to the even code, in 64 bits."""
    e = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -9)))
    e = e - (torch.exp2(e) > x.abs()).double() + (torch.exp2(e + 1) <= x.abs()).double()
    step = torch.exp2(e.clamp(min=-6.0) - 3.0)
    return torch.round(x / step) * step


def exact(case, seed):
    s = prepare(case, seed)
    c = case
    f64 = torch.float64
    B, Hkv, d = c["B"], c["Hkv"], c["d"]
    table = s["table"].cpu().tolist()
    if c["op"] == "append":
        valid = s["valid"].tolist() if s["valid"] is not None else [c["n"]] * B
        pos = s["pos"].tolist()
        res = {}
        for name in ("k", "v"):
            codes, scales = s[name].to(f64), s[name + "s"].to(f64)
            for b in range(B):
                lo, hi = pos[b], pos[b] + valid[b]
                if hi == lo:
                    continue
                p0, p1 = lo // PAGE, (hi + PAGE - 1) // PAGE
                blk = torch.tensor(table[b][p0:p1], device="cuda")
                rows = torch.zeros(((p1 - p0) * PAGE, Hkv, d), dtype=f64, device="cuda")
                rows[lo - p0 * PAGE:hi - p0 * PAGE] = s[name + "_new"][b, :valid[b]].to(f64)
                rows = rows.view(p1 - p0, PAGE, Hkv, d).permute(0, 2, 1, 3)
                top = rows.abs().amax((2, 3))
                sc = torch.exp2(torch.ceil(torch.log2(top.clamp(min=2.0 ** -118) / E4M3_MAX)).clamp(min=-126.0))
                sc = torch.where((top <= sc / 2 * E4M3_MAX) & (sc > 2.0 ** -126), sc / 2, sc)   # log2 next to a border
                head = lo - p0 * PAGE                      # earlier rows of the first page
                if head:
                    was = scales[blk[0]].clone()
                    sc[0] = torch.where(top[0] <= was * E4M3_MAX, was, sc[0])
                    scale_by = (was / sc[0])[:, None, None]
                    codes[blk[0], :, :head] = _nearest_e4m3(codes[blk[0], :, :head] * scale_by)
                q = _nearest_e4m3(rows / sc[:, :, None, None]).permute(0, 2, 1, 3).reshape(-1, Hkv, d)
                j = torch.arange(lo, hi, device="cuda")
                codes[blk[j // PAGE - p0], :, j % PAGE] = q[lo - p0 * PAGE:hi - p0 * PAGE]
                scales[blk] = sc
            res[name], res[name + "_scale"] = codes, scales
        return dict(k=res["k"], v=res["v"], k_scale=res["k_scale"], v_scale=res["v_scale"])

    def rows_of(name, b, j):
        blk = torch.tensor(table[b], device="cuda")[j // PAGE]
        return s[name][blk, :, j % PAGE].to(f64) * s[name + "s"][blk].to(f64)[:, :, None]   # [n, Hkv, d]

    if c["op"] == "read":
        res = {"k": s["k_out"].to(f64), "v": s["v_out"].to(f64)}
        for b in range(B):
            n = c["n"] if s["valid"] is None else int(s["valid"][b])
            j = int(s["pos"][b]) + torch.arange(n, device="cuda")
            for name in ("k", "v"):
                res[name][b, :n] = rows_of(name, b, j)
        return res
    Hq, G = c["Hq"], c["Hq"] // Hkv
    prefix = s["prefix"].tolist()
    if c["op"] == "verify":
        R, P = c["R"], c["P"]
        out = torch.zeros((B, R, Hq, d), dtype=f64, device="cuda")
        logits = torch.zeros((B, 2, Hq, P), dtype=f64, device="cuda") if c["collect"] else None
        partial = torch.zeros((B, Hkv, P), dtype=f64, device="cuda") if c["collect"] else None
        for b in range(B):
            Pb = prefix[b]
            j = torch.arange(Pb + R, device="cuda")
            k, v = rows_of("k", b, j), rows_of("v", b, j)
            for g in range(Hkv):
                heads = slice(g * G, (g + 1) * G)
                for r in range(R):
                    n = Pb + r + 1
                    z = (s["q"][b, r, heads].to(f64) @ k[:, g].T) * s["scale"]
                    out[b, r, heads] = torch.softmax(z[:, :n], 1) @ v[:n, g]
                    if c["collect"]:
                        for slot, row in ((0, 0), (1, R - 1)):
                            if row == r:
                                logits[b, slot, heads, :Pb] = z[:, :Pb]
                                partial[b, g, :Pb] += z[:, :Pb].sum(0)
        return dict(out=out, logits=logits, partial=partial) if c["collect"] else dict(out=out)
    out = torch.zeros((B, Hq, d), dtype=f64, device="cuda")
    for b in range(B):
        j = torch.cat([s["idx"][b, :int(s["n_sel"][b])].long(),
                       torch.arange(prefix[b], int(s["seq"][b]), device="cuda")])
        k, v = rows_of("k", b, j), rows_of("v", b, j)
        for h in range(Hq):
            z = (k[:, h // G] @ s["q"][b, h].to(f64)) * s["scale"]
            out[b, h] = torch.softmax(z, 0) @ v[:, h // G]
    return dict(out=out)


# ------------------------------------------------------------------ what a pass needs
def work(case):
    c = case
    B, Hkv, d = c["B"], c["Hkv"], c["d"]
    share = 0.5 if c["ragged"] else 1.0           # mean length of a ragged batch, of the full one
    share = (1.0 + share * (B - 1)) / B           # one sequence is full
    if c["op"] in ("append", "read"):
        rows = B * c["n"] * share
        return dict(bytes=rows * Hkv * 2 * (3 * d + 4 / PAGE) + rows / PAGE * 4, flops=4 * rows * Hkv * d)
    Hq = c["Hq"]
    if c["op"] == "verify":
        keys = B * (c["P"] * share + c["R"])
        q_out = 2 * 2 * B * c["R"] * Hq * d
        collected = 4 * (2 * Hq + Hkv) * B * c["P"] * share if c["collect"] else 0
        return dict(bytes=keys * (Hkv * 2 * (d + 4 / PAGE) + 4 / PAGE) + q_out + collected,
                    flops=4 * keys * c["R"] * Hq * d)
    rows = B * (c["k"] * share + c["tail"])
    # a selected row lies in a page of its own: its scales and table entry are read for it
    return dict(bytes=rows * (Hkv * 2 * (d + 4) + 8) + 2 * 2 * B * Hq * d, flops=4 * rows * Hq * d)
