"""What the calls of normed and rotated rows, accumulated weights and eviction refuse on the host."""
import ctypes
import math
from fractions import Fraction

import pytest
import torch

from tests.test_quant_cache_refusals import GEOMETRIES, geom, lib, off, p  # noqa: F401


class Rows(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("batch", ctypes.c_int64), ("row", ctypes.c_int64), ("head", ctypes.c_int64)]


class Rope(ctypes.Structure):
    _fields_ = [("turns", ctypes.c_void_p), ("rot_dim", ctypes.c_int), ("interleaved", ctypes.c_int),
                ("amplitude", ctypes.c_float), ("q_weight", ctypes.c_void_p), ("k_weight", ctypes.c_void_p),
                ("eps", ctypes.c_float)]


FAR = 1 << 30   # (addresses that nothing reads: the checks come before any use)


def rows(p, batch=16384, row=4096, head=128):  # noqa: F811
    return Rows(p.value + FAR if p is not None else None, batch, row, head)


def rope(p, **kw):  # noqa: F811
    a = dict(turns=p.value, rot_dim=128, interleaved=0, amplitude=1.0, q_weight=None, k_weight=None, eps=1e-6)
    a.update(kw)
    return Rope(*(a[n] for n, _ in Rope._fields_))


def ref_of(x):
    return None if x is None else ctypes.byref(x)


def norm(lib, g, p, n=4, **kw):  # noqa: F811
    a = dict(q=rows(p), k=rows(off(p, 1 << 20)), r=rope(p), pos=p, nv=None, qo=p, ko=off(p, 1 << 20), z=0)
    a.update(kw)
    return lib.vsd_norm_rope(g, n, ref_of(a["q"]), ref_of(a["k"]), ref_of(a["r"]), a["pos"], 0, a["nv"], a["qo"],
                             a["ko"], a["z"], None)


def store(lib, g, p, n=4, **kw):  # noqa: F811
    a = dict(q=rows(p), k=rows(off(p, 1 << 20)), v=rows(off(p, 2 << 20)), r=rope(p), bt=p, pos=p, rb=None, nv=None, qo=p, z=0, kc=p, vc=p)
    a.update(kw)
    return lib.vsd_norm_rope_append_kv(g, n, ref_of(a["q"]), ref_of(a["k"]), ref_of(a["v"]), ref_of(a["r"]), a["bt"],
                                       a["pos"], 0, a["rb"], a["nv"], a["qo"], a["z"], a["kc"], a["vc"], None)


def store_quant(lib, g, p, n=4, **kw):  # noqa: F811
    a = dict(q=rows(p), k=rows(off(p, 1 << 20)), v=rows(off(p, 2 << 20)), r=rope(p), bt=p, pos=p, rb=None, nv=None, qo=p, z=0, kc=p, vc=p, ks=p,
             vs=p)
    a.update(kw)
    return lib.vsd_norm_rope_append_kv_quant(g, n, ref_of(a["q"]), ref_of(a["k"]), ref_of(a["v"]), ref_of(a["r"]),
                                             a["bt"], a["pos"], 0, a["rb"], a["nv"], a["qo"], a["z"], a["kc"],
                                             a["vc"], a["ks"], a["vs"], None)


def weights(lib, g, p, R=4, which=(0, 3), P_max=512, scale=0.1, stride=512, quant=False, **kw):  # noqa: F811
    a = dict(lg=p, q=p, kc=p, ks=p, bt=p, pl=p, w=p, rows=(ctypes.c_int * max(1, len(which)))(*which))
    a.update(kw)
    head = (g, R, len(which), a["rows"], a["lg"], a["q"], a["kc"])
    tail = (a["bt"], a["pl"], P_max, ctypes.c_float(scale), a["w"], stride, None)
    return lib.vsd_accumulate_weights_quant(*head, a["ks"], *tail) if quant else \
        lib.vsd_accumulate_weights(*head, *tail)


def compact(lib, g, p, dst=16, heads=1, k=64, ws=512, wos=512, quant=False, **kw):  # noqa: F811
    a = dict(bt=p, dt=p, pl=p, idx=p, ns=p, kc=p, vc=p, ks=p, vs=p, w=p, wo=off(p, 1 << 20))
    a.update(kw)
    head = (g, a["bt"], a["dt"], dst, a["pl"], a["idx"], a["ns"], heads, k, a["kc"], a["vc"])
    tail = (a["w"], ws, a["wo"], wos, None)
    return lib.vsd_compact_kv_quant(*head, a["ks"], a["vs"], *tail) if quant else lib.vsd_compact_kv(*head, *tail)


def weights_quant(lib, g, p, **kw):  # noqa: F811
    return weights(lib, g, p, quant=True, **kw)


def compact_quant(lib, g, p, **kw):  # noqa: F811
    return compact(lib, g, p, quant=True, **kw)


@pytest.mark.parametrize("call", [store, store_quant, weights, weights_quant, compact, compact_quant])
@pytest.mark.parametrize("kw,code", GEOMETRIES)
def test_geometry(lib, p, call, kw, code):  # noqa: F811
    assert call(lib, geom(**kw), p) == code
    assert call(lib, None, p) == -1


@pytest.mark.parametrize("call", [norm, store, store_quant])
def test_row_calls(lib, p, call):  # noqa: F811
    ptr = ["pos", "qo"] + (["ko"] if call is norm else ["bt", "kc", "vc"]) + (["ks", "vs"] if call is store_quant else [])
    for name in ptr:
        assert call(lib, geom(), p, **{name: None}) == -1
    for name in [x for x in ptr if x in ("qo", "ko", "kc", "vc")]:
        assert call(lib, geom(), p, **{name: off(p, 8)}) == -1
    for name in [x for x in ptr if x in ("bt", "pos", "ks", "vs")] + ["nv"]:
        assert call(lib, geom(), p, **{name: off(p, 2)}) == -1
    for name in ["q", "k"] + ([] if call is norm else ["v"]):
        for bad in (rows(None), rows(off(p, 8)), rows(p, batch=4), rows(p, row=12), rows(p, head=129)):
            assert call(lib, geom(), p, **{name: bad}) == -1
    assert call(lib, geom(), p, q=None) == -1
    if call is not norm:
        assert call(lib, geom(), p, k=None) == -1 and call(lib, geom(), p, v=None) == -1
        assert call(lib, geom(), p, rb=off(p, 2)) == -1
    assert call(lib, geom(), p, r=None) == -1
    for bad in (dict(rot_dim=-8), dict(rot_dim=136), dict(amplitude=math.inf), dict(eps=math.nan), dict(eps=-1.0),
                dict(turns=None), dict(turns=p.value + 4), dict(q_weight=p.value + 2), dict(k_weight=p.value + 8)):
        assert call(lib, geom(), p, r=rope(p, **bad)) == -1
    assert call(lib, geom(), p, r=rope(p, rot_dim=12)) == -2
    assert call(lib, geom(), p, z=4) == -1
    assert call(lib, geom(), p, n=-1) == -1
    assert call(lib, geom(B=2 ** 16), p, n=2 ** 16) == -2      # more warps than 32 bits count
    assert call(lib, geom(Hq=2 ** 19), p, n=1) == -2            # more heads than a token may have
    assert call(lib, geom(), p, n=0, q=None) == 0              # nothing to do: no device needed
    assert call(lib, geom(B=0), p, q=None) == 0


def test_outputs_that_overlap_rows(lib, p):  # noqa: F811
    """Refused, but for each row's own place.  (Zero rows of a bad count show what passed: the next check.)"""
    def call(**kw):
        return norm(lib, geom(Hq=32, Hkv=8), p, n=4, **kw)
    at = p.value + FAR
    for qo in (at - 16, at + 16, at + 4 * 4096 * 2 - 16, at - 4 * 4096 * 2 + 16):
        assert call(qo=ctypes.c_void_p(qo)) == -1
    # its own place: passes (and fails where there is no GPU, or is not run there: a null k_out is next)
    assert call(qo=ctypes.c_void_p(at), ko=None) == -1
    for bad in (rows(p, row=6144), rows(p, head=0), rows(p, head=256, row=8192)):
        assert call(q=bad, qo=ctypes.c_void_p(at)) == -1
    kat = at + (1 << 20)
    for ko in (kat + 16, kat - 16, at, p.value, p.value + 16):
        assert call(k=rows(off(p, 1 << 20), row=1024), ko=ctypes.c_void_p(ko)) == -1
    assert call(qo=ctypes.c_void_p(kat)) == -1                       # the queries over the keys
    assert store(lib, geom(), p, qo=ctypes.c_void_p(at + (2 << 20))) == -1      # over the values
    assert store_quant(lib, geom(), p, qo=ctypes.c_void_p(at + (2 << 20) + 64)) == -1


def test_norm_rope_needs_no_cache(lib, p):  # noqa: F811
    assert norm(lib, geom(page_size=0, num_blocks=0, max_blocks_per_seq=0, B=0), p) == 0
    assert norm(lib, geom(head_dim=96), p) == -2
    assert norm(lib, geom(Hq=30), p) == -1


@pytest.mark.parametrize("quant", [False, True])
def test_weights_call(lib, p, quant):  # noqa: F811
    def call(g=None, **kw):
        return weights(lib, g or geom(), p, quant=quant, **kw)
    for name in ["lg", "q", "kc", "bt", "pl", "w", "rows"] + (["ks"] if quant else []):
        assert call(**{name: None}) == -1
    for name in ("q", "kc"):
        assert call(**{name: off(p, 8)}) == -1
    for name in ["lg", "bt", "pl", "w"] + (["ks"] if quant else []):
        assert call(**{name: off(p, 2)}) == -1
    for which in ((0, 4), (-2, 0)):
        assert call(which=which) == -1
    assert call(stride=511) == -1
    assert call(scale=math.inf) == -1
    assert call(R=0) == -1 and call(R=17) == -2
    assert call(P_max=-1) == -1
    assert call(P_max=2 ** 30 + 1, stride=2 ** 31 - 1) == -2
    assert call(R=8, which=(0,) * 17, g=geom(Hq=8)) == -2
    assert call(R=8, which=(0,) * 9, g=geom(Hq=64)) == -2       # 72 columns
    assert call(g=geom(B=2 ** 23, Hkv=8)) == -2
    assert call(g=geom(B=0), lg=None) == 0
    assert call(P_max=0, stride=0, lg=None) == 0
    assert call(which=(-1, -1), lg=None) == 0                   # nothing counts
    assert call(which=(), lg=None) == 0


@pytest.mark.parametrize("quant", [False, True])
def test_compact_call(lib, p, quant):  # noqa: F811
    def call(g=None, **kw):
        return compact(lib, g or geom(), p, quant=quant, **kw)
    for name in ["bt", "dt", "pl", "idx", "ns", "kc", "vc"] + (["ks", "vs"] if quant else []):
        assert call(**{name: None}) == -1
    for name in ("kc", "vc"):
        assert call(**{name: off(p, 8)}) == -1
    for name in ["bt", "dt", "pl", "idx", "ns", "w", "wo"] + (["ks", "vs"] if quant else []):
        assert call(**{name: off(p, 2)}) == -1
    assert call(w=None) == -1 and call(wo=None) == -1
    assert call(wos=63) == -1 and call(ws=-1) == -1
    assert call(wo=p, ws=512, wos=256) == -1                    # in place with two strides
    for d in (4, 8 * 512 * 4 - 4):
        assert call(wo=off(p, d)) == -1 and call(w=off(p, d), wo=p) == -1      # partly over each other
    assert call(heads=2) == -1 and call(heads=0) == -1
    assert call(k=-1) == -1 and call(dst=-1) == -1
    assert call(k=2 ** 30 + 1, wos=2 ** 31 - 1) == -2
    assert call(g=geom(B=2 ** 23)) == -2
    assert call(g=geom(B=0), bt=None) == 0


def test_binding_refuses_wrong_tensors():
    import sparse_attention_speculative_gb300 as vsd
    B, n, Hq, Hkv, d, NB = 1, 3, 4, 2, 64, 4
    q, k = torch.zeros((B, n, Hq, d)).bfloat16(), torch.zeros((B, n, Hkv, d)).bfloat16()
    kc = torch.zeros((NB, Hkv, 16, d)).bfloat16()
    codes = torch.zeros((NB, Hkv, 16, d), dtype=torch.uint8).view(torch.float8_e4m3fn)
    s, f = torch.ones((NB, Hkv)), torch.zeros((B, Hkv, 8))
    bt, pos = torch.zeros((B, 4), dtype=torch.int32), torch.zeros((B,), dtype=torch.int32)
    turns = torch.zeros((32,), dtype=torch.int64)
    lg = torch.zeros((B, 2, Hq, 8))
    for call in (lambda: vsd.vsd_norm_rope(q, k, turns, pos),
                 lambda: vsd.vsd_norm_rope_append_kv(q, k, k, kc, kc, bt, pos, turns),
                 lambda: vsd.vsd_norm_rope_append_kv_quant(q, k, k, codes, codes, s, s, bt, pos, turns),
                 lambda: vsd.vsd_accumulate_weights(lg, q, kc, bt, pos, f, scale=1.0),
                 lambda: vsd.vsd_accumulate_weights_quant(lg, q, codes, s, bt, pos, f, scale=1.0),
                 lambda: vsd.vsd_compact_kv(kc, kc, bt, bt, pos, bt, pos),
                 lambda: vsd.vsd_compact_kv_quant(codes, codes, s, s, bt, bt, pos, bt, pos)):
        with pytest.raises(ValueError, match="CUDA"):            # host tensors
            call()
    for call in (lambda: vsd.vsd_norm_rope([0], k, turns, pos),
                 lambda: vsd.vsd_accumulate_weights(lg, q.float(), kc, bt, pos, f, scale=1.0),
                 lambda: vsd.vsd_norm_rope_append_kv_quant(q, k, k, codes, codes, s, None, bt, pos, turns),
                 lambda: vsd.vsd_accumulate_weights_quant(lg, q, codes, None, bt, pos, f, scale=1.0),
                 lambda: vsd.vsd_compact_kv_quant(codes, codes, None, s, bt, bt, pos, bt, pos)):
        with pytest.raises(TypeError):
            call()


# ------------------------------------------------------------------ the rotation's table
@pytest.mark.parametrize("rot", [8, 64, 128])
def test_turns_are_exact_for_far_positions(rot):
    """The table's product with a position, modulo 2^64, is the angle: within 2^-52 of a turn a
    position times the frequency's own rounding, for positions up to 2^31."""
    import sparse_attention_speculative_gb300 as vsd
    from tests.cache_life_ref import inv_freq
    f = inv_freq(rot)
    t = vsd.vsd_rope_turns(f, device="cpu")
    assert t.dtype == torch.int64 and t.shape == (rot // 2,)
    two_pi = Fraction("6.283185307179586476925286766559005768394338798750211641949889")
    for x, ft in zip(t.tolist(), f.tolist()):
        for pos in (1, 131071, 2 ** 31 - 1):
            have = Fraction((x * pos) % 2 ** 64, 2 ** 64)
            want = Fraction(ft) / two_pi * pos
            d = abs((have - want + Fraction(1, 2)) % 1 - Fraction(1, 2))
            # f / (2 pi) in 64 bits: pi's and the quotient's rounding, 2^-52 of the value; its last place 2^-64
            assert d <= pos * (Fraction(ft) / two_pi * Fraction(1, 2 ** 52) + Fraction(1, 2 ** 63))


def test_turns_of_other_frequencies():
    """Above a turn a position and below zero: the same angles."""
    import sparse_attention_speculative_gb300 as vsd
    f = torch.tensor([0.25, 7.0, -0.25, 0.0], dtype=torch.float64)
    t = [x % 2 ** 64 for x in vsd.vsd_rope_turns(f, device="cpu").tolist()]
    for x, ft in zip(t, f.tolist()):
        assert abs((x / 2.0 ** 64 - ft / (2 * math.pi) + 0.5) % 1 - 0.5) < 1e-15
    assert vsd.vsd_rope_turns([1.0], device="cpu").item() == vsd.vsd_rope_turns(torch.ones(1), device="cpu").item()
