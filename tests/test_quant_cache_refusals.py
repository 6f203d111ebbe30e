"""What the 8-bit cache's calls refuse on the host, and the pins of their reference."""
import ctypes
import math

import pytest
import torch

from tests import quant_ref as ref


@pytest.fixture(scope="module")
def lib():
    from sparse_attention_speculative_gb300 import build
    from sparse_attention_speculative_gb300._lib import load
    build.build()
    return load()


def geom(**kw):
    from sparse_attention_speculative_gb300._lib import Geom
    base = dict(B=1, Hq=32, Hkv=8, head_dim=128, page_size=16, max_blocks_per_seq=64, num_blocks=64)
    base.update(kw)
    return ctypes.byref(Geom(**base))


@pytest.fixture()
def p():
    buf = ctypes.create_string_buffer(8192)
    yield ctypes.c_void_p((ctypes.addressof(buf) + 255) & ~255)


def off(p, n):
    return ctypes.c_void_p(p.value + n)


GEOMETRIES = [(dict(Hq=30), -1), (dict(head_dim=96), -2), (dict(page_size=32), -2), (dict(Hq=24), -2),
              (dict(num_blocks=0), -1), (dict(B=-1), -1)]


def append(lib, g, p, n=4, **kw):
    a = dict(k=p, v=p, bt=p, pos=p, nv=None, kc=p, vc=p, ks=p, vs=p)
    a.update(kw)
    return lib.vsd_append_kv_quant(g, n, a["k"], a["v"], a["bt"], a["pos"], 0, a["nv"], a["kc"], a["vc"], a["ks"],
                                   a["vs"], None)


def read(lib, g, p, n=4, **kw):
    a = dict(k=p, v=p, bt=p, pos=p, nv=None, kc=p, vc=p, ks=p, vs=p)
    a.update(kw)
    return lib.vsd_read_kv_quant(g, n, a["kc"], a["vc"], a["ks"], a["vs"], a["bt"], a["pos"], 0, a["nv"], a["k"],
                                 a["v"], None)


def verify(lib, g, p, R=4, P_max=512, row0=0, row1=3, scale=0.1, ws=None, wsb=0, **kw):
    a = dict(q=p, kc=p, vc=p, ks=p, vs=p, bt=p, pl=p, lg=p, ps=p, sc=None, hist=None, out=p, sink=0, recent=0)
    a.update(kw)
    return lib.vsd_verify_attn_collect_quant(g, R, a["q"], a["kc"], a["vc"], a["ks"], a["vs"], a["bt"], a["pl"],
                                             row0, row1, P_max, ctypes.c_float(scale), a["lg"], a["ps"], a["sc"],
                                             a["hist"], a["sink"], a["recent"], a["out"], ws, wsb, None)


def draft(lib, g, p, k_max=16, max_tail=4, scale=0.1, ws=None, wsb=0, **kw):
    a = dict(q=p, kc=p, vc=p, ks=p, vs=p, bt=p, idx=p, ns=p, t0=p, t1=p, out=p)
    a.update(kw)
    return lib.vsd_sparse_decode_attn_quant(g, a["q"], a["kc"], a["vc"], a["ks"], a["vs"], a["bt"], a["idx"],
                                            a["ns"], k_max, a["t0"], a["t1"], max_tail, ctypes.c_float(scale),
                                            a["out"], ws, wsb, None)


@pytest.mark.parametrize("call", [append, read, verify, draft])
@pytest.mark.parametrize("kw,code", GEOMETRIES)
def test_geometry(lib, p, call, kw, code):
    assert call(lib, geom(**kw), p) == code
    assert call(lib, None, p) == -1


@pytest.mark.parametrize("call", [append, read])
def test_row_calls(lib, p, call):
    for name in ("k", "v", "bt", "pos", "kc", "vc", "ks", "vs"):
        assert call(lib, geom(), p, **{name: None}) == -1
    for name in ("k", "v", "kc", "vc"):
        assert call(lib, geom(), p, **{name: off(p, 8)}) == -1
    for name in ("bt", "pos", "nv", "ks", "vs"):
        assert call(lib, geom(), p, **{name: off(p, 2)}) == -1
    assert call(lib, geom(), p, n=-1) == -1
    assert call(lib, geom(B=2 ** 20), p, n=2 ** 20) == -2   # more parts than 32 bits count
    assert call(lib, geom(), p, n=0, k=None) == 0        # nothing to do: no device needed
    assert call(lib, geom(B=0), p, k=None) == 0


def test_verify_call(lib, p):
    for name in ("q", "kc", "vc", "ks", "vs", "bt", "pl", "out"):
        assert verify(lib, geom(), p, **{name: None}) == -1
    for name in ("q", "kc", "vc", "lg", "ps", "out"):
        assert verify(lib, geom(), p, **{name: off(p, 8)}) == -1
    assert verify(lib, geom(), p, ks=off(p, 2)) == -1
    assert verify(lib, geom(), p, R=0) == -1
    assert verify(lib, geom(), p, R=17) == -2
    assert verify(lib, geom(Hq=128), p, R=5) == -2       # R * G = 80
    assert verify(lib, geom(Hq=256), p, R=1) == -2       # G = 32
    assert verify(lib, geom(), p, P_max=-1) == -1
    assert verify(lib, geom(), p, P_max=2 ** 31 - 1) == -2
    assert verify(lib, geom(), p, row0=4) == -1
    assert verify(lib, geom(), p, row1=-1) == -1
    assert verify(lib, geom(), p, scale=math.inf) == -1
    assert verify(lib, geom(), p, sc=p) == -1            # a score without its histogram
    assert verify(lib, geom(), p, sc=p, hist=p, ps=None) == -1
    assert verify(lib, geom(), p, sink=-1) == -1
    assert verify(lib, geom(B=0), p, q=None) == 0


def test_draft_call(lib, p):
    for name in ("q", "kc", "vc", "ks", "vs", "bt", "idx", "ns", "t0", "t1", "out"):
        assert draft(lib, geom(), p, **{name: None}) == -1
    for name in ("q", "kc", "vc", "out"):
        assert draft(lib, geom(), p, **{name: off(p, 8)}) == -1
    assert draft(lib, geom(Hq=256), p) == -2
    assert draft(lib, geom(B=65536), p) == -2
    assert draft(lib, geom(num_blocks=2 ** 30), p) == -2  # cache rows past 2^31
    assert draft(lib, geom(), p, k_max=-1) == -1
    assert draft(lib, geom(), p, max_tail=-1) == -1
    assert draft(lib, geom(), p, k_max=2 ** 30, max_tail=2 ** 30) == -2
    assert draft(lib, geom(), p, scale=math.nan) == -1
    assert draft(lib, geom(B=0), p, q=None) == 0


def test_binding_refuses_wrong_tensors():
    import sparse_attention_speculative_gb300 as vsd
    NB, Hkv, d, B = 4, 2, 64, 1
    rows = torch.zeros((B, 3, Hkv, d), dtype=torch.bfloat16)
    kc = torch.zeros((NB, Hkv, 16, d), dtype=torch.uint8).view(torch.float8_e4m3fn)
    s = torch.ones((NB, Hkv))
    bt = torch.zeros((B, 4), dtype=torch.int32)
    pos = torch.zeros((B,), dtype=torch.int32)
    with pytest.raises(TypeError):                      # fp32 rows
        vsd.vsd_append_kv_quant(rows.float(), rows, kc, kc, s, s, bt, pos)
    with pytest.raises(ValueError):                     # host tensors
        vsd.vsd_append_kv_quant(rows, rows, kc, kc, s, s, bt, pos)
    with pytest.raises((TypeError, ValueError)):
        vsd.vsd_read_kv_quant(kc, kc, s, s, bt, pos, n=3)
    with pytest.raises((TypeError, ValueError)):
        vsd.vsd_verify_attn_collect_quant(rows, kc, kc, s, s, bt, pos, P_max=8, scale=1.0)
    with pytest.raises((TypeError, ValueError)):
        vsd.vsd_sparse_decode_attn_quant(rows[:, 0], kc, kc, s, s, bt, None, None, pos, pos, scale=1.0, max_tail=1)


# ------------------------------------------------------------------ the reference itself
def test_reference_encoding_inverts_decoding():
    codes = torch.arange(256, dtype=torch.uint8)
    real = (codes & 0x7F) != 0x7F
    back = ref.encode(ref.decode(codes))
    assert torch.equal(back[real], codes[real]) and torch.all(back[~real] == ref.NAN_CODE)


def test_reference_encoding_agrees_with_torch():
    """torch's own conversion (on the CPU) rounds alike, for values within the range."""
    g = torch.Generator().manual_seed(0)
    x = torch.cat([torch.randn(20000, generator=g) * 100, torch.randn(20000, generator=g) * 0.01,
                   torch.arange(-448, 449).float(), torch.arange(0, 1024).float() * 2.0 ** -11]).clamp(-448, 448)
    assert torch.equal(ref.encode(x.double()), x.to(torch.float8_e4m3fn).view(torch.uint8))


@pytest.mark.parametrize("amax,want", [(0.0, 2.0 ** -126), (448.0, 1.0), (448.5, 2.0), (224.0, 0.5), (1.75, 2.0 ** -8),
                                       (1.7578125, 2.0 ** -7), (3.3895313892515355e38, 2.0 ** 120), (2.0 ** -133, 2.0 ** -126)])
def test_reference_scale(amax, want):
    assert ref.page_scale(amax) == want


def test_reference_append_by_hand():
    """Two rows, then a louder one: the first two are requantised, the scale doubles."""
    codes = torch.zeros((1, 1, 16, 64), dtype=torch.uint8)
    scales = torch.full((1, 1), math.nan)
    x = torch.zeros((1, 2, 1, 64), dtype=torch.float64)
    x[0, 0, 0, 0], x[0, 1, 0, 1] = 448.0, -3.0
    ref.append(codes, scales, x, torch.zeros((1, 1), dtype=torch.int32), [0], [2])
    assert scales.item() == 1.0
    assert ref.decode(codes[0, 0, 0, 0]) == 448 and ref.decode(codes[0, 0, 1, 1]) == -3
    ref.append(codes, scales, x[:, :1] * 2, torch.zeros((1, 1), dtype=torch.int32), [2], [1])
    assert scales.item() == 2.0
    assert [float(ref.decode(codes[0, 0, r, c])) for r, c in ((0, 0), (1, 1), (2, 0))] == [224.0, -1.5, 448.0]
