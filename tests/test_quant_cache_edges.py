"""What the 8-bit cache's calls refuse on the host, beside test_quant_cache_refusals.py, and
how their extension module is built."""
import ctypes
import os
import types

import pytest

from sparse_attention_speculative_gb300._lib import Geom
from tests.test_quant_cache_refusals import geom, lib, off, p, verify  # noqa: F401


def test_zeroed_read_call(lib, p):  # noqa: F811
    def call(g, n=4, zeroed=3, **kw):
        a = dict(k=p, v=p, bt=p, pos=p, nv=None, kc=p, vc=p, ks=p, vs=p)
        a.update(kw)
        return lib.vsd_read_kv_quant_zeroed(g, n, a["kc"], a["vc"], a["ks"], a["vs"], a["bt"], a["pos"], 0, a["nv"],
                                            a["k"], a["v"], zeroed, None)
    assert call(geom(B=0)) == 0 and call(geom(), n=0) == 0
    assert call(geom(B=0), zeroed=4) == -1
    assert call(geom(), n=-1) == -1
    for name in ("k", "v", "kc", "vc"):
        assert call(geom(), **{name: None}) == -1
        assert call(geom(), **{name: off(p, 8)}) == -1


@pytest.mark.parametrize("kw,P_max,code", [
    (dict(B=2 ** 16, Hkv=2 ** 16, Hq=2 ** 16), 0, -2),      # 2^32 pairs: none in 32 bits
    (dict(B=2 ** 20, Hkv=2 ** 12, Hq=2 ** 12), 1000, -2),
    (dict(B=2 ** 15, Hkv=2 ** 14, Hq=2 ** 14), 16, -2),     # 2^29 pairs of 10 tiles and more
    (dict(B=1, Hkv=8, Hq=32), 2 ** 30 + 1, -2),
    (dict(B=256, Hkv=1, Hq=1), 2 ** 30, -2),
])
def test_verifications_that_32_bits_do_not_count(lib, p, kw, P_max, code):  # noqa: F811
    size = ctypes.c_size_t(0)
    assert lib.vsd_verify_quant_workspace_size(geom(**kw), 1, P_max, ctypes.byref(size)) == code
    assert verify(lib, geom(**kw), p, R=1, P_max=P_max, row1=0) == code


def test_scored_verifications_of_too_many_sequences(lib, p):  # noqa: F811
    """4096 bins for each of 2^19 sequences are more than the kernels number."""
    many = dict(B=2 ** 19, Hkv=1, Hq=1)
    assert verify(lib, geom(**many), p, P_max=16, sc=p, hist=p) == -2
    assert lib.vsd_verify_attn_collect_scored(ctypes.cast(geom(**many), ctypes.POINTER(Geom)), 1, p, p, p, p, p, 0, 0,
                                              16, 0.1, None, p, p, p, 0, 0, 0, None, None, p, None, 0, None) == -2


# ------------------------------------------------------------------ the extension module
@pytest.fixture()
def builder(lib, monkeypatch):  # noqa: F811
    """build.py with everything built, and compilers that fail the test."""
    from sparse_attention_speculative_gb300 import build
    assert build.up_to_date()

    def no(*a, **k):
        raise AssertionError("compiled something")
    monkeypatch.setattr(build, "nvcc", no)
    return build


def test_the_library_does_not_need_the_module(builder, monkeypatch, tmp_path):
    """Where the module cannot be built the library is built and returned all the same."""
    monkeypatch.setattr(builder, "BINDING", str(tmp_path / "_binding.so"))

    def fails():
        raise RuntimeError("no such header")
    monkeypatch.setattr(builder, "build_binding", fails)
    assert builder.library_up_to_date() and not builder.up_to_date()
    with pytest.warns(RuntimeWarning, match="no such header"):
        assert builder.build() == builder.LIB


def test_the_library_is_linked_where_the_module_fails(builder, monkeypatch, tmp_path):
    """The same where the library is compiled too: it is linked before the module's error
    counts."""
    monkeypatch.setattr(builder, "LIB", str(tmp_path / "libvsd.so"))
    monkeypatch.setattr(builder, "BINDING", str(tmp_path / "_binding.so"))
    monkeypatch.setattr(builder, "BUILD", str(tmp_path / "obj"))
    monkeypatch.setattr(builder, "nvcc", lambda: "nvcc")
    monkeypatch.setattr(builder, "build_binding", lambda: 1 // 0)

    def run(cmd, **kw):
        with open(cmd[cmd.index("-o") + 1], "w"):
            return types.SimpleNamespace(returncode=0, stderr="", stdout="")
    monkeypatch.setattr(builder.subprocess, "run", run)
    with pytest.warns(RuntimeWarning, match="division"):
        assert builder.build() == builder.LIB
    assert os.path.exists(builder.LIB)


def test_the_module_is_built_again_for_another_torch(builder, monkeypatch):
    import torch
    built = []
    monkeypatch.setattr(builder, "build_binding", lambda: built.append(1))
    assert builder.build() == builder.LIB and not built
    monkeypatch.setattr(torch, "__version__", "0.0.1")
    assert builder.library_up_to_date() and not builder.binding_up_to_date()
    assert builder.build() == builder.LIB and built == [1]


def test_a_module_built_for_another_torch_is_refused(builder, monkeypatch):
    import torch
    from sparse_attention_speculative_gb300 import _lib
    _lib._bound()
    monkeypatch.setattr(torch, "__version__", "0.0.1")
    with pytest.raises(RuntimeError, match="0.0.1"):
        _lib._bound()
