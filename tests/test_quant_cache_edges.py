"""What the 8-bit cache's calls refuse on the host, beside test_quant_cache_refusals.py, and
how their extension module is built."""
import os
import types

import pytest

from tests.test_quant_cache_refusals import geom, lib, off, p  # noqa: F401


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
