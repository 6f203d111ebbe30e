"""What the 8-bit cache's calls refuse on the host, beside test_quant_cache_refusals.py."""
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
