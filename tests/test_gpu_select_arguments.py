"""What vsd_select_topk refuses of its tensors, by way of the extension module and without it.  The
library's call is a stand-in that launches nothing and says that it was reached."""
import ctypes

import pytest
import torch

import sparse_attention_speculative_gb300 as pkg
from sparse_attention_speculative_gb300 import _lib

pytestmark = pytest.mark.gpu
ROWS, HKV, P_MAX, K = 4, 2, 96, 40


@pytest.fixture(params=["module", "ctypes"])
def reached(request, monkeypatch):
    lib, calls = _lib.load(), []
    module = _lib._bound()
    P, I, SZ = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
    CALL = ctypes.CFUNCTYPE(I, I, I, P, P, I, I, I, I, P, P, P, P, SZ, P)
    call = CALL(lambda *a: calls.append(a) or 0)
    if request.param == "module":
        at = [ctypes.cast(f, ctypes.c_void_p).value for f in (
            lib.vsd_norm_rope, lib.vsd_norm_rope_append_kv, lib.vsd_norm_rope_append_kv_quant,
            lib.vsd_accumulate_weights, lib.vsd_accumulate_weights_quant, lib.vsd_compact_kv, lib.vsd_compact_kv_quant,
            call)]
        module.attach_more(*at)
    else:
        class Library:
            vsd_select_topk = staticmethod(call)
        monkeypatch.setattr(_lib, "_binding", None)
        monkeypatch.setattr(_lib, "_no_binding", True)
        monkeypatch.setattr(_lib, "load", lambda: Library)
    yield calls
    monkeypatch.undo()
    _lib._bound()          # (the library's own calls again)


def run(partial=None, prefix=None, **kw):
    partial = torch.zeros((ROWS, HKV, P_MAX), device="cuda") if partial is None else partial
    prefix = torch.full((ROWS,), P_MAX, dtype=torch.int32, device="cuda") if prefix is None else prefix
    return pkg.vsd_select_topk(partial, prefix, k=K, n_sink=1, n_recent=2, **kw)


def i32(*shape, device="cuda"):
    return torch.zeros(shape, dtype=torch.int32, device=device)


def test_what_is_taken(reached):
    idx, n, scores = run()
    assert idx.shape == (ROWS, K) and n.shape == (ROWS,) and scores is None
    assert run(want_scores=True)[2].shape == (ROWS, P_MAX)
    mine = dict(idx=i32(ROWS, K), n_sel=i32(ROWS), scores_out=torch.zeros((ROWS, P_MAX), device="cuda"))
    got = run(prefix=i32(2, ROWS // 2), **mine)                  # lengths [layers, sequences]
    assert all(a is b for a, b in zip(got, mine.values()))
    assert len(reached) == 3
    assert reached[-1][8:11] == tuple(t.data_ptr() for t in mine.values())


@pytest.mark.parametrize("what,kind", [
    (lambda: dict(prefix=i32(ROWS // HKV)), ValueError),             # a length a sequence, for rows of heads
    (lambda: dict(prefix=i32(ROWS + 1)), ValueError),
    (lambda: dict(prefix=i32(2 * ROWS)[::2]), ValueError),
    (lambda: dict(prefix=i32(ROWS, device="cpu")), ValueError),
    (lambda: dict(prefix=i32(ROWS).long()), TypeError),
    (lambda: dict(idx=i32(ROWS, K - 1)), ValueError),
    (lambda: dict(idx=i32(ROWS, K + 1)), ValueError),
    (lambda: dict(idx=i32(ROWS - 1, K)), ValueError),
    (lambda: dict(idx=i32(ROWS, 2 * K)[:, :K]), ValueError),
    (lambda: dict(idx=i32(ROWS, K, device="cpu")), ValueError),
    (lambda: dict(idx=i32(ROWS, K).long()), TypeError),
    (lambda: dict(n_sel=i32(1)), ValueError),
    (lambda: dict(n_sel=i32(ROWS, device="cpu")), ValueError),
    (lambda: dict(n_sel=torch.zeros(ROWS, device="cuda")), TypeError),
    (lambda: dict(scores_out=torch.zeros((ROWS, P_MAX - 1), device="cuda")), ValueError),
    (lambda: dict(scores_out=torch.zeros((ROWS, P_MAX))), ValueError),
    (lambda: dict(scores_out=torch.zeros((ROWS, P_MAX), device="cuda").double()), TypeError),
    (lambda: dict(partial=torch.zeros((ROWS, P_MAX), device="cuda")), ValueError),
    (lambda: dict(partial=torch.zeros((ROWS, HKV, 2 * P_MAX), device="cuda")[..., ::2]), ValueError),
    (lambda: dict(partial=torch.zeros((ROWS, HKV, P_MAX), device="cuda").half()), TypeError),
])
def test_what_is_refused(reached, what, kind):
    with pytest.raises(kind):
        run(**what())
    assert not reached
