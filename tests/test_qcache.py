"""Refusals of the 8-bit cache and of the sampled acceptance that need no GPU: host argument checks of the
library and of the binding."""
import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def sdv():
    from speculative_decoding_verify_02_gb300 import build
    build.build()
    import speculative_decoding_verify_02_gb300 as sdv
    return sdv


def _cfg(sdv, **kw):
    c = dict(n_layers=2, n_q_heads=8, n_kv_heads=2, head_dim=128, page_size=16, n_pages=8, scale_block=16, max_batch=2,
             max_rows=32, max_span=16, max_context=128)
    c.update(kw)
    return sdv.QCacheCfg(*c.values())


def _bytes(sdv, cfg):
    n = [ctypes.c_size_t() for _ in range(3)]
    r = sdv.lib().sdv_qcache_bytes(ctypes.byref(cfg) if cfg else None, *(ctypes.byref(x) for x in n))
    return r, [x.value for x in n]


def test_sizes(sdv):
    r, (codes, scales, ws) = _bytes(sdv, _cfg(sdv, scale_block=4))
    assert r == 0 and codes == 2 * 8 * 2 * 2 * 16 * 128 and scales == 2 * 8 * 2 * 2 * 4 * 4 and ws >= 256


@pytest.mark.parametrize("kw, code", [
    (dict(n_q_heads=7), "ARG"), (dict(n_kv_heads=0), "ARG"), (dict(scale_block=3), "ARG"), (dict(scale_block=32), "ARG"),
    (dict(page_size=0), "ARG"), (dict(n_pages=0), "ARG"), (dict(max_batch=257), "ARG"), (dict(max_span=33), "ARG"),
    (dict(max_context=15), "ARG"), (dict(head_dim=96), "UNSUPPORTED"), (dict(head_dim=256), "UNSUPPORTED"),
    (dict(n_layers=0), "ARG")])
def test_configuration_refusals(sdv, kw, code):
    assert _bytes(sdv, _cfg(sdv, **kw))[0] == getattr(sdv, "SDV_ERR_" + code)


def test_null_arguments(sdv):
    L, err = sdv.lib(), sdv.SDV_ERR_ARG
    assert _bytes(sdv, None)[0] == err
    assert L.sdv_qcache_bytes(ctypes.byref(_cfg(sdv)), None, None, None) == err
    out = ctypes.c_void_p()
    assert L.sdv_qcache_create(ctypes.byref(_cfg(sdv)), None, None, None, None, ctypes.byref(out)) == err
    assert L.sdv_qcache_write(None, 0, None, 0, None, 0, 0, 1, None, None, None, 1, 1, None) == err
    assert L.sdv_qcache_read(None, 0, None, None, None, 1, 1, None, 0, None, 0, 0, 1, None) == err
    assert L.sdv_qcache_attention(None, 0, None, 0, 0, 1, None, None, None, 1, 1, 0, None, 0, None) == err
    assert L.sdv_qcache_get_status(None, None) == err
    assert L.sdv_qcache_destroy(None) == 0
    assert L.sdv_accept_sampled(None, None, None, None, 0, None, None, None, 0, None, 0, 1, 1, 1, None, None, None, None,
                                None) == err


def test_binding_refuses_host_tensors_types_and_shapes(sdv):
    q = object.__new__(sdv.QuantCache)
    q._dim = 64
    q._dtypes = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
    for t in (torch.zeros(2, 2, 64, dtype=torch.bfloat16), torch.zeros(2, 2, 64, dtype=torch.float64),
              torch.zeros(2, 128, dtype=torch.bfloat16)):
        with pytest.raises(ValueError, match="k: a device tensor"):
            q._rows(t, 2, "k")
    with pytest.raises(ValueError, match="base"):
        sdv._vector(torch.zeros(2, dtype=torch.int64), 2, "base", torch.int32)
    with pytest.raises(ValueError, match="logits"):
        sdv._f32_rows(torch.zeros(2, 8), 2, 8, "logits")


def test_loop_refuses_uniforms_without_temperature(sdv):
    from speculative_decoding_verify_02_gb300.runner import SpecLoop
    loop = object.__new__(SpecLoop)
    loop.v, loop.B = None, 1
    with pytest.raises(ValueError, match="temperature"):
        loop.step(uniforms=torch.zeros(1))


class _Held:
    """What the binding looks at of a device tensor."""
    def __init__(self, *shape, dtype=torch.int32):
        self.shape, self.dtype, self.is_cuda, self.device = torch.Size(shape), dtype, True, "cuda:0"

    def numel(self):
        return self.shape.numel()

    def dim(self):
        return len(self.shape)

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 4096


def test_page_tables_of_another_width_are_refused(sdv, monkeypatch):
    """The kernels step from one sequence's pages to the next by the cache's own width: a wider table would give the
    second sequence pages of the first. One sequence's entries begin alike in a table of any width."""
    monkeypatch.setattr(sdv, "_many", False)
    q = object.__new__(sdv.QuantCache)
    q.pages_per_seq = 8
    off, base = _Held(3), _Held(2)
    for table in (_Held(2, 8), _Held(16), _Held(5, 8), _Held(1, 2, 8)):
        assert q._index(table, off, base, 2) == (4096, 4096, 4096)
    for table in (_Held(2, 9), _Held(4, 4), _Held(2, 16), _Held(2, 2, 16)):
        with pytest.raises(ValueError, match="page_table"):
            q._index(table, off, base, 2)
    assert q._index(_Held(1, 16), off, base, 1) == (4096, 4096, 4096)


def test_committed_rows_of_another_width_are_refused(sdv, monkeypatch):
    """accept_sampled writes row b at b * max_commit: a wider matrix would be filled across its rows."""
    import types
    calls = []
    monkeypatch.setattr(sdv, "_many", False)
    monkeypatch.setattr(sdv, "_stream", lambda s: 0)
    monkeypatch.setattr(sdv, "lib", lambda: types.SimpleNamespace(sdv_accept_sampled=lambda *a: calls.append(a) or 0))
    v = object.__new__(sdv.Verifier)
    v.ctx, v.mcfg, v.ccfg = None, types.SimpleNamespace(vocab=70), types.SimpleNamespace(max_rows=32)

    def matrix(rows):
        t = _Held(rows, 70, dtype=torch.float32)
        t.stride = lambda: (70, 1)
        return t

    def accept(B, max_commit, committed):
        f32 = torch.float32
        v.accept_sampled(_Held(12), _Held(B + 1), matrix(12), _Held(B, dtype=f32), _Held(12, dtype=f32), matrix(B), B,
                         max_commit, _Held(B), committed, _Held(B), _Held(B))

    for committed in (_Held(3, 4), _Held(12), _Held(4, 4)):
        accept(3, 4, committed)
    accept(1, 4, _Held(1, 17))
    assert len(calls) == 4
    for committed in (_Held(3, 5), _Held(3, 17), _Held(6, 2)):
        with pytest.raises(ValueError, match="committed"):
            accept(3, 4, committed)
    assert len(calls) == 4
    v.ctx = None


@pytest.mark.parametrize("kw", [dict(noise=1), dict(draft_probs=1), dict(noise=1, draft_probs=1),
                                dict(noise=1, temperature=1), dict(draft_probs=1, temperature=1)])
def test_loop_refuses_noise_and_draft_probs_without_uniforms(sdv, kw):
    """They belong to the acceptance against probabilities; without uniforms the loop matches tokens, another law."""
    from speculative_decoding_verify_02_gb300.runner import SpecLoop
    loop = object.__new__(SpecLoop)
    loop.v, loop.B = None, 1
    with pytest.raises(ValueError, match="uniforms"):
        loop.step(**{k: torch.zeros(1) for k in kw})
