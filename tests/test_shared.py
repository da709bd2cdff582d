"""Refusals of the shared-prefix attention, of forks and of the filtered sampling that need no GPU: host argument checks of the
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
    c = dict(n_layers=2, n_q_heads=8, n_kv_heads=2, head_dim=128, page_size=16, n_pages=8, dtype=0, max_batch=2, max_rows=32,
             max_span=16, max_context=128)
    c.update(kw)
    return sdv.SharedCfg(*c.values())


def _bytes(sdv, cfg):
    n = [ctypes.c_size_t() for _ in range(2)]
    r = sdv.lib().sdv_shared_bytes(ctypes.byref(cfg) if cfg else None, *(ctypes.byref(x) for x in n))
    return r, [x.value for x in n]


def test_sizes(sdv):
    r, (pool, ws) = _bytes(sdv, _cfg(sdv))
    assert r == 0 and pool == 2 * 8 * 2 * 2 * 16 * 128 * 2
    # a row's parts: of its own keys and of the prefix's
    assert ws >= 2 * 32 * 8 * (128 + 2) * 4


@pytest.mark.parametrize("kw, code", [
    (dict(n_q_heads=7), "ARG"), (dict(n_kv_heads=0), "ARG"), (dict(page_size=0), "ARG"), (dict(n_pages=0), "ARG"),
    (dict(max_batch=257), "ARG"), (dict(max_span=33), "ARG"), (dict(max_context=15), "ARG"), (dict(n_layers=0), "ARG"),
    (dict(head_dim=96), "UNSUPPORTED"), (dict(head_dim=256), "UNSUPPORTED"), (dict(dtype=2), "UNSUPPORTED"),
    (dict(max_rows=65537), "UNSUPPORTED"), (dict(page_size=1 << 20, n_pages=1 << 12), "UNSUPPORTED"),
    (dict(max_context=1 << 30, max_batch=256, n_kv_heads=8), "UNSUPPORTED")])
def test_configuration_refusals(sdv, kw, code):
    cfg = _cfg(sdv, **kw)
    want = getattr(sdv, "SDV_ERR_" + code)
    assert _bytes(sdv, cfg)[0] == want
    out = ctypes.c_void_p()
    assert sdv.lib().sdv_shared_create(ctypes.byref(cfg), 256, 256, None, ctypes.byref(out)) == want and not out.value


def test_null_and_misaligned_arguments(sdv):
    L, cfg, out = sdv.lib(), _cfg(sdv), ctypes.c_void_p()
    assert _bytes(sdv, None)[0] == sdv.SDV_ERR_ARG
    for pool, ws in ((0, 256), (256, 0), (257, 256), (256, 272)):
        assert L.sdv_shared_create(ctypes.byref(cfg), pool, ws, None, ctypes.byref(out)) == sdv.SDV_ERR_ARG
    assert L.sdv_shared_attention(None, 0, 256, 1024, 1, 256, 256, 256, 1, 0, 0, 0, 1, 0, 0.0, 0, 256, 1024, None) == sdv.SDV_ERR_ARG
    assert L.sdv_shared_get_status(None, ctypes.byref(ctypes.c_int32())) == sdv.SDV_ERR_ARG
    assert L.sdv_shared_destroy(None) == sdv.SDV_OK
    assert L.sdv_fork_seq(None, 256, 256, 1, None) == sdv.SDV_ERR_ARG
    assert L.sdv_filter_logits(None, 256, 8, 1, 256, 1, 256, 0, 0, 0, 256, 8, 0, None) == sdv.SDV_ERR_ARG
    assert L.sdv_sample(None, 256, 8, 1, 256, 256, 8, 1, 256, 0, 0, 0, 256, 0, None) == sdv.SDV_ERR_ARG


def test_types_are_checked_before_any_call(sdv):
    with pytest.raises(ValueError, match="dtype"):
        sdv.SharedAttention(1, 8, 2, 128, dtype=torch.float32)


def test_a_prompt_to_share_has_tokens(sdv):
    from speculative_decoding_verify_02_gb300.runner import SpecLoop
    loop = SpecLoop.__new__(SpecLoop)
    loop.v, loop.B = None, 4
    with pytest.raises(ValueError, match="empty"):
        loop.prefill_shared([])


def test_a_step_with_cuts_needs_uniforms(sdv):
    from speculative_decoding_verify_02_gb300.runner import SpecLoop
    loop = SpecLoop.__new__(SpecLoop)
    loop.v, loop.B = None, 1
    for kw in (dict(top_k=1), dict(top_p=1), dict(min_p=1)):
        with pytest.raises(ValueError, match="uniforms"):
            loop.step(**kw)


def test_a_drawn_first_token_needs_noise(sdv):
    from speculative_decoding_verify_02_gb300.runner import SpecLoop
    loop = SpecLoop.__new__(SpecLoop)
    loop.v, loop.B = None, 4
    for kw in (dict(temperature=1), dict(top_k=1), dict(top_p=1), dict(min_p=1), dict(temperature=1, top_p=1), dict(noise=1),
               dict(noise=1, top_k=1)):
        with pytest.raises(ValueError, match="temperature and noise"):
            loop.prefill_shared([1, 2], chunk=1, **kw)


def test_a_step_with_cuts_leaves_the_callers_logits(sdv):
    """The model's logits stay in the caller's tensor; the filter writes, and the acceptance reads, another one, the same for the
    same shape. Without a tensor of the caller's the filter works in place."""
    from speculative_decoding_verify_02_gb300.runner import SpecLoop
    calls = {}

    class Fake:
        mcfg = sdv.ModelCfg(vocab=6)

        def __getattr__(self, name):
            return lambda *a, **kw: calls.setdefault(name, []).append(a)

    loop = SpecLoop.__new__(SpecLoop)
    loop.v, loop.B, loop.max_rows, loop.max_span, loop.logits, loop.cut_logits = Fake(), 2, 4, 2, torch.zeros(4, 6), {}
    for name in ("tokens", "row_off", "required", "argmax", "n_accept", "committed", "n_commit", "new_len"):
        setattr(loop, name, None)
    kw = dict(temperature=1, uniforms=1, noise=1, top_k=1)
    mine, other = torch.zeros(4, 6), torch.zeros(5, 6)
    for t in (mine, mine, other, None):
        loop.step(logits=t, **kw)
    loop.step(logits=mine, temperature=1, uniforms=1, noise=1)
    model, (src, out), read = [c[-1] for c in calls["spec_forward"]], zip(*((c[0], c[3]) for c in calls["filter_logits"])), \
        [c[2] for c in calls["accept_sampled"]]
    assert model[0] is mine and model[2] is other and model[3] is loop.logits and model[4] is mine
    assert all(a is b for a, b in zip(src, model)) and all(a is b for a, b in zip(read, out)) and read[4] is mine
    assert out[0] is not mine and out[0].shape == mine.shape and out[1] is out[0] and out[2].shape == other.shape and out[3] is loop.logits
