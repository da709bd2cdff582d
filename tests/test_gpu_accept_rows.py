"""Sampled acceptance where a row leaves nothing to draw from, at vocabularies that end inside and at the end of a
chunk of 4,096 logits."""
import numpy as np
import pytest

from tests.test_gpu_accept_sampled import _forward, _inputs, _lengths, _ref, _run, _verifier

pytestmark = pytest.mark.gpu


def _nan(row):
    row[:] = np.nan


def _minus_inf(row):
    row[:] = -np.inf


def _nan_first(row):
    row[:] = -np.inf
    row[0] = np.nan


def _nan_but_one(row):
    row[:] = np.nan
    row[len(row) // 2] = -np.inf


@pytest.mark.parametrize("kind", [_nan, _minus_inf, _nan_first, _nan_but_one])
@pytest.mark.parametrize("probs", [False, True])
@pytest.mark.parametrize("V", [1, 2, 1500, 4096, 4097, 5000, 151936])
def test_row_without_a_logit_commits_token_zero(V, probs, kind):
    """The first row of a span with the draft 0 and with another, its last row, and the row after an accepted draft, at
    temperatures above zero and at zero: the draft is refused, token 0 is committed and the status says so."""
    rng = np.random.default_rng(V)
    spans = [3, 3, 1, 3, 2]
    off = np.concatenate([[0], np.cumsum(spans)])
    v = _verifier(V, len(spans), 3)
    _forward(v, spans)
    x = _inputs(rng, spans, V, probs, [1.0, 0.7, 1.3, 0.5, 0.0])
    rows = [off[0], off[1], off[2], off[3] + 1, off[4]]
    x["tokens"][off[0] + 1] = 0
    x["tokens"][off[1] + 1] = V - 1
    d = x["tokens"][off[3] + 1]
    x["u"][off[3]] = 0.0                                              # accepted whatever its probability is
    assert x["logits"][off[3], d] > -np.inf
    x["tokens"][off[3] + 2] = 0
    for r in rows:
        kind(x["logits"][r])
    got, ref = _run(v, x), _ref(x, _lengths(v, len(spans)))
    assert v.get_status() == -4
    for g, r in zip(got, ref):
        np.testing.assert_array_equal(g, r)
    assert got[0].tolist() == [0, 0, 0, 1, 0]
    assert [int(got[1][b, m]) for b, m in enumerate(got[0])] == [0] * 5
    v.close()


@pytest.mark.parametrize("V, probs, spread", [(151936, False, 0.5), (151936, True, 0.5), (151936, True, 6.0), (9001, False, 1.0)])
def test_draws_next_to_the_border(V, probs, spread):
    """Uniforms 2^-23 of the draft's p / q below and above it, in rows whose sum is carried by their whole vocabulary. A
    float32 sum of such a row is off by about as much: the decision has to be made in 64 bits. (A uniform is within
    2^-24 of the number it is rounded from, so each lies at least 2^-24 from the border.)"""
    rng = np.random.default_rng(V + int(10 * spread))
    B = 64
    spans = [2] * B
    v = _verifier(V, B, 2)
    _forward(v, spans)
    logits = rng.uniform(-spread, spread, (2 * B, V)).astype(np.float32)
    temps = rng.uniform(0.6, 1.5, B).astype(np.float32)
    tokens = np.zeros(2 * B, dtype=np.int64)
    u = np.zeros(2 * B, dtype=np.float32)
    q = np.full((2 * B, V), 1.0 / V, dtype=np.float32) if probs else None
    above = np.arange(B) % 2 == 1
    for b in range(B):
        x = logits[2 * b].astype(np.float64)
        w = np.exp((x - x.max()) / float(temps[b]))
        p = w / w.sum()
        d = int(rng.integers(V))
        tokens[2 * b + 1] = d
        if probs:
            q[2 * b, d] = np.float32(p[d] * rng.uniform(1.1, 4.0))
        border = p[d] / (float(q[2 * b, d]) if probs else 1.0)
        u[2 * b] = border * (1 + (2.0 ** -23 if above[b] else -2.0 ** -23))
        assert u[2 * b] < 1 and abs(u[2 * b] / border - 1) >= 2.0 ** -24
    x = dict(spans=spans, V=V, logits=logits, probs=q, tokens=tokens, u=u, temps=temps,
             noise=rng.exponential(size=(B, V)).astype(np.float32))
    got = _run(v, x)
    np.testing.assert_array_equal(got[0], np.where(above, 0, 1))
    for g, r in zip(got, _ref(x, _lengths(v, B))):
        np.testing.assert_array_equal(g, r)
    assert v.get_status() == 0
    v.close()
