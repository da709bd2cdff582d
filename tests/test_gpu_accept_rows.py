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
