"""Pins of the oracle for continuations of one prompt: hand-worked pools and cuts, attention against torch in float64, the law
of the draw."""
import numpy as np
import pytest

import oracle


def test_fork_shares_whole_pages_and_copies_the_partial_one():
    p = oracle.SharedPool(8, 4, 4, 4)
    p.ensure_capacity([10])
    p.set_length(0, 10)
    assert p.fork([0, 0], [1, 3]) == [(2, 3, 2), (2, 4, 2)]
    assert p.table == [[0, 1, 2], [0, 1, 3], [], [0, 1, 4]] and p.length == [10, 10, 0, 10]
    p.rewind([-1, 8, -1, -1])              # page 3 goes back, the shared ones stay
    assert p.free == [7, 6, 5, 3]
    with pytest.raises(ValueError):
        p.rewind([-1, 6])                  # into page 1, which 0 and 3 hold
    p.rewind([0, 0, -1, 0])                # 3 lets go first, 0 gives the pages back
    assert p.free == [7, 6, 5, 3, 4, 2, 1, 0] and p.table == [[]] * 4


def test_fork_is_all_or_nothing():
    p = oracle.SharedPool(3, 4, 4, 4)
    p.ensure_capacity([6])
    p.set_length(0, 6)
    with pytest.raises(oracle.CapacityError):
        p.fork([0, 0], [1, 2])
    for src, dst in (([0], [0]), ([0, 0], [1, 1]), ([1], [0])):
        with pytest.raises(ValueError):
            p.fork(src, dst)
    assert p.table == [[0, 1], [], [], []] and p.free == [2]


@pytest.mark.parametrize("window, cap, slope", [(0, 0.0, 0.0), (3, 0.0, 0.0), (0, 2.0, 0.0), (5, 1.0, 0.25)])
def test_attention_against_torch(window, cap, slope):
    import torch
    rng = np.random.default_rng(0)
    q, k, v = rng.normal(size=(4, 8)), rng.normal(size=(9, 8)), rng.normal(size=(9, 8))
    pos = np.array([0, 3, 7, 8])
    z = torch.from_numpy(q) @ torch.from_numpy(k).T / 8 ** 0.5
    if cap:
        z = cap * torch.tanh(z / cap)
    t, p = torch.arange(9)[None], torch.from_numpy(pos)[:, None]
    z = z - slope * (p - t)
    hidden = (t > p) | ((t <= p - window) if window else False)
    ref = torch.softmax(z.masked_fill(hidden, -torch.inf), -1) @ torch.from_numpy(v)
    np.testing.assert_allclose(oracle.attend(oracle.scores(q, k, pos, window, cap, slope), v), ref.numpy(), rtol=1e-12)


def test_unseen_keys_do_not_count_whatever_they_hold():
    q, k, v = np.ones((1, 2)), np.ones((3, 2)), np.ones((3, 2))
    k[2], v[2] = np.nan, np.inf
    np.testing.assert_array_equal(oracle.attend(oracle.scores(q, k, [1]), v), [[1.0, 1.0]])


LOGITS = np.log([0.1, 0.4, 0.1, 0.3, 0.1])


@pytest.mark.parametrize("kw, kept", [
    (dict(), [1, 3, 0, 2, 4]), (dict(top_k=3), [1, 3, 0]), (dict(top_k=1), [1]), (dict(top_k=9), [1, 3, 0, 2, 4]),
    (dict(top_p=0.3), [1]), (dict(top_p=0.5), [1, 3]), (dict(top_p=0.75), [1, 3, 0]), (dict(top_p=0.0), [1]),
    (dict(top_k=2, top_p=0.5), [1]),       # of the two's weight, 0.7
    (dict(min_p=0.5), [1, 3]), (dict(min_p=1.0), [1]), (dict(min_p=2.0), [1]), (dict(top_p=0.95, min_p=0.7), [1, 3])])
def test_cuts(kw, kept):
    assert oracle.kept_tokens(LOGITS, 1.0, **kw)[0].tolist() == kept


def test_cuts_of_odd_rows():
    inf = np.inf
    assert oracle.kept_tokens(np.array([2.0, -inf, np.nan, 2.0, 1.0]), 1.0, top_k=2)[0].tolist() == [0, 3]
    assert oracle.kept_tokens(np.array([1.0, 5.0, 5.0]), 0.0)[0].tolist() == [1]
    assert len(oracle.kept_tokens(np.array([-inf, np.nan]), 1.0)[0]) == 0
    assert oracle.kept_tokens(np.array([inf, 3.0, inf]), 1.0, top_p=0.9)[0].tolist() == [0, 2]
    assert oracle.kept_tokens(np.array([-0.0, 0.0]), 1.0, top_k=1)[0].tolist() == [0]


def test_draws_follow_the_weights():
    rng = np.random.default_rng(3)
    tokens, w = oracle.kept_tokens(LOGITS, 1.0, top_p=0.85)
    n = 20000
    counts = np.bincount([oracle.draw_kept(tokens, w, rng.exponential(size=5)) for _ in range(n)], minlength=5)
    p = np.zeros(5)
    p[tokens] = w / w.sum()
    assert (np.abs(counts / n - p) <= 5 * np.sqrt(p * (1 - p) / n)).all()  # five standard deviations
