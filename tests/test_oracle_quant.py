"""Pins of the 8-bit cache and sampled acceptance oracle: hand-worked values, torch's e4m3 type, dense
attention in torch float64, and the acceptance rule's own law (the committed token is the target's)."""
import math

import numpy as np
import pytest

import oracle
import synth


def test_e4m3_values_and_rounding():
    import torch
    codes = np.arange(256, dtype=np.uint8)
    ref = torch.from_numpy(codes).view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(oracle.code_values(codes), ref)
    x = np.concatenate([np.linspace(-460, 460, 4001), np.linspace(-0.02, 0.02, 4001), ref[np.isfinite(ref)]])
    x = np.clip(x, -448, 448).astype(np.float32)
    ref = torch.from_numpy(x).to(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(oracle.e4m3(x), ref)
    # hand-worked: ties go to even, a subnormal step is 2^-9, clamping and NaN as a write stores them
    assert oracle.e4m3(1.0625) == 1.0 and oracle.e4m3(1.1875) == 1.25
    assert oracle.e4m3(2.0 ** -10) == 0.0 and oracle.e4m3(3 * 2.0 ** -10) == 2.0 ** -8
    assert oracle.e4m3(np.inf) == 448 and oracle.e4m3(-1e9) == -448 and oracle.e4m3(np.nan) == 0


@pytest.mark.parametrize("amax, exp", [(448.0, 0), (448.5, 1), (1.0, -8), (0.875, -9), (0.8750001, -8), (1e38, 118),
                                       (0.0, -126), (1e-42, -126)])
def test_needed_scale(amax, exp):
    assert oracle.needed_scale(amax) == 2.0 ** exp


def test_scale_growth_rounds_live_rows_once_more():
    """One head, D = 2 (any): 1.125 at scale 2^-8 is 288 = code 288 exactly; a later row of 600 needs
    2; the live row becomes e4m3(1.125 / 2) = 0.5625 exactly, and 2^-9-sized ones round away."""
    pool = oracle.QuantPool(1, 1, 4, 2, 4)
    pool.write([0], 0, np.array([[[1.125, 0.001]]]), np.array([[[1.0, 1.0]]]))
    assert pool.scale[0, 0, 0, 0] == 2.0 ** -8 and pool.val[0, 0, 0, 0, 0] == 288
    pool.write([0], 1, np.array([[[600.0, 0.0]]]), np.array([[[1.0, 1.0]]]))
    assert pool.scale[0, 0, 0, 0] == 2.0 and pool.scale[0, 1, 0, 0] == 2.0 ** -8
    np.testing.assert_array_equal(pool.val[0, 0, 0, :2], [[0.5625, 0.0], [288.0, 0.0]])  # 300 lies between 288 and 320


def test_attention_matches_dense_softmax():
    import torch
    rng = np.random.default_rng(3)
    pool = oracle.QuantPool(6, 2, 8, 16, 4)
    pages = [4, 1, 5, 0]
    pool.write(pages, 0, rng.normal(size=(29, 2, 16)), rng.normal(size=(29, 2, 16)))
    q = rng.normal(size=(5, 4, 16))
    for window in (0, 7):
        o, mag, _ = pool.attention(pages, 24, q, window)
        k, v = (torch.from_numpy(t).permute(1, 0, 2).repeat_interleave(2, 0) for t in pool.rows(pages, 0, 29))
        pos, key = torch.arange(24, 29)[:, None], torch.arange(29)[None]
        hidden = key > pos
        if window:
            hidden |= key <= pos - window
        z = torch.from_numpy(q).permute(1, 0, 2) @ k.transpose(1, 2) / 4
        ref = (torch.softmax(z.masked_fill(hidden, -math.inf), -1) @ v).permute(1, 0, 2).numpy()
        np.testing.assert_allclose(o, ref, rtol=0, atol=1e-13)
        assert (np.abs(o) <= mag + 1e-12).all()


def test_accept_sampled_hand_worked():
    x = np.log(np.array([[0.5, 0.3, 0.2], [0.1, 0.8, 0.1]]))
    q = np.array([[0.2, 0.6, 0.2], [1.0, 0.0, 0.0]])
    one = np.ones(3)
    # draft 1 has p/q = 0.5: accepted below, refused at it; the residue (0.3, 0, 0) leaves token 0
    assert oracle.accept_sampled([9, 1], x, 1.0, [0.49, 0], one, q) == (1, [1, 1])
    assert oracle.accept_sampled([9, 1], x, 1.0, [0.51, 0], one, q) == (0, [0])
    # certain drafts: accepted with p(d) itself; refused, the draft is out of the draw
    assert oracle.accept_sampled([9, 0], x, 1.0, [0.49, 0], one) == (1, [0, 1])
    assert oracle.accept_sampled([9, 0], x, 1.0, [0.51, 0], one) == (0, [1])
    # temperature 0: the argmax alone
    assert oracle.accept_sampled([9, 0], x, 0.0, [0.99, 0], one, q) == (1, [0, 1])
    assert oracle.accept_sampled([9, 2], x, 0.0, [0.0, 0], one, q) == (0, [0])
    # the noise decides the draw: weights 0.1, 0.8, 0.1 over noise 0.1, 1, 0.2
    assert oracle.accept_sampled([9], x[1:], 1.0, [0], np.array([0.1, 1.0, 0.2])) == (0, [0])


def test_accept_sampled_commits_the_targets_law():
    """Over many draws the first committed token is distributed as p whatever q is. 20,000 draws: a
    share's standard deviation is at most 0.0036, so 0.018 is five of them."""
    rng = np.random.default_rng(11)
    p, q = np.array([0.45, 0.25, 0.2, 0.1]), np.array([0.1, 0.6, 0.1, 0.2])
    x = np.log(np.stack([p, p]))
    n, seen = 20000, np.zeros(4)
    for _ in range(n):
        d = rng.choice(4, p=q)
        _, toks = oracle.accept_sampled([0, d], x, 1.0, rng.random(2), rng.exponential(size=4), np.stack([q, q]))
        seen[toks[0]] += 1
    assert np.abs(seen / n - p).max() < 0.018
