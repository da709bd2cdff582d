"""Top-k, top-p and min-p cuts and draws from them on the GPU against the float64 oracle: every kept set and token equal.

The kernel decides what exact arithmetic would, to 2^-37 of a row's weight; the oracle's own sums are off by 2^-40 or less at
these sizes. No tolerance: a row in which the two could differ has a border within that, one row in 2^20 or fewer."""
import numpy as np
import pytest

import oracle
import synth

pytestmark = pytest.mark.gpu


def _i32(a):
    import torch
    return torch.as_tensor(np.asarray(a, dtype=np.int32)).cuda()


def _f32(a):
    import torch
    return torch.as_tensor(np.asarray(a, dtype=np.float32)).cuda()


_made = {}


def _verifier(vocab, max_batch=64, max_span=17, max_rows=128):
    """A context of any vocabulary: zero weights, one layer of the smallest shape."""
    import torch
    from speculative_decoding_verify_02_gb300 import Verifier
    key = vocab, max_batch, max_span, max_rows
    if key not in _made:
        _made.clear()
        shape = synth.Shape("filter", 1, 128, 2, 2, 64, 128, vocab)
        w = {n: torch.zeros(d, dtype=torch.bfloat16, device="cuda") for n, d in shape.tensor_shapes().items()}
        _made[key] = Verifier(shape, w, page_size=16, n_pages=16, max_batch=max_batch, max_rows=max_rows, max_span=max_span,
                              max_context=256)
    return _made[key]


def _check(v, x, noise, off, T, k=None, p=None, m=None, status=0):
    """Filter (with n_kept), filter in place, and sample the rows of spans `off`; compare every row."""
    import torch
    B, R = len(off) - 1, len(x)
    dx, dn, d_off, dT = _f32(x), _f32(noise), _i32(off), _f32(T)
    cuts = dict(top_k=None if k is None else _i32(k), top_p=None if p is None else _f32(p), min_p=None if m is None else _f32(m))
    out, kept = torch.full_like(dx, 5.0), _i32(np.full(R, -3))
    v.filter_logits(dx, d_off, B, out, kept, dT, **cuts)
    again = dx.clone()
    v.filter_logits(again, d_off, B, again, None, dT, **cuts)
    tok, kept2 = _i32(np.full(R, -3)), _i32(np.full(R, -3))
    v.sample(dx, d_off, dn, B, tok, dT, n_kept=kept2, **cuts)
    torch.cuda.synchronize()
    assert v.get_status() == status
    out, again, kept, kept2, tok = (t.cpu().numpy() for t in (out, again, kept, kept2, tok))
    live = np.zeros(R, dtype=bool)
    for b in range(B):
        for r in range(off[b], off[b + 1]):
            live[r] = True
            toks, w = oracle.kept_tokens(x[r], np.float32(T[b]), 0 if k is None else k[b], 1.0 if p is None else np.float32(p[b]),
                                         0.0 if m is None else np.float32(m[b]))
            want = np.full(x.shape[1], -np.inf, dtype=np.float32)
            want[toks] = x[r, toks]
            assert kept[r] == len(toks) and kept2[r] == len(toks), (r, kept[r], kept2[r], len(toks))
            np.testing.assert_array_equal(out[r], want)
            np.testing.assert_array_equal(again[r], want)
            assert tok[r] == oracle.draw_kept(toks, w, noise[r]), r
    assert (out[~live] == 5).all() and (kept[~live] == -3).all() and (tok[~live] == -3).all()
    np.testing.assert_array_equal(again[~live], x[~live])


def _rows(rng, R, V, kind):
    if kind == "peaks":
        x = 2 * rng.normal(size=(R, V))
        for r in range(R):
            x[r, rng.integers(0, V, 30)] += 4 + 12 * rng.random(30)
    elif kind == "flat":
        x = 0.05 * rng.normal(size=(R, V))
    elif kind == "ties":
        x = np.round(4 * rng.normal(size=(R, V))) / 2
    elif kind == "equal":
        x = np.full((R, V), 1.25)
    elif kind == "steep":
        x = -40 * rng.exponential(size=(R, V))
    else:
        x = rng.normal(size=(R, V)) * 1e30
    return x.astype(np.float32)


KINDS = ["peaks", "flat", "ties", "equal", "steep", "huge"]


@pytest.mark.parametrize("V", [1, 2, 5, 511, 2047, 2048, 2049, 4097, 30001])
@pytest.mark.parametrize("kind", KINDS)
def test_cuts_of_many_rows(kind, V):
    rng = np.random.default_rng(V)
    R = 24
    x, noise = _rows(rng, R, V, kind), rng.exponential(size=(R, V))
    T = np.exp(rng.normal(size=R))
    T[rng.random(R) < 0.1] = 0
    v = _verifier(V)
    off = np.arange(R + 1)
    k = np.exp(rng.uniform(0, np.log(V + 1), R)).astype(int)
    k[:3] = 0, V, V + 7
    p, m = rng.uniform(0.01, 1, R), rng.uniform(0, 0.4, R) ** 2
    p[3:6] = 1.0, 0.0, 1 - 2.0 ** -24
    m[6:9] = 0.0, 1.0, 1.5
    for cuts in (dict(), dict(k=k), dict(p=p), dict(m=m), dict(k=k, p=p), dict(k=k, p=p, m=m)):
        _check(v, x, noise, off, T, **cuts)


@pytest.mark.parametrize("kind", ["peaks", "flat", "ties", "equal"])
def test_full_vocabulary(kind):
    rng = np.random.default_rng(7)
    V, R = 151936, 6
    x, noise = _rows(rng, R, V, kind), rng.exponential(size=(R, V))
    v = _verifier(V)
    T = [1.0, 0.7, 1.3, 0.0, 2.0, 0.05]
    _check(v, x, noise, np.arange(R + 1), T, p=[0.5, 0.9, 0.99, 0.9, 0.999, 0.3])
    _check(v, x, noise, np.arange(R + 1), T, k=[1, 50, 3000, 7, 100000, 2048])
    _check(v, x, noise, np.arange(R + 1), T, k=[1, 50, 3000, 7, 100000, 2048], p=[0.5, 0.9, 0.99, 0.9, 0.8, 0.3], m=[0.1, 0.01, 0, 0.1, 0.5, 0.001])


@pytest.mark.parametrize("V", [2049, 30001])
def test_lists_that_crowd(V):
    """Rows whose likely tokens lie close together: some hundreds to two thousand equal or nearly equal logits above the rest, or
    below a single large one; infinite temperatures."""
    rng = np.random.default_rng(11)
    x = (rng.normal(size=(10, V)) - 50).astype(np.float32)
    for r, n in enumerate((200, 255, 300, 900, 1990)):
        at = rng.choice(V, n, replace=False)
        x[2 * r, at] = 1.25                                        # equal
        x[2 * r + 1, at] = 1.25 + 2.0 ** -20 * rng.integers(0, 40, n)  # nearly
        if r % 2:
            x[2 * r:2 * r + 2, at[0]] = 3e4                        # one far above
    noise = rng.exponential(size=x.shape)
    v = _verifier(V)
    off = np.arange(11)
    for T in ([1.0] * 10, [3e4] * 10, [np.inf] * 10):
        for cuts in (dict(k=[150] * 10), dict(p=[0.4] * 10), dict(k=[180] * 10, p=[0.7] * 10), dict(k=[1500] * 10, p=[0.9] * 10, m=[1e-3] * 10)):
            _check(v, x, noise, off, T, **cuts)


def test_largest_vocabulary():
    """The largest that is taken, and one token more."""
    from speculative_decoding_verify_02_gb300 import SdvError
    rng = np.random.default_rng(13)
    V, R = 393216, 4
    x, noise = _rows(rng, R, V, "peaks"), rng.exponential(size=(R, V))
    x[2] = 0.0
    v = _verifier(V, max_batch=8)
    for cuts in (dict(k=[40, 300, 200000, 7], p=[0.9, 0.99, 0.5, 1.0]), dict(p=[0.9, 0.7, 0.25, 0.9], m=[0.01, 0, 0, 0.2])):
        _check(v, x, noise, np.arange(R + 1), [1.0, 0.8, 1.0, 1.5], **cuts)
    v = _verifier(V + 1, max_batch=8)
    big = _f32(np.zeros((1, V + 1)))
    with pytest.raises(SdvError):
        v.filter_logits(big, _i32([0, 1]), 1, big, None, _f32([1.0]))


def test_tokens_of_one_corner():
    """All tokens above -inf lie next to one another, so that few threads hold them."""
    rng = np.random.default_rng(12)
    V = 30001
    x = np.full((8, V), -np.inf, dtype=np.float32)
    for r, (at, n) in enumerate(((0, 2500), (3800, 2500), (27000, 3001), (0, 2049), (100, 4000), (15000, 9000), (29999, 2), (7, 2100))):
        x[r, at:at + n] = 2 * rng.normal(size=min(n, V - at))
    noise = rng.exponential(size=x.shape)
    v = _verifier(V)
    for k in (5, 60, 100, 250, 256, 257, 1500):
        _check(v, x, noise, np.arange(9), [0.8] * 8, k=[k] * 8, p=[0.95] * 8)


def test_borders_next_to_a_token():
    """Equal weights, whose sums lie on p's border in exact arithmetic: the token at the border is dropped, since the weight
    before it is not less; one unit of p more keeps it."""
    V = 4096
    x = np.zeros((4, V), dtype=np.float32)
    noise = np.random.default_rng(1).exponential(size=x.shape)
    v = _verifier(V)
    p = np.array([0.5, np.nextafter(np.float32(0.5), np.float32(1)), 0.25, np.nextafter(np.float32(0.25), np.float32(0))])
    _check(v, x, noise, np.arange(5), [1.0] * 4, p=p)
    x[:, V // 2:] = -np.inf                  # half of them, and a list instead of a search
    _check(v, x, noise, np.arange(5), [1.0] * 4, p=p)


def test_odd_rows():
    inf, nan = np.inf, np.nan
    rng = np.random.default_rng(5)
    for V in (40, 9001):
        x = rng.normal(size=(9, V)).astype(np.float32)
        x[0, 1:] = -inf
        x[1, ::2] = nan
        x[2, [3, V - 1]] = inf
        x[3, 7] = inf
        x[4] = -inf
        x[4, V - 1] = -1e38
        x[5] = np.where(rng.random(V) < 0.5, 0.0, -0.0)
        x[6] = -3e38
        x[6, 5] = 3e38
        x[7, 3:] = nan
        noise = rng.exponential(size=x.shape)
        v = _verifier(V)
        for cuts in (dict(), dict(k=[3] * 9), dict(p=[0.6] * 9), dict(m=[0.2] * 9), dict(k=[30] * 9, p=[0.9] * 9, m=[0.01] * 9)):
            _check(v, x, noise, np.arange(10), [1.0, 0.5, 1, 1, 1, 1, 1, 1e30, 1e-30], **cuts)


def test_rows_without_a_token():
    from speculative_decoding_verify_02_gb300 import SDV_ERR_DEVICE
    for V in (50, 5000):
        x = np.zeros((3, V), dtype=np.float32)
        x[1] = -np.inf
        x[1, ::3] = np.nan
        _check(_verifier(V), x, np.ones_like(x), np.arange(4), [1.0, 1.0, 0.0], k=[4, 4, 4], status=SDV_ERR_DEVICE)


@pytest.mark.parametrize("off", [[0, 3, 3, 8], [2, 4, 9, 10]])
def test_spans_and_rows_of_none(off):
    rng = np.random.default_rng(2)
    x, noise = _rows(rng, 12, 3000, "peaks"), rng.exponential(size=(12, 3000))
    _check(_verifier(3000), x, noise, np.asarray(off), [0.8, 1.0, 1.5], k=[5, 500, 40], p=[0.9, 0.8, 0.95])


def test_spans_that_do_not_fit_are_refused():
    import torch
    from speculative_decoding_verify_02_gb300 import SDV_ERR_ARG
    v = _verifier(3000)
    x, tok = torch.randn(20, 3000, device="cuda"), _i32(np.full(20, -3))
    for off, rows in (([0, 18, 20], range(18, 20)), ([0, 2, 30], range(2)), ([0, -1, 3], []), ([-1, 2, 4], range(2, 4))):
        tok.fill_(-3)
        v.sample(x, _i32(off), torch.ones_like(x), 2, tok, _f32([0.0, 0.0]))
        torch.cuda.synchronize()
        assert v.get_status() == SDV_ERR_ARG
        got = tok.cpu().numpy()
        assert (got[list(rows)] == x.argmax(-1).cpu().numpy()[list(rows)]).all()
        assert (np.delete(got, list(rows)) == -3).all()


@pytest.mark.parametrize("V", [777, 5003])
def test_strided_rows(V):
    """Rows of a wider matrix at odd offsets, every stride of its own; what lies between the rows stays."""
    import torch
    v = _verifier(V)
    R = 5
    x, e = torch.randn(R, V, device="cuda") * 3, torch.empty(R, V, device="cuda").exponential_()
    off, T, p = _i32(np.arange(R + 1)), _f32([1.0] * R), _f32([0.8] * R)
    ref, kept, tok = torch.empty_like(x), _i32(np.zeros(R)), _i32(np.zeros(R))
    v.filter_logits(x, off, R, ref, kept, T, top_p=p)
    v.sample(x, off, e, R, tok, T, top_p=p)
    for shift in (0, 1, 2, 3):
        wide, noise, out = (torch.full((R, V + 9 + i), 4.0, device="cuda") for i in range(3))
        wide[:, shift:shift + V] = x
        noise[:, 1:1 + V] = e
        tok2 = _i32(np.zeros(R))
        v.filter_logits(wide[:, shift:shift + V], off, R, out[:, 3 - shift:3 - shift + V], None, T, top_p=p)
        v.sample(wide[:, shift:shift + V], off, noise[:, 1:1 + V], R, tok2, T, top_p=p)
        torch.cuda.synchronize()
        assert torch.equal(out[:, 3 - shift:3 - shift + V], ref) and torch.equal(tok2, tok)
        assert (out[:, :3 - shift] == 4).all() and (out[:, 3 - shift + V:] == 4).all()


def test_equal_scores_draw_the_lowest_token():
    import torch
    v = _verifier(6000)
    x, e = torch.zeros(2, 6000, device="cuda"), torch.full((2, 6000), 2.0, device="cuda")
    e[:, [17, 4000]] = 1.0
    tok = _i32([0, 0])
    v.sample(x, _i32([0, 1, 2]), e, 2, tok, _f32([1.0, 1.0]))
    assert tok.tolist() == [17, 17]
    e[:, 17] = float(np.nextafter(np.float32(1), np.float32(2)))      # nearer than fp32 scores tell apart
    v.sample(x, _i32([0, 1, 2]), e, 2, tok, _f32([1.0, 1.0]))
    assert tok.tolist() == [4000, 4000]


def test_the_draw_follows_the_filtered_distribution():
    """4,096 draws of a kept set of seven: each share within five standard deviations."""
    import torch
    V, n = 3001, 128
    v = _verifier(V)
    x = torch.full((1, V), -4.0, device="cuda")
    x[0, torch.tensor([5, 70, 900, 2048, 2999, 3000, 1])] = torch.tensor([3.0, 2.5, 2.0, 1.5, 1.0, 0.5, 0.0], device="cuda")
    x = x.expand(n, V).contiguous()
    g = torch.Generator(device="cuda").manual_seed(3)
    tok, T, k = _i32(np.zeros(n)), _f32([0.9] * 64), _i32([7] * 64)
    counts = np.zeros(V)
    off = _i32(np.arange(65) * 2)
    for _ in range(32):
        v.sample(x, off, torch.empty(n, V, device="cuda").exponential_(generator=g), 64, tok, T, top_k=k)
        counts += np.bincount(tok.cpu().numpy(), minlength=V)
    toks, w = oracle.kept_tokens(x[0].cpu().numpy(), np.float32(0.9), top_k=7)
    p = np.zeros(V)
    p[toks] = w / w.sum()
    total = counts.sum()
    assert (np.abs(counts / total - p) <= 5 * np.sqrt(p * (1 - p) / total)).all()


def test_graph_and_side_stream():
    import torch
    v = _verifier(20000)
    R = 8
    x, e = torch.randn(R, 20000, device="cuda") * 4, torch.empty(R, 20000, device="cuda").exponential_()
    off, T, k, p = _i32(np.arange(R + 1)), _f32([0.9] * R), _i32([40] * R), _f32([0.9] * R)
    out, tok, kept = torch.empty_like(x), _i32(np.zeros(R)), _i32(np.zeros(R))

    def both(stream=None):
        v.filter_logits(x, off, R, out, kept, T, top_k=k, top_p=p, stream=stream)
        v.sample(x, off, e, R, tok, T, top_k=k, top_p=p, stream=stream)

    both()
    torch.cuda.synchronize()
    ref = out.clone(), tok.clone(), kept.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out.zero_(), tok.zero_()
    torch.cuda.synchronize()
    both(side)
    torch.cuda.synchronize()
    assert torch.equal(out, ref[0]) and torch.equal(tok, ref[1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        both()
    x.mul_(0.5)
    p.fill_(0.5)
    g.replay()
    torch.cuda.synchronize()
    got = out.clone(), tok.clone(), kept.clone()
    both()
    torch.cuda.synchronize()
    assert torch.equal(out, got[0]) and torch.equal(tok, got[1]) and torch.equal(kept, got[2]) and not torch.equal(got[2], ref[2])


def test_binding_refusals():
    import torch
    from speculative_decoding_verify_02_gb300 import SdvError
    v = _verifier(3000)
    x, off, T, tok = torch.zeros(4, 3000, device="cuda"), _i32(range(5)), _f32([1] * 4), _i32([0] * 4)
    ok = dict(logits=x, row_off=off, noise=torch.ones_like(x), B=4, tokens=tok, temperature=T)
    for bad in (dict(logits=x.double()), dict(logits=x[:, :2999]), dict(logits=x.t()), dict(logits=x.cpu()), dict(row_off=off[:4]),
                dict(noise=torch.ones(3, 3000, device="cuda")), dict(tokens=tok[:3]), dict(tokens=tok.long()), dict(temperature=T[:3]),
                dict(top_k=T), dict(top_p=tok), dict(min_p=T.double()), dict(n_kept=tok[:2])):
        with pytest.raises(ValueError):
            v.sample(**dict(ok, **bad))
    with pytest.raises(ValueError):
        v.filter_logits(x, off, 4, x[:3], None, T)
    with pytest.raises(SdvError):
        v.sample(**dict(ok, B=0))



def _crowds(rng, V, T, heavy, light):
    """A row of one largest logit, `heavy` tokens of about its weight, and two crowds of light ones, 2^-3 to 2^-8, a unit of the last
    place apart, in any order; a p whose border lies at most three tokens before the first crowd's end."""
    T, m = np.float32(T), np.float32(rng.normal())
    a = np.float32(m - T * rng.choice([0.0144, 0.02, 0.5, 1.01]) * np.log(2))
    b = np.float32(m - T * rng.uniform(3, 8) * np.log(2))
    x = np.full(V, np.nextafter(b, np.float32(-np.inf)))
    x[0], x[1:1 + heavy], x[1 + heavy:1 + heavy + light] = m, a, b
    w = np.exp((x.astype(np.float64) - float(m)) / float(T))
    p = np.float32((w[:1 + heavy + light].sum() - rng.uniform(0, 3) * w[1 + heavy]) / w.sum())
    return x[rng.permutation(V)], p


def test_borders_between_neighbouring_logits():
    """Sums of fp32 weights cannot tell the border, those that decide are exact, also of what lies before the crowd."""
    V, rng = 393216, np.random.default_rng(17)
    v = _verifier(V, max_batch=8)
    noise = np.ones((8, V), dtype=np.float32)
    for T in (0.2, 0.5, 0.8, 1.0, 1.3, 2.0):
        x, p = zip(*(_crowds(rng, V, T, 49152 * int(rng.integers(1, 4)), int(rng.integers(20000, 220000))) for _ in range(8)))
        _check(v, np.stack(x), noise, np.arange(9), [T] * 8, p=p)


@pytest.mark.parametrize("least", [-32, -35.5])
def test_borders_of_crowds_of_equal_weights(least):
    """Some hundred thousand tokens of two neighbouring logits behind a large one, and a p that brings the border within 2^least to
    2^(least + 2) of the row's weight to a token's edge. A row's border in tokens of the first crowd is (p total - 1) / w."""
    import torch
    V, rng = 393216, np.random.default_rng(23)
    v = _verifier(V, max_batch=8)
    for T in (0.3, 0.5, 0.7, 0.9, 1.0, 1.3, 1.7, 2.4):
        x, p, want = np.empty((8, V), dtype=np.float32), np.empty(8, dtype=np.float32), []
        for r in range(8):
            m = np.float32(rng.normal())
            b = np.float32(m - np.float32(T) * rng.uniform(17, 21) * np.log(2))
            c = np.nextafter(b, np.float32(-np.inf))
            wb, wc = (np.exp((np.float64(y) - np.float64(m)) / np.float64(np.float32(T))) for y in (b, c))
            n = int(rng.integers(100000, 250000))
            total = 1 + n * wb + (V - 1 - n) * wc
            tried = np.float32((1 + 0.9 * n * wb) / total) * np.float32(1) - np.arange(1 << 18) * np.float32(2.0 ** -24)
            k = (tried.astype(np.float64) * total - 1) / wb
            off = np.abs(k - np.rint(k)) * wb / total
            i = int(np.flatnonzero((off > 2.0 ** least) & (off < 2.0 ** (least + 2)) & (k > 1) & (k < n - 2))[0])
            x[r], x[r, 1:n + 1], x[r, 0], p[r] = c, b, m, tried[i]
            x[r] = x[r, rng.permutation(V)]
            want.append(1 + int(np.ceil(k[i])))
        out, kept = _f32(x), _i32([0] * 8)
        v.filter_logits(out, _i32(range(9)), 8, out, kept, _f32([T] * 8), top_p=_f32(p))
        torch.cuda.synchronize()
        assert kept.tolist() == want and (out > -np.inf).sum(-1).tolist() == want


@pytest.mark.parametrize("V", [40, 2048, 9001])
def test_noise_of_any_size(V):
    """Noise from the smallest positive fp32 to the largest: quotients past fp32's range are compared like all others."""
    rng = np.random.default_rng(V)
    R = 60
    x = (-60 * rng.random((R, V))).astype(np.float32)
    noise = np.maximum(10.0 ** rng.uniform(-46, 3, (R, V)), 1.5e-45).astype(np.float32)
    noise[8:16] = rng.exponential(size=(8, V))
    for r in range(8, 16):          # a few tiny ones among usual ones
        noise[r, rng.integers(0, V, 3)] = [1.5e-45, 1e-39, 1e-30]
    x[16:] *= 3
    noise[56:] = 10.0 ** rng.uniform(-20, 38, (4, V))
    v = _verifier(V)
    assert (noise > 0).all() and np.isfinite(noise).all()
    for cuts in (dict(), dict(k=[30] * R), dict(p=[0.999] * R), dict(m=[1e-30] * R)):
        _check(v, x, noise, np.arange(R + 1), [1.0] * R, **cuts)


def test_in_place_rows_lie_where_the_logits_do():
    import torch
    from speculative_decoding_verify_02_gb300 import SdvError
    v = _verifier(3000)
    room = torch.randn(8 * 3000, device="cuda")
    x, far = room[:4 * 3000].view(4, 3000), room.as_strided((4, 3000), (6000, 1))
    keep, off, T = room.clone(), _i32(range(5)), _f32([1.0] * 4)
    with pytest.raises(SdvError):
        v.filter_logits(x, off, 4, far, None, T, top_k=_i32([3] * 4))
    assert torch.equal(room, keep)
    v.filter_logits(far, off, 4, far, None, T, top_k=_i32([3] * 4))
    assert ((far > -np.inf).sum(-1) == 3).all() and torch.equal(room[3000:6000], keep[3000:6000])
    v.filter_logits(x[:1], off[:2], 1, room.as_strided((1, 3000), (6000, 1)), None, T, top_k=_i32([2]))
    assert int((x[0] > -np.inf).sum()) == 2
