"""Attention for groups of sequences that share a prefix, on the GPU against the float64 oracle.

Tolerances, for a result o = sum p v / sum p with A = sum p |v| / sum p, n keys and scores up to Z before the cap: a weight's
relative error is that of its exponent, (D + 2) 2^-24 Z' for the product's roundings (Z' = the sum of |q_d k_d| / sqrt(D)), three
roundings of the exponent itself (3 2^-24 times the largest exponent, cap and distance included), 2^-22 of the exponential and
of the cap's, 2^-16 of the two planes of a probability (bf16; fewer in fp16); it counts twice, in the sum with v and in the sum
of weights. Sums of n terms in fp32 add n 2^-24 each, and the result is rounded once, eps / 2."""
import numpy as np
import pytest

import oracle

pytestmark = pytest.mark.gpu


def _dev(a, dtype=None):
    import torch
    t = torch.as_tensor(np.ascontiguousarray(a))
    return t.to("cuda", dtype) if dtype is not None else t.to("cuda")


def _i32(a):
    return _dev(np.asarray(a, dtype=np.int32))


class Setup:
    """Groups of sequences (a list of sizes and of prefix lengths), the positions of each beyond its group's prefix and its
    span. Whole pages of a prefix are shared, the rest of it is a copy of each sequence's; everything else in the pool is NaN."""

    def __init__(self, sizes, prefix, own, spans, nq=8, nkv=2, D=128, ps=16, dtype="bf16", seed=0, groups=True, room=0, junk=True,
                 max_span=None, layers=1, layer=0):
        import torch
        from speculative_decoding_verify_02_gb300 import SharedAttention
        rng = self.rng = np.random.default_rng(seed)
        self.nq, self.nkv, self.D, self.ps, self.layer = nq, nkv, D, ps, layer
        self.B, self.G = len(own), len(sizes) if groups else 0
        self.group = np.repeat(np.arange(len(sizes)), sizes)
        self.prefix, self.spans = np.asarray(prefix), np.asarray(spans)
        self.base = self.prefix[self.group] + np.asarray(own)
        self.off = np.concatenate([[0], np.cumsum(spans)])
        self.rows = int(self.off[-1])
        end = self.base + self.spans
        per = -(-int(end.max() + room) // ps)
        self.max_span = max_span or max(1, int(self.spans.max()))
        T = torch.bfloat16 if dtype == "bf16" else torch.float16
        # keys and values of every position, rounded to the type, then laid into pages
        n_pages = 3 + sum(-(-int(e) // ps) for e in end) + 1
        ids = list(rng.permutation(n_pages))
        pool = np.full((n_pages, 2, nkv, ps, D), np.nan if junk else 0.0, dtype=np.float32)
        self.kv, table, whole = [], np.full((self.B, per), -1), {}
        shared = [np.asarray(_dev(rng.normal(size=(2, max(1, p), nkv, D)).astype(np.float32), T).float().cpu()) for p in self.prefix]
        for b in range(self.B):
            g, P = self.group[b], int(self.prefix[self.group[b]])
            kv = _dev(rng.normal(size=(2, int(end[b]), nkv, D)).astype(np.float32), T).float().cpu().numpy()
            kv[:, :P] = shared[g][:, :P]
            self.kv.append(kv)
            for j in range(-(-int(end[b]) // ps)):
                if groups and (j + 1) * ps <= P and (g, j) in whole:
                    table[b, j] = whole[g, j]
                else:
                    table[b, j] = ids.pop()
                    whole[g, j] = table[b, j]
                stop = min(int(end[b]), (j + 1) * ps)
                pool[table[b, j], :, :, :stop - j * ps] = kv[:, j * ps:stop].transpose(0, 2, 1, 3)
        self.table = table
        self.pool = torch.zeros(layers, *pool.shape, dtype=T, device="cuda")
        self.pool[layer] = _dev(pool).to(T)
        self.T, self.eps = T, torch.finfo(T).eps
        self.d_table, self.d_off, self.d_base = _i32(table), _i32(self.off), _i32(self.base)
        self.d_group = _i32(np.concatenate([[0], np.cumsum(sizes)])) if groups else None
        self.d_prefix = _i32(self.prefix) if groups else None
        self.plan = SharedAttention(layers, nq, nkv, D, page_size=ps, n_pages=n_pages, max_batch=self.B,
                                    max_rows=max(self.rows, self.max_span), max_span=self.max_span,
                                    max_context=max(per * ps if room else int(end.max()), self.max_span), dtype=T, pool=self.pool)
        self.q = _dev((1.5 * rng.normal(size=(max(1, self.rows), nq, D))).astype(np.float32), T)

    def run(self, q=None, out=None, **kw):
        import torch
        q = self.q if q is None else q
        out = torch.full_like(q, 7.0) if out is None else out
        kw.setdefault("group_off", self.d_group)
        kw.setdefault("prefix_len", self.d_prefix)
        self.plan.attention(self.layer, q, self.d_table, self.d_off, self.d_base, self.B, self.max_span, out, G=self.G, **kw)
        torch.cuda.synchronize()
        return out

    def check(self, out, q=None, window=0, cap=0.0, slopes=None, skip=(), kv=None):
        q = (self.q if q is None else q).double().cpu().numpy()
        o = out.double().cpu().numpy()
        grp, worst = self.nq // self.nkv, 0.0
        for b in range(self.B):
            rows = slice(self.off[b], self.off[b + 1])
            if b in skip or self.spans[b] == 0:
                continue
            pos = self.base[b] + np.arange(self.spans[b])
            k, v = (self.kv if kv is None else kv)[b].astype(np.float64)
            for h in range(self.nq):
                s = 0.0 if slopes is None else float(slopes[h])
                z = oracle.scores(q[rows, h], k[:, h // grp], pos, window, cap, s)
                ref = oracle.attend(z, v[:, h // grp])
                seen = z > -np.inf
                w = np.exp(z - z.max(-1, keepdims=True))
                w /= w.sum(-1, keepdims=True)
                mag = np.where(seen, np.abs(q[rows, h]) @ np.abs(np.nan_to_num(k[:, h // grp])).T, 0).max() / np.sqrt(self.D)
                top = np.abs(np.where(seen, z, 0)).max() + cap + s * len(k)
                A = np.stack([w[i, m] @ np.abs(v[m, h // grp]) for i, m in enumerate(seen)])
                e = (self.D + 2) * 2.0 ** -24 * mag + 3 * 2.0 ** -24 * 1.45 * top + 2.0 ** -22 * (1 + 3 * cap) + 2.0 ** -16
                tol = (2 * e + 2 * len(k) * 2.0 ** -24) * A + self.eps / 2 * np.abs(ref) * 1.01 + 2.0 ** -24
                d = np.abs(o[rows, h] - ref)
                assert np.isfinite(o[rows, h]).all(), f"sequence {b} head {h}"
                assert (d <= tol).all(), f"sequence {b} head {h}: {d.max()} over {tol.flat[d.argmax()]}"
                worst = max(worst, float((d / tol).max()))
        return worst


CASES = {
    "one row alone": dict(sizes=[1], prefix=[0], own=[0], spans=[1], groups=False),
    "one row, prefix of one": dict(sizes=[1], prefix=[1], own=[0], spans=[1]),
    "no groups": dict(sizes=[1] * 3, prefix=[0] * 3, own=[5, 300, 127], spans=[4, 1, 9], groups=False),
    "a whole chunk": dict(sizes=[1], prefix=[0], own=[127], spans=[1], groups=False),
    "prefix ends a chunk": dict(sizes=[3], prefix=[256], own=[0, 128, 5], spans=[2, 1, 3]),
    "prefix ends inside a page": dict(sizes=[4], prefix=[203], own=[0, 1, 130, 13], spans=[3, 1, 2, 5]),
    "two groups, one without prefix": dict(sizes=[2, 3], prefix=[0, 500], own=[40, 0, 3, 0, 200], spans=[2, 3, 1, 4, 2]),
    "empty spans": dict(sizes=[3, 2], prefix=[100, 60], own=[0, 7, 3, 0, 0], spans=[0, 2, 0, 0, 0]),
    "tiles above 256 rows": dict(sizes=[40, 2], prefix=[700, 100], own=[i % 7 * 9 for i in range(42)], spans=[1 + i % 4 for i in range(42)]),
    "a span of many tiles": dict(sizes=[2], prefix=[130], own=[20, 0], spans=[150, 77]),
    "129 rows": dict(sizes=[1], prefix=[140], own=[0], spans=[129], nq=1, nkv=1, D=64),
    "heads as they are": dict(sizes=[3], prefix=[90], own=[4, 0, 60], spans=[2, 5, 1], nq=6, nkv=6, D=64),
    "one kv head": dict(sizes=[5], prefix=[1000], own=[0, 9, 3, 100, 0], spans=[1, 3, 1, 2, 1], nq=16, nkv=1),
    "five heads a kv head": dict(sizes=[7], prefix=[333], own=[5] * 7, spans=[1, 2, 3, 4, 5, 6, 7], nq=20, nkv=4),
    "pages of 8": dict(sizes=[3], prefix=[77], own=[0, 33, 9], spans=[4, 1, 2], ps=8),
    "pages of 24": dict(sizes=[3], prefix=[300], own=[0, 33, 9], spans=[4, 1, 2], ps=24, D=64),
    "pages of 10": dict(sizes=[3], prefix=[300], own=[0, 33, 9], spans=[4, 1, 2], ps=10),
    "pages of 7": dict(sizes=[2], prefix=[140], own=[0, 33], spans=[4, 1], ps=7, D=64),
    "pages of one": dict(sizes=[2], prefix=[40], own=[0, 9], spans=[2, 1], ps=1, D=64),
    "pages of 128": dict(sizes=[3], prefix=[300], own=[0, 33, 9], spans=[4, 1, 2], ps=128),
    "pages of 256": dict(sizes=[2], prefix=[600], own=[0, 33], spans=[4, 1], ps=256, D=64),
    "200 sequences": dict(sizes=[150, 50], prefix=[65, 33], own=[i % 5 for i in range(200)], spans=[1] * 200, D=64, nq=4, nkv=2),
    "256 sequences in 128 groups": dict(sizes=[2] * 128, prefix=[16 + i for i in range(128)], own=[0, 1] * 128, spans=[1] * 256, D=64, nq=2),
    "long": dict(sizes=[4], prefix=[9000], own=[0, 40, 5, 700], spans=[2, 1, 8, 3], nq=4, nkv=1),
}


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("name", CASES)
def test_attention(name, dtype):
    s = Setup(dtype=dtype, **CASES[name])
    s.check(s.run())
    assert s.plan.get_status() == 0


@pytest.mark.parametrize("window", [1, 2, 16, 100, 129, 5000])
@pytest.mark.parametrize("name", ["prefix ends inside a page", "two groups, one without prefix", "tiles above 256 rows", "pages of 10"])
def test_window(name, window):
    s = Setup(**CASES[name])
    s.check(s.run(window=window), window=window)
    # tables without the pages before every row's window
    for b in range(s.B):
        lowest = min(s.base[i] for i in range(s.B) if s.group[i] == s.group[b])
        s.table[b, :max(0, (lowest - window + 1)) // s.ps] = -1
    s.d_table = _i32(s.table)
    s.check(s.run(window=window), window=window)
    assert s.plan.get_status() == 0


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("cap, bias, window", [(2.0, False, 0), (50.0, False, 40), (0.0, True, 0), (10.0, True, 100)])
def test_cap_and_bias(cap, bias, window, dtype):
    for name in ("prefix ends inside a page", "tiles above 256 rows", "heads as they are", "one row alone"):
        s = Setup(dtype=dtype, **CASES[name])
        slopes = 2.0 ** (-8 * np.arange(1, s.nq + 1) / s.nq) if bias else None
        out = s.run(window=window, softcap=cap, slopes=None if slopes is None else _dev(slopes.astype(np.float32)))
        s.check(out, window=window, cap=cap, slopes=None if slopes is None else slopes.astype(np.float32))


@pytest.mark.parametrize("cap", [0.0, 5.0])
def test_large_scores(cap):
    """Scores of hundreds either way: one key takes all, references move by far, early parts vanish beside late ones."""
    s = Setup(**CASES["long"])
    s.q *= 40
    s.check(s.run(softcap=cap), cap=cap)


def test_rising_scores():
    """Each chunk's scores above the last one's: the reference moves in every step."""
    s = Setup(sizes=[2], prefix=[1500], own=[0, 300], spans=[1, 40], nq=4, nkv=1)
    ramp = np.linspace(0, 12, int(max(s.base + s.spans)))
    q = np.zeros((s.rows, 4, 128), dtype=np.float32)
    q[..., 0] = 16
    s.q = _dev(q, s.T)
    for b in range(s.B):
        s.kv[b][0, :, :, 0] = _dev(ramp[:s.kv[b].shape[1], None].astype(np.float32), s.T).float().cpu().numpy()
        for j in range(-(-s.kv[b].shape[1] // s.ps)):
            stop = min(s.kv[b].shape[1], (j + 1) * s.ps)
            s.pool[0, s.table[b, j], :, :, :stop - j * s.ps] = _dev(s.kv[b][:, j * s.ps:stop].transpose(0, 2, 1, 3).copy(), s.T)
    s.check(s.run())


@pytest.mark.parametrize("bad", [np.nan, np.inf, -np.inf])
@pytest.mark.parametrize("which", [0, 1])
@pytest.mark.parametrize("spans", [[6, 3], [60, 40]])
def test_what_a_row_does_not_see_does_not_reach_it(which, bad, spans):
    """One position of a span holds K or V that is not finite: the rows before it keep their results bit by bit, the rows
    that see it are spoilt; other sequences and heads keep theirs."""
    import torch
    kw = dict(sizes=[2], prefix=[150], own=[10, 0], spans=spans, nq=4, nkv=2)
    s = Setup(**kw)
    clean = s.run()
    p = int(s.base[0]) + 3
    s.pool[0, int(s.table[0, p // s.ps]), which, 1, p % s.ps, 5] = float(bad)
    out = s.run()
    same = torch.ones(s.rows, s.nq, dtype=torch.bool, device="cuda")
    same[3:spans[0], 2:] = False
    assert torch.equal(out[same], clean[same])
    if which == 1:
        assert not torch.isfinite(out[3:spans[0], 2:]).all(-1).any()
    elif not np.isneginf(bad) and not np.isposinf(bad):
        assert torch.isnan(out[3:spans[0], 2:]).all()


def test_positions_that_left_the_window_do_not_reach_a_row():
    import torch
    s = Setup(sizes=[3], prefix=[200], own=[0, 30, 9], spans=[5, 2, 1], nq=4, nkv=2)
    clean = s.run(window=20)
    dead = int(min(s.base)) - 20            # below every row's window, in the chunk that it begins in
    assert dead // 128 == (dead + 1) // 128
    for t in range(dead // 128 * 128, dead + 1):
        s.pool[0, int(s.table[0, t // s.ps]), :, :, t % s.ps] = float("nan")
    assert torch.equal(s.run(window=20), clean)


def test_nan_queries_spoil_their_own_row_and_head_only():
    import torch
    s = Setup(**CASES["tiles above 256 rows"])
    clean = s.run()
    s.q[5, 3, 17] = float("nan")
    s.q[60, 0, 0] = float("inf")
    out = s.run()
    same = torch.ones(s.rows, s.nq, dtype=torch.bool, device="cuda")
    same[5, 3] = same[60, 0] = False
    assert torch.equal(out[same], clean[same]) and torch.isnan(out[5, 3]).all() and torch.isnan(out[60, 0]).any()


@pytest.mark.parametrize("shift", [0, 1, 4])
def test_strided_rows(shift):
    """Queries and results as parts of wider rows, aligned to 16 bytes and not."""
    import torch
    s = Setup(**CASES["prefix ends inside a page"])
    ref = s.run()
    wide = torch.full((s.rows, 3 * s.nq * s.D + 8), 5.0, dtype=s.T, device="cuda")
    q = wide[:, shift:shift + s.nq * s.D].view(s.rows, s.nq, s.D)
    q.copy_(s.q)
    out = wide[:, s.nq * s.D + 8 + shift:][:, :s.nq * s.D].view(s.rows, s.nq, s.D)
    keep = wide.clone()
    s.run(q, out)
    assert torch.equal(out, ref)
    out.copy_(keep[:, s.nq * s.D + 8 + shift:][:, :s.nq * s.D].view(s.rows, s.nq, s.D))
    assert torch.equal(wide, keep)


def test_rows_of_no_span_are_left_alone():
    import torch
    s = Setup(**CASES["prefix ends inside a page"])
    ref = s.run()
    q = torch.cat([s.q, s.q[:3]])
    out = torch.full_like(q, 9.0)
    s.plan.cfg  # the handle takes as many rows as max_rows says
    big = Setup(**CASES["prefix ends inside a page"], max_span=20)
    big.run(q, out)
    assert torch.equal(out[:s.rows], ref) and (out[s.rows:] == 9).all()


def test_repeated_calls_layers_streams_and_graphs():
    """The same bits each time, in another layer, on a side stream and from a graph that is replayed with other lengths."""
    import torch
    s = Setup(**CASES["tiles above 256 rows"], layers=3, layer=2)
    ref = s.run()
    assert torch.equal(s.run(), ref)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = torch.zeros_like(ref)
    with torch.cuda.stream(side):
        s.run(out=out)
    assert torch.equal(out, ref)
    g = torch.cuda.CUDAGraph()
    out.zero_()
    with torch.cuda.graph(g):
        s.plan.attention(2, s.q, s.d_table, s.d_off, s.d_base, s.B, s.max_span, out, group_off=s.d_group, prefix_len=s.d_prefix, G=s.G)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, ref)
    # shorter prefixes (the rest becomes each sequence's own) and spans cut to one row
    spans = np.minimum(s.spans, 1)
    s.d_prefix.copy_(_i32(s.prefix - 33))
    s.d_off.copy_(_i32(np.concatenate([[0], np.cumsum(spans)])))
    g.replay()
    torch.cuda.synchronize()
    t = Setup(**dict(CASES["tiles above 256 rows"], spans=spans.tolist()))
    t.q[:] = s.q[:t.rows]
    t.kv = [kv[:, :int(b + n)] for kv, b, n in zip(s.kv, s.base, spans)]
    t.check(out[:t.rows])
    assert s.plan.get_status() == 0


def test_two_handles_at_once():
    import torch
    a, b = Setup(**CASES["long"]), Setup(**CASES["tiles above 256 rows"])
    ra, rb = a.run(), b.run()
    oa, ob = torch.zeros_like(ra), torch.zeros_like(rb)
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    sa.wait_stream(torch.cuda.current_stream())
    sb.wait_stream(torch.cuda.current_stream())
    for _ in range(10):
        a.plan.attention(0, a.q, a.d_table, a.d_off, a.d_base, a.B, a.max_span, oa, group_off=a.d_group, prefix_len=a.d_prefix, G=a.G, stream=sa)
        b.plan.attention(0, b.q, b.d_table, b.d_off, b.d_base, b.B, b.max_span, ob, group_off=b.d_group, prefix_len=b.d_prefix, G=b.G, stream=sb)
    torch.cuda.synchronize()
    assert torch.equal(oa, ra) and torch.equal(ob, rb)


# ---------------------------------------------------------------- refusals

def test_host_refusals():
    import torch
    from speculative_decoding_verify_02_gb300 import SdvError, SharedAttention
    s = Setup(**CASES["prefix ends inside a page"])
    for kw in (dict(window=-1), dict(softcap=-1.0), dict(softcap=float("nan")), dict(softcap=float("inf"))):
        with pytest.raises(SdvError):
            s.run(**kw)
    with pytest.raises(SdvError):
        s.run(out=s.q)
    with pytest.raises(SdvError):
        s.plan.attention(1, s.q, s.d_table, s.d_off, s.d_base, s.B, s.max_span, s.q.clone())
    with pytest.raises(SdvError):
        s.plan.attention(0, s.q, s.d_table, s.d_off, s.d_base, s.B, s.max_span + 1, s.q.clone())
    with pytest.raises(SdvError):
        s.plan.attention(0, s.q, s.d_table, s.d_off, s.d_base, s.B, s.max_span, s.q.clone(), group_off=_i32(range(6)),
                         prefix_len=_i32([0] * 5), G=5)   # more groups than sequences
    with pytest.raises(ValueError):
        s.run(group_off=None)
    with pytest.raises(ValueError):
        s.plan.attention(0, s.q, s.d_table, s.d_off, s.d_base, s.B, s.max_span, s.q.clone(), prefix_len=s.d_prefix)
    with pytest.raises(ValueError):
        s.run(slopes=torch.ones(s.nq - 1, device="cuda"))
    with pytest.raises(ValueError):
        s.run(q=s.q.float())
    with pytest.raises(ValueError):
        s.run(out=s.q[:1].clone())
    with pytest.raises(ValueError):
        s.run(q=s.q.transpose(0, 1).contiguous().transpose(0, 1)[:, :, ::2])
    with pytest.raises(ValueError, match="pool"):
        SharedAttention(1, 8, 2, 128, n_pages=4, pool=torch.zeros(8, dtype=torch.bfloat16, device="cuda"))


def test_device_refusals():
    """A sequence that breaks the rules gives NaN rows and the status; the others keep their results."""
    import torch
    from speculative_decoding_verify_02_gb300 import SDV_ERR_ARG, SDV_ERR_CAPACITY
    s = Setup(**CASES["two groups, one without prefix"])
    ref = s.run()

    def after(code, bad, **kw):
        out = s.run(**kw)
        for b in range(s.B):
            rows = slice(s.off[b], s.off[b + 1])
            if b in bad:
                assert torch.isnan(out[rows]).all(), b
            else:
                assert torch.equal(out[rows], ref[rows]), b
        assert s.plan.get_status() == code and s.plan.get_status() == 0

    after(SDV_ERR_ARG, {2, 3, 4}, prefix_len=_i32([0, -1]))
    after(SDV_ERR_ARG, {0, 1, 2, 3, 4}, group_off=_i32([0, 2, 4]))
    after(SDV_ERR_ARG, {0, 1, 2, 3, 4}, group_off=_i32([1, 2, 5]))
    after(SDV_ERR_ARG, {0, 1, 2, 3, 4}, group_off=_i32([0, 6, 5]))
    keep = s.d_base.clone()
    s.d_base[3] = 499                        # a row before the end of the prefix
    after(SDV_ERR_ARG, {3})
    s.d_base[3] = 1 << 20
    after(SDV_ERR_CAPACITY, {3})
    s.d_base[3] = -1
    after(SDV_ERR_CAPACITY, {3})
    s.d_base.copy_(keep)
    after(0, set())


def test_spans_that_do_not_fit():
    import torch
    from speculative_decoding_verify_02_gb300 import SDV_ERR_ARG
    s = Setup(sizes=[3], prefix=[40], own=[0, 9, 3], spans=[2, 5, 3])
    ref = s.run()
    s.max_span = 4                           # the second one's is longer
    out = s.run()
    assert torch.equal(out[:2], ref[:2]) and torch.equal(out[7:], ref[7:]) and torch.isnan(out[2:7]).all()
    assert s.plan.get_status() == SDV_ERR_ARG
    s.max_span = 5
    for off in ([0, 2, 7, 99], [0, 2, 1, 4], [-4, 2, 7, 10]):
        s.d_off = _i32(off)
        s.run()
        assert s.plan.get_status() == SDV_ERR_ARG


@pytest.mark.parametrize("ps", [16, 10])
def test_pages_outside_of_the_pool_read_as_zeros(ps):
    from speculative_decoding_verify_02_gb300 import SDV_ERR_CAPACITY
    s = Setup(sizes=[2], prefix=[60], own=[0, 90], spans=[3, 2], ps=ps)
    for bad in (-1, s.pool.shape[1], 2 ** 31 - 1, -2 ** 31, -2):
        kv = [x.copy() for x in s.kv]
        for b in range(2):                   # the group's second page, and one of the second sequence's own
            kv[b][:, ps:2 * ps] = 0
        j = (60 + 90) // ps
        kv[1][:, j * ps:(j + 1) * ps] = 0
        table = s.table.copy()
        table[:, 1] = bad
        table[1, j] = bad
        s.d_table = _i32(table)
        s.check(s.run(), kv=kv)
        assert s.plan.get_status() == SDV_ERR_CAPACITY


# ---------------------------------------------------------------- values that are not finite, where a CTA does many tiles

def _bad_values(s, at, bad, window=0):
    """V of sequence b's position at[b] becomes `bad` in one dim of kv head 1: rows that see it are spoilt in that head, all
    others keep their bits."""
    import torch
    clean = s.run(window=window)
    assert torch.isfinite(clean).all()
    sees = torch.zeros(s.rows, s.nq, dtype=torch.bool, device="cuda")
    grp = s.nq // s.nkv
    for b, p in at.items():
        s.pool[s.layer, int(s.table[b, p // s.ps]), 1, 1, p % s.ps, 5] = float(bad)
        for r in range(s.off[b], s.off[b + 1]):
            pos = int(s.base[b]) + r - s.off[b]
            if p <= pos and (not window or p > pos - window):
                sees[r, grp:2 * grp] = True
    out = s.run(window=window)
    assert sees.any() and not sees.all()
    assert torch.equal(out[~sees], clean[~sees]), f"{int((out != clean).any(-1)[~sees].sum())} rows and heads of others changed"
    assert not torch.isfinite(out[sees]).all(-1).any()


@pytest.mark.parametrize("bad", [np.nan, np.inf])
@pytest.mark.parametrize("which", [(0,), (63,), range(0, 64, 3), range(64)])
def test_one_sequences_bad_value_reaches_no_other(which, bad):
    """More tiles than CTAs, of seven chunks each: a mark that outlives its tile would meet the next sequence's last chunk."""
    s = Setup(sizes=[1] * 64, prefix=[0] * 64, own=[840] * 64, spans=[8] * 64, groups=False, nq=32, nkv=8, D=64)
    _bad_values(s, {b: 840 + 3 for b in which}, bad)


@pytest.mark.parametrize("lengths", [[140], [300], [140, 270, 400], [300, 900]])
def test_bad_values_where_lengths_differ(lengths):
    B = 96
    own = [lengths[i % len(lengths)] + i % 5 for i in range(B)]
    s = Setup(sizes=[1] * B, prefix=[0] * B, own=own, spans=[4] * B, groups=False, nq=16, nkv=4, D=64)
    _bad_values(s, {b: own[b] + 2 for b in range(0, B, 2)}, np.nan)


@pytest.mark.parametrize("at", [2, 12, 40])
def test_a_bad_value_that_left_the_window(at):
    """Chunks that all rows see between two that they do not: rows behind whose window the bad value lies keep their results, in
    the last chunk too. Of 60 sequences, five chunks each."""
    s = Setup(sizes=[1] * 60, prefix=[0] * 60, own=[515] * 60, spans=[60] * 60, groups=False, nq=4, nkv=4, D=64)
    _bad_values(s, {b: 515 - 510 + 1 + at for b in range(0, 60, 2)}, np.nan, window=510)


@pytest.mark.parametrize("spans", [[8, 40], [40, 8, 8], [72, 1], [33, 1, 64]])
@pytest.mark.parametrize("own", [[100], [300, 130], [700, 60, 300]])
def test_bad_values_where_narrow_and_wide_tiles_take_turns(spans, own):
    """Tiles of up to 128 rows, of which two warpgroups take every other chunk, and of more, whose V both look at."""
    B = 72
    n, o = [spans[i % len(spans)] for i in range(B)], [own[i % len(own)] + i % 3 for i in range(B)]
    s = Setup(sizes=[1] * B, prefix=[0] * B, own=o, spans=n, groups=False, nq=16, nkv=4, D=64)
    for at in (0, 1):
        _bad_values(s, {b: o[b] + min(at, n[b] - 1) for b in range(at, B, 2)}, np.nan)
        s.pool.nan_to_num_(0.5)


@pytest.mark.parametrize("own", [40, 260])
def test_bad_values_of_tiles_that_both_warpgroups_look_at(own):
    """300 rows a head: a wide tile, then one of 44, an odd number of chunks each, so that the warpgroups' steps come apart. Every
    row that sees a bad V is spoilt in every head."""
    import torch
    s = Setup(sizes=[1] * 60, prefix=[0] * 60, own=[own] * 60, spans=[75] * 60, groups=False, nq=32, nkv=8, D=64)
    clean = s.run()
    for b in range(60):
        p = own + 5 + b
        s.pool[0, int(s.table[b, p // s.ps]), 1, :, p % s.ps, b] = float("nan")
    out, sees = s.run(), torch.zeros(s.rows, dtype=torch.bool, device="cuda")
    for b in range(60):
        sees[75 * b + 5 + b:75 * b + 75] = True
    assert torch.equal(out[~sees], clean[~sees])
    assert not torch.isfinite(out[sees]).all(-1).any()


def test_bad_values_behind_a_shared_prefix():
    B = 48
    s = Setup(sizes=[30, 18], prefix=[400, 150], own=[i % 9 * 31 for i in range(B)], spans=[1 + i % 7 * 6 for i in range(B)], nq=16, nkv=4, D=64)
    _bad_values(s, {b: int(s.base[b]) + min(2, int(s.spans[b]) - 1) for b in range(1, B, 3)}, np.nan)


def test_many_tiles_of_one_chunk():
    """A CTA's queries follow one another as fast as they can: no warp may miss those it waits for. No wait runs out, the same bits."""
    import torch
    s = Setup(sizes=[1] * 250, prefix=[0] * 250, own=[i % 90 for i in range(250)], spans=[1 + i % 3 for i in range(250)], groups=False,
              nq=16, nkv=8, D=128)
    ref = s.run()
    s.check(ref)
    out = torch.zeros_like(ref)
    for _ in range(200):
        s.plan.attention(0, s.q, s.d_table, s.d_off, s.d_base, s.B, s.max_span, out)
    assert torch.equal(out, ref) and s.plan.get_status() == 0


# ---------------------------------------------------------------- caps of any size

def _check_cap(s, out, cap, window=0):
    """As Setup.check with a cap's own error. Up to 64, cap (1 - 2 / (1 + e)): half of e's relative error, 2^-22 and three roundings,
    2^-22 of the quotient, below 1, and a rounding: 2^-21 of the cap covers them. Above, 2^-21.3 of the score and its exponent's
    roundings: 2^-20 |z|, however large the cap."""
    q = s.q.double().cpu().numpy()
    o = out.double().cpu().numpy()
    grp = s.nq // s.nkv
    for b in range(s.B):
        rows, pos = slice(s.off[b], s.off[b + 1]), s.base[b] + np.arange(s.spans[b])
        k, v = s.kv[b].astype(np.float64)
        for h in range(s.nq):
            z = oracle.scores(q[rows, h], k[:, h // grp], pos, window, float(np.float32(cap)), 0.0)
            ref = oracle.attend(z, v[:, h // grp])
            seen = z > -np.inf
            w = np.exp(z - z.max(-1, keepdims=True))
            w /= w.sum(-1, keepdims=True)
            mag = np.where(seen, np.abs(q[rows, h]) @ np.abs(k[:, h // grp]).T, 0).max() / np.sqrt(s.D)
            top = np.abs(np.where(seen, z, 0)).max()
            A = np.stack([w[i, m] @ np.abs(v[m, h // grp]) for i, m in enumerate(seen)])
            off = 2.0 ** -21 * cap if cap <= 64 else 2.0 ** -20 * top
            e = (s.D + 2) * 2.0 ** -24 * mag + 3 * 2.0 ** -24 * 1.45 * top + off + 2.0 ** -22 + 2.0 ** -16
            tol = (2 * e + 2 * len(k) * 2.0 ** -24) * A + s.eps / 2 * np.abs(ref) * 1.01 + 2.0 ** -24
            d = np.abs(o[rows, h] - ref)
            assert np.isfinite(o[rows, h]).all(), f"sequence {b} head {h}"
            assert (d <= tol).all(), f"sequence {b} head {h}: {d.max()} over {tol.flat[d.argmax()]}"


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("cap", [0.3, 5.0, 50.0, 64.0, 65.0, 1e3, 1e4, 1e5, 1e6, 1e8, 1e20, 1e30, 3e38])
@pytest.mark.parametrize("name", ["prefix ends inside a page", "one kv head"])
def test_caps_of_any_size(name, cap, dtype):
    s = Setup(dtype=dtype, **CASES[name])
    _check_cap(s, s.run(softcap=cap), cap)


@pytest.mark.parametrize("cap", [20.0, 60.0, 1e3])
def test_caps_of_scores_around_them(cap):
    """Scores from far below the cap to far above it, in one row."""
    s = Setup(**CASES["two groups, one without prefix"])
    s.q *= 12
    _check_cap(s, s.run(softcap=cap), cap)


def test_a_large_cap_is_none():
    """At a cap of 10^6 tanh takes a score's square times 3 10^-13 of it: the results are those without a cap, to a rounding."""
    import torch
    s = Setup(**CASES["tiles above 256 rows"])
    a, b = s.run().float(), s.run(softcap=1e6).float()
    assert (a - b).abs().max() <= 2 * s.eps * a.abs().max() and torch.isfinite(b).all()


@pytest.mark.parametrize("cap", [1e-3, 1e-20, 1.2e-38, 1e-40, 1.5e-45])
def test_tiny_caps(cap):
    """All scores equal but for the cap: a mean of V, also of rows whose score is zero."""
    s = Setup(**CASES["prefix ends inside a page"])
    s.q[1] = 0
    _check_cap(s, s.run(softcap=cap), cap)
