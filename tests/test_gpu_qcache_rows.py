"""Rows of the 8-bit cache's attention: what a value that is not finite spoils, how near the result is to 64 bits when only
the roundings that the kernel makes are counted, that a call repeats itself, and caches whose limit is far above the call."""
import numpy as np
import pytest

from tests.test_gpu_qcache import Setup, _i32

pytestmark = pytest.mark.gpu

# heads, kv heads, dim, lengths, spans, window: tiles of 16, 32 and 64 rows; one part, parts that a cluster joins, parts
# that a kernel joins
SHAPES = [
    (4, 2, 64, [40], [3], 0),
    (32, 8, 128, [848], [4], 0),
    (32, 8, 128, [848], [8], 0),
    (8, 1, 128, [700], [7], 300),
    (32, 8, 128, [900], [16], 0),
    (16, 2, 64, [1100], [8], 0),
    (4, 2, 64, [5000], [2], 0),
    (16, 4, 64, [9000, 300], [6, 3], 0),
    (16, 1, 128, [20000], [9], 0),
]


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("nq, nkv, D, lengths, spans, window", SHAPES)
def test_a_value_that_is_not_finite_spoils_its_own_row_and_head(nq, nkv, D, lengths, spans, window, dtype):
    """Every other row and head keeps the bits that it has beside a zero in that place; those two give NaN throughout."""
    import torch
    s = Setup(nq, nkv, D, 16, 16, lengths, spans, seed=nq + D)
    s.fill()
    q, _ = s.values((s.rows, nq, D), dtype, 0.5)
    places = [(0, 0, 0), (s.rows - 1, nq - 1, D - 1), (s.rows // 2, nq // 2, D // 3)]
    for r, h, d in places:
        q[r, h, d] = 0
    clean, out = torch.empty_like(q), torch.empty_like(q)
    s.cache.attention(1, q, *s.args(), clean, window=window)
    assert bool(clean.isfinite().all())
    for bad in (np.nan, np.inf, -np.inf):
        for r, h, d in places:
            x = q.clone()
            x[r, h, d] = bad
            s.cache.attention(1, x, *s.args(), out, window=window)
            assert bool(out[r, h].isnan().all())
            rest = torch.ones(s.rows, nq, dtype=torch.bool, device="cuda")
            rest[r, h] = False
            assert torch.equal(out[rest], clean[rest])
    x = torch.full_like(q, float("nan"))
    s.cache.attention(1, x, *s.args(), out, window=window)
    assert bool(out.isnan().all()) and s.cache.get_status() == 0


def _reference(s, b, q, window):
    """(result, bound of the products' error, bound of the other errors' factor) of the rows of sequence b in 64 bits.

    With s the scores in units of log 2, w_t = s_t + log2 of key t's V scale and M the row's largest w, key t weighs
    x_t = 2^(w_t - M) <= 1 on its bare codes c_t and the result is 2^M sum x_t c_t / sum 2^s_t. The kernel's reference is
    M or less than one below it, and less for the chunks and parts before and beside the largest. It rounds 64 x 2^(M - ref)
    to fp16, half a step of 2^-11 relative (2^-25 absolute where that is no normal number), and its three planes hold that
    down to 2^-20: an error of 2^-11 x_t + 2^-26 + 2^-31 of 2^M |c_t|."""
    k, v = s.pool.rows(s.table[b], 0, s.lengths[b] + s.spans[b])
    keys = len(k)
    slots = np.arange(keys)
    pages = np.asarray(s.table[b])[slots // s.ps]
    vscale = s.pool.scale[pages, 1][np.arange(keys), :, (slots % s.ps) // s.sb]     # [keys, heads]
    S, nq, D = q.shape
    grp = nq // s.nkv
    o, err, mag, top = (np.zeros((S, nq, D)) for _ in range(4))
    for i in range(S):
        pos = s.lengths[b] + i
        lo = max(0, pos - window + 1) if window else 0
        for h in range(nq):
            kk, vv, vs = k[lo:pos + 1, h // grp], v[lo:pos + 1, h // grp], vscale[lo:pos + 1, h // grp]
            z = kk @ q[i, h] / np.sqrt(D) * np.log2(np.e)
            w = z + np.log2(vs)
            M = w.max()
            x, c = np.exp2(w - M), vv / vs[:, None]
            l = np.exp2(z - M).sum()
            o[i, h] = (x @ c) / l
            err[i, h] = (2.0 ** -11 * x + 2.0 ** -26 + 2.0 ** -31) @ np.abs(c) / l
            mag[i, h] = (x @ np.abs(c)) / l
            top[i, h] = (np.abs(kk) @ np.abs(q[i, h])).max() / np.sqrt(D)
    return o, err, mag, top


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("nq, nkv, D, lengths, spans, window", SHAPES)
def test_only_the_roundings_that_the_kernel_makes(nq, nkv, D, lengths, spans, window, dtype):
    """The result's own rounding is half a step of its type (bf16 2^-8, fp16 2^-11 of it, 2^-25 where fp16 has no normal
    number); the products' is _reference's, alike for both types. Scores: D products summed in fp32, each addition off by
    2^-23 of top = max sum |q k| / sqrt(D) at most, scaling and the exponent by 2^-22 of it, so (D + 8) 2^-23 top in
    natural units, on a weight and on the sum; the sums of positive terms 2^-16 (2^8 roundings of 2^-24) of sum p |v|."""
    s = Setup(nq, nkv, D, 16, 4, lengths, spans, seed=3 * nq + D)
    s.fill()
    qt, q = s.values((s.rows, nq, D), dtype, 0.3)
    out = qt.clone()
    s.cache.attention(1, qt, *s.args(), out, window=window)
    got = out.double().cpu().numpy()
    half, tiny = {"bfloat16": (2.0 ** -8, 0.0), "float16": (2.0 ** -11, 2.0 ** -25)}[dtype]
    for b in range(s.B):
        r = slice(s.off[b], s.off[b + 1])
        o, err, mag, top = _reference(s, b, q[r], window)
        other = err + mag * (2 * np.expm1((D + 8) * 2.0 ** -23 * top) + 2.0 ** -16)
        tol = half * (np.abs(o) + other) + tiny + other
        worst = float((np.abs(got[r] - o) / tol).max())
        print(f"worst error / tolerance {worst:.3f}")
        assert worst <= 1
    assert s.cache.get_status() == 0


@pytest.mark.parametrize("nq, nkv, D, lengths, spans, window", SHAPES + [(8, 2, 64, [70 * i + 3 for i in range(40)], [2] * 40, 0)])
def test_a_call_repeats_itself(nq, nkv, D, lengths, spans, window):
    """Which CTA takes which unit, and when, changes no bit of a result."""
    import torch
    s = Setup(nq, nkv, D, 16, 16, lengths, spans, seed=nq)
    s.fill()
    q, _ = s.values((s.rows, nq, D), "bfloat16", 0.5)
    first = torch.empty_like(q)
    s.cache.attention(1, q, *s.args(), first, window=window)
    for _ in range(20):
        out = torch.empty_like(q)
        s.cache.attention(1, q, *s.args(), out, window=window)
        assert torch.equal(out, first)


@pytest.mark.parametrize("limit", [32768, 131072])
@pytest.mark.parametrize("nq, nkv, D, lengths, spans", [
    (4, 2, 64, [0], [1]), (16, 2, 64, [848], [8]), (8, 1, 128, [300], [1]), (16, 1, 64, [5, 1000, 0, 127], [9, 1, 0, 4]),
    (4, 2, 64, [60 * i for i in range(16)], [3] * 16)])
def test_caches_whose_limit_is_far_above_the_call(nq, nkv, D, lengths, spans, limit):
    """The number of parts follows the cache's limit: sequences of a few chunks in a cache of many."""
    import torch
    ctx = max(l + n for l, n in zip(lengths, spans))
    tight = Setup(nq, nkv, D, 16, 16, lengths, spans, seed=7)
    tight.fill()
    q, q64 = tight.values((tight.rows, nq, D), "bfloat16", 0.3)
    from speculative_decoding_verify_02_gb300 import QuantCache
    cache = QuantCache(1, nq, nkv, D, page_size=16, n_pages=tight.n_pages, max_batch=tight.B, max_rows=max(tight.rows, max(spans)),
                       max_span=max(spans), max_context=limit, scale_block=16)
    cache.codes[0].copy_(tight.cache.codes[1])
    cache.scales[0].copy_(tight.cache.scales[1])
    table = torch.full((tight.B, limit // 16), -1, dtype=torch.int32, device="cuda")
    table[:, :tight.table.shape[1]] = tight.d_table
    out = torch.full_like(q, 5.0)
    cache.attention(0, q, table, tight.d_off, tight.d_base, tight.B, max(spans), out)
    got = out.double().cpu().numpy()
    for b in range(tight.B):
        if spans[b]:
            r = slice(tight.off[b], tight.off[b + 1])
            o, err, mag, top = _reference(tight, b, q64[r], 0)
            other = err + mag * (2 * np.expm1((D + 8) * 2.0 ** -23 * top) + 2.0 ** -16)
            assert (np.abs(got[r] - o) <= 2.0 ** -8 * (np.abs(o) + other) + other).all()
    assert cache.get_status() == 0 and ctx <= limit


def test_cache_made_and_used_on_a_side_stream():
    """A cache that a side stream clears, writes, reads and attends on gives what the current stream's gives."""
    import torch
    from speculative_decoding_verify_02_gb300 import QuantCache
    s = Setup(4, 2, 64, 16, 16, [0], [40], seed=1)
    kv, _ = s.values((s.rows, 2, 2, 64), "bfloat16")
    q, _ = s.values((s.rows, 4, 64), "bfloat16")
    side, results = torch.cuda.Stream(), []
    for stream in (None, side):
        torch.cuda.synchronize()
        cache = QuantCache(2, 4, 2, 64, n_pages=s.n_pages, max_rows=s.rows, max_span=s.rows, max_context=64, stream=stream)
        table = _i32(np.resize(s.table, (1, 4)))
        k, v, out = torch.zeros_like(kv[:, 0]), torch.zeros_like(kv[:, 1]), torch.zeros_like(q)
        torch.cuda.synchronize()
        cache.write(1, kv[:, 0], kv[:, 1], table, s.d_off, s.d_base, 1, s.rows, stream=stream)
        cache.read(1, table, s.d_off, s.d_base, 1, s.rows, k, v, stream=stream)
        cache.attention(1, q, table, s.d_off, s.d_base, 1, s.rows, out, stream=stream)
        torch.cuda.synchronize()
        assert cache.get_status() == 0 and int(cache.codes[0].sum()) == 0
        results.append((k, v, out))
    for a, b in zip(*results):
        assert torch.equal(a, b) and bool(a.ne(0).any())
