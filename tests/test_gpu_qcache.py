"""The 8-bit cache on the GPU against the float64 oracle (oracle/quant.py): codes and scales exactly, attention
within tolerances derived below."""
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
    """A cache with sequences of the given lengths (before the span) and spans, pages in a random order."""

    def __init__(self, nq, nkv, D, ps, sb, lengths, spans, seed=0, max_span=None, layers=2, layer=1, spare=3, room=0):
        from speculative_decoding_verify_02_gb300 import QuantCache
        self.rng = np.random.default_rng(seed)
        self.nq, self.nkv, self.D, self.ps, self.sb, self.layer = nq, nkv, D, ps, sb, layer
        self.lengths, self.spans, self.B = list(lengths), list(spans), len(lengths)
        self.max_span = max_span or max(spans)
        ctx = max(l + s for l, s in zip(lengths, spans)) + room
        ctx = max(ctx, self.max_span)
        per = -(-ctx // ps)
        self.n_pages = self.B * per + spare
        self.table = self.rng.permutation(self.n_pages)[:self.B * per].reshape(self.B, per)
        self.off = np.concatenate([[0], np.cumsum(spans)])
        self.rows = int(self.off[-1])
        self.cache = QuantCache(layers, nq, nkv, D, page_size=ps, n_pages=self.n_pages, max_batch=self.B,
                                max_rows=max(self.rows, self.max_span), max_span=self.max_span, max_context=ctx,
                                scale_block=sb)
        self.pool = oracle.QuantPool(self.n_pages, nkv, ps, D, sb)
        self.d_table, self.d_off, self.d_base = _i32(self.table), _i32(self.off), _i32(self.lengths)

    def fill(self):
        """Random contents of the whole layer: codes without NaN, scales of several powers of two."""
        c = self.cache
        codes = self.rng.integers(0, 256, tuple(c.codes[self.layer].shape), dtype=np.uint8)
        codes[(codes & 127) == 127] = 0x30
        scales = np.exp2(self.rng.integers(-10, -6, tuple(c.scales[self.layer].shape))).astype(np.float32)
        c.codes[self.layer].copy_(_dev(codes))
        c.scales[self.layer].copy_(_dev(scales))
        self.pool.val, self.pool.scale = oracle.code_values(codes), scales.astype(np.float64)

    def values(self, shape, dtype, spread=1.0):
        """Rows as a device tensor of `dtype` and as the float64 values it holds."""
        import torch
        x = self.rng.normal(size=shape) * np.exp(spread * self.rng.normal(size=shape[:-1] + (1,)))
        t = _dev(x.astype(np.float32)).to(getattr(torch, dtype))
        return t, t.double().cpu().numpy()

    def args(self):
        return self.d_table, self.d_off, self.d_base, self.B, self.max_span

    def check_pool(self):
        codes = self.cache.codes[self.layer].cpu().numpy()
        np.testing.assert_array_equal(self.cache.scales[self.layer].double().cpu().numpy(), self.pool.scale)
        np.testing.assert_array_equal(oracle.code_values(codes), self.pool.val)


WRITES = [
    # nkv, D, page, block, lengths, spans
    (1, 64, 16, 16, [0], [1]),
    (2, 128, 16, 16, [5, 31, 0, 16], [7, 2, 40, 0]),
    (8, 128, 16, 4, [848], [8]),
    (3, 64, 24, 8, [23, 24, 25], [1, 49, 17]),
    (2, 128, 16, 1, [3, 100], [9, 17]),
    (2, 64, 1, 1, [3, 0], [9, 4]),
    (5, 128, 128, 128, [60, 127], [130, 1]),
    (1, 128, 7, 7, [6, 2], [20, 3]),
    (2, 64, 16, 2, [31, 7, 100], [70, 1, 33]),
    (2, 128, 4, 2, [13, 6], [37, 2]),
    (1, 64, 8, 8, [5, 35], [45, 60]),
    (2, 128, 24, 8, [13, 22], [30, 5]),
    (1, 128, 12, 4, [6, 2], [40, 3]),
    (1, 64, 12, 12, [6, 30], [40, 7]),
]


@pytest.mark.parametrize("dtype", ["bfloat16", "float16", "float32"])
@pytest.mark.parametrize("nkv, D, ps, sb, lengths, spans", WRITES)
def test_write_and_read_back(nkv, D, ps, sb, lengths, spans, dtype):
    """Codes and scales of two writes (the second starting inside blocks that the first left) equal the oracle's
    exactly, everything else untouched; the rows read back are code * scale rounded once."""
    import torch
    s = Setup(nkv, nkv, D, ps, sb, lengths, spans, seed=len(spans) + sb, room=max(spans))
    s.fill()
    finite = True
    for again in range(2):
        kt, k = s.values((s.rows, nkv, D), dtype)
        vt, v = s.values((s.rows, nkv, D), dtype, 3.0)
        finite = finite and bool(np.isfinite(v).all())                # fp16 may overflow at this spread
        s.cache.write(s.layer, kt, vt, *s.args())
        for b in range(s.B):
            r = slice(s.off[b], s.off[b + 1])
            s.pool.write(s.table[b], s.lengths[b], k[r], v[r])
        s.check_pool()
        ko, vo = torch.full_like(kt, 7.0), torch.full_like(vt, 7.0)
        s.cache.read(s.layer, *s.args(), ko, vo)
        for b in range(s.B):
            if spans[b]:
                rk, rv = s.pool.rows(s.table[b], s.lengths[b], s.lengths[b] + spans[b])
                for got, ref in ((ko, rk), (vo, rv)):
                    ref = torch.from_numpy(ref).float().to(kt.dtype)
                    assert torch.equal(got[s.off[b]:s.off[b + 1]].cpu(), ref)
        # the next write begins one row into this one: lower rows live, later rows overwritten
        s.lengths = [l + 1 if n > 1 else l for l, n in zip(s.lengths, spans)]
        s.d_base = _i32(s.lengths)
    assert s.cache.get_status() == (0 if finite else -4)
    assert int(s.cache.codes[0].sum()) == 0 and float(s.cache.scales[0].sum()) == 0  # the other layer


def test_strided_and_unaligned_rows():
    """K and V inside one projection row, and rows that start off a 16-byte boundary, give the same codes."""
    import torch
    s = Setup(2, 2, 64, 16, 8, [10, 3], [5, 12], seed=5)
    wide, ref = s.values((s.rows, 9, 64), "bfloat16")
    s.cache.write(1, wide[:, 2:4], wide[:, 7:9], *s.args())
    for b in range(2):
        r = slice(s.off[b], s.off[b + 1])
        s.pool.write(s.table[b], s.lengths[b], ref[r, 2:4], ref[r, 7:9])
    s.check_pool()
    flat = torch.zeros(s.rows * 259 + 3, dtype=torch.bfloat16, device="cuda")
    odd = flat[1:1 + s.rows * 259].view(s.rows, 259)
    odd[:, :128] = wide[:, 2:4].reshape(s.rows, 128)
    odd[:, 129:257] = wide[:, 7:9].reshape(s.rows, 128)
    k, v = odd[:, :128].unflatten(1, (2, 64)), odd[:, 129:257].unflatten(1, (2, 64))
    s.cache.codes.zero_()
    s.cache.scales.zero_()
    s.cache.write(1, k, v, *s.args())
    s.check_pool()
    before = flat.clone()
    k.zero_(), v.zero_()
    s.cache.read(1, *s.args(), k, v)
    rest = torch.ones_like(flat, dtype=torch.bool)
    rest[1:1 + s.rows * 259].view(s.rows, 259)[:, :128] = False
    rest[1:1 + s.rows * 259].view(s.rows, 259)[:, 129:257] = False
    assert torch.equal(flat[rest], before[rest])                   # between the rows nothing is written
    for b in range(2):
        rk, rv = s.pool.rows(s.table[b], s.lengths[b], s.lengths[b] + s.spans[b])
        assert torch.equal(k[s.off[b]:s.off[b + 1]].double().cpu(), torch.from_numpy(rk).bfloat16().double())
        assert torch.equal(v[s.off[b]:s.off[b + 1]].double().cpu(), torch.from_numpy(rv).bfloat16().double())


def test_write_of_extremes():
    """Zeros, the largest and the smallest magnitudes; NaN and infinities are stored finite, do not set the scale and
    raise the status."""
    s = Setup(1, 1, 64, 8, 8, [0], [8], layers=1, layer=0)
    x = np.zeros((8, 1, 64), dtype=np.float32)
    x[1, 0, :4] = [3.0e38, 1e-45, 1.0, -3.0e38]
    v = np.full((8, 1, 64), 1e-45, dtype=np.float32)
    s.cache.write(0, _dev(x), _dev(v), *s.args())
    s.pool.write(s.table[0], 0, x, v)
    s.check_pool()
    assert s.cache.get_status() == 0
    x = s.rng.normal(size=(8, 1, 64)).astype(np.float32)
    x[2, 0, 5], x[3, 0, 6], x[4, 0, 7] = np.nan, np.inf, -np.inf
    s.cache.write(0, _dev(x), _dev(np.full_like(x, np.nan)), *s.args())
    s.pool.write(s.table[0], 0, x, np.full_like(x, np.nan))
    s.check_pool()
    assert s.cache.get_status() == -4 and s.cache.get_status() == 0


def test_scale_block_one_forgets_rejected_drafts():
    """With a scale for every token, writing drafts, rewinding and writing other rows leaves the same codes and scales
    as never having drafted; with larger blocks a rejected row may leave a larger scale, never a smaller one."""
    import torch
    for sb in (1, 16):
        pools = []
        for drafted in (True, False):
            s = Setup(2, 2, 64, 16, sb, [20], [6], seed=1)
            kv, _ = s.values((6, 2, 2, 64), "bfloat16")
            if drafted:
                big = kv * 50
                s.cache.write(1, big[:, 0], big[:, 1], *s.args())
            s.cache.write(1, kv[:, 0], kv[:, 1], *s.args())
            pools.append((s.cache.codes.clone(), s.cache.scales.clone()))
        if sb == 1:
            assert torch.equal(pools[0][0], pools[1][0]) and torch.equal(pools[0][1], pools[1][1])
        else:
            assert (pools[0][1] >= pools[1][1]).all()


# ------------------------------------------------------------------ attention
def _tolerance(ref, mag, top, D, dtype):
    """|o - ref| of one element. The output is rounded once: eps / 2 of it, and the smallest subnormal's half. The
    probabilities are rounded to the width that their type's products carry: at most 2^-8 of each for bf16 outputs and
    2^-11 for fp16 ones, so that much of sum p |v|. A score is a sum of D products in fp32, each addition off by at most
    2^-23 of the partial sums' bound sum |q_d k_d| / sqrt(D) = top, and scaling and the exponent's argument by 2^-22 of
    it: (D + 8) 2^-23 top, natural units; a probability and the sum it is divided by each move by e^that - 1. Sums over
    the keys are fp32 sums of positive terms in any order: 2^-16 of sum p |v| covers 2^8 roundings in a row of 2^-24."""
    eps = {"bfloat16": 2.0 ** -8, "float16": 2.0 ** -11}[dtype]
    tiny = {"bfloat16": 0.0, "float16": 2.0 ** -25}[dtype]
    ds = np.expm1((D + 8) * 2.0 ** -23 * top)
    return eps * np.abs(ref) + tiny + mag * (eps + 2 * ds + 2.0 ** -16)


def _check_attention(s, dtype, window=0, spread=0.5, q_tensor=None):
    import torch
    qt, q = s.values((s.rows, s.nq, s.D), dtype, spread)
    if q_tensor is not None:
        q_tensor.copy_(qt)
        qt = q_tensor
    out = torch.full((s.rows + 2, s.nq, s.D), 5.0, dtype=qt.dtype, device="cuda")
    s.cache.attention(s.layer, qt, *s.args(), out[:s.rows], window=window)
    got = out.double().cpu().numpy()
    assert (got[s.rows:] == 5.0).all()                              # rows behind the last sequence
    worst = 0.0
    for b in range(s.B):
        if s.spans[b]:
            r = slice(s.off[b], s.off[b + 1])
            ref, mag, top = s.pool.attention(s.table[b], s.lengths[b], q[r], window)
            tol = _tolerance(ref, mag, top, s.D, dtype)
            err = np.abs(got[r] - ref)
            assert np.isfinite(got[r]).all()
            worst = max(worst, float((err / np.maximum(tol, 1e-300)).max()))
            assert (err <= tol).all(), (b, float((err / tol).max()), np.argwhere(err > tol)[:5].tolist())
    return out[:s.rows], worst


ATTENTION = [
    # nq, nkv, D, page, block, lengths, spans, window
    (4, 1, 128, 16, 16, [0], [1], 0),                                # one token, one key
    (32, 8, 128, 16, 16, [848], [8], 0),
    (32, 8, 128, 16, 4, [848], [1], 0),
    (4, 2, 64, 16, 16, [126, 127, 128, 129, 255, 0], [1, 2, 1, 3, 1, 5], 0),
    (6, 3, 64, 24, 8, [500, 77, 0, 1000], [5, 0, 3, 8], 0),          # an odd page, an empty span
    (12, 2, 64, 24, 8, [700, 1300], [5, 9], 256),                    # window
    (8, 8, 128, 7, 7, [300, 41], [4, 17], 1),                        # a window of one position
    (8, 2, 128, 1, 1, [130, 64], [3, 2], 100),                       # pages of one token
    (16, 1, 128, 128, 128, [1000, 3], [17, 9], 0),                   # many rows a kv head
    (5, 5, 64, 16, 16, [40, 200], [60, 33], 0),                      # spans longer than their prefix
    (40, 8, 128, 32, 16, [2000], [13], 0),                           # five heads a kv head
    (32, 8, 64, 24, 8, [1100, 1150], [14, 9], 0),                    # tiles of 64 rows, more clusters than fit at once
    (16, 2, 64, 16, 16, [1100], [8], 0),                             # tiles of 64 rows, clusters
    (32, 8, 128, 16, 16, [4090], [8], 0),
    (128, 1, 128, 16, 16, [200], [1], 0),                            # more heads than a tile
]


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("nq, nkv, D, ps, sb, lengths, spans, window", ATTENTION)
def test_attention_matches_oracle(nq, nkv, D, ps, sb, lengths, spans, window, dtype):
    s = Setup(nq, nkv, D, ps, sb, lengths, spans, seed=nq + D + sum(lengths))
    s.fill()
    _, worst = _check_attention(s, dtype, window)
    assert s.cache.get_status() == 0
    print(f"worst error / tolerance {worst:.3f}")


@pytest.mark.parametrize("B, nq, nkv, longest, window", [(256, 4, 2, 200, 0), (20, 16, 16, 700, 0), (33, 40, 20, 300, 50)])
def test_attention_of_many_sequences(B, nq, nkv, longest, window):
    """More units than the GPU holds at once: the CTAs take turns, up to 32 sequences by length."""
    rng = np.random.default_rng(B)
    s = Setup(nq, nkv, 64, 16, 16, rng.integers(0, longest, B).tolist(), rng.integers(0, 3, B).tolist(), seed=B)
    s.fill()
    for dtype in ("bfloat16", "float16"):
        _check_attention(s, dtype, window)
    assert s.cache.get_status() == 0


def test_attention_of_peaked_and_flat_rows():
    """Scores spread over hundreds of units (one key takes all), rows of zeros (all keys alike), and a long flat tail
    under one large score."""
    import torch
    s = Setup(8, 2, 128, 16, 16, [3000], [4], seed=9)
    s.fill()
    _check_attention(s, "bfloat16", spread=2.0)
    qt = torch.zeros(4, 8, 128, dtype=torch.bfloat16, device="cuda")
    out = torch.empty_like(qt)
    s.cache.attention(s.layer, qt, *s.args(), out)
    ref, mag, top = s.pool.attention(s.table[0], 3000, np.zeros((4, 8, 128)))
    assert (np.abs(out.double().cpu().numpy() - ref) <= _tolerance(ref, mag, top, 128, "bfloat16")).all()
    # a tail of 20,000 equal keys 11 units (about 2^-16) under one: together a quarter of the weight
    for dtype in ("bfloat16", "float16"):
        t = Setup(1, 1, 64, 16, 16, [20000], [1], seed=2)
        codes = np.zeros((t.n_pages, 2, 1, 16, 64), dtype=np.uint8)
        codes[:, 1] = 0x38                                           # values 1.0
        codes[:, 0, 0, :, 0] = 0x38
        page, slot = t.table[0, 137 // 16], 137 % 16
        codes[page, 0, 0, slot, 0] = 0x60                            # this key: 64
        codes[page, 1, 0, slot] = 0xb8                               # and its value -1
        t.cache.codes[1].copy_(_dev(codes))
        t.cache.scales[1].fill_(1.0)
        t.pool.val, t.pool.scale = oracle.code_values(codes), np.ones_like(t.pool.scale)
        q = torch.zeros(1, 1, 64, dtype=getattr(torch, dtype), device="cuda")
        q[0, 0, 0] = 11.0 * 8 / 63                                   # 63 units of q_0 / 8 apart
        out = torch.empty_like(q)
        t.cache.attention(1, q, *t.args(), out)
        ref, mag, top = t.pool.attention(t.table[0], 20000, q.double().cpu().numpy())
        assert (np.abs(out.double().cpu().numpy() - ref) <= _tolerance(ref, mag, top, 64, dtype)).all()


@pytest.mark.parametrize("nq, nkv, length, span", [(16, 1, 1500, 9), (16, 4, 1500, 6), (8, 4, 1500, 2)])
@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
def test_attention_whose_maximum_keeps_growing(nq, nkv, length, span, dtype):
    """Keys that grow along the sequence, in tiles of 64, 32 and 16 rows: the references move from chunk to chunk."""
    s = Setup(nq, nkv, 128, 16, 16, [length], [span], seed=21)
    s.fill()
    for p, page in enumerate(s.table[0]):
        s.pool.scale[page, 0] = 2.0 ** -12 * (1 + p // 8)
    s.cache.scales[1].copy_(_dev(s.pool.scale.astype(np.float32)))
    _check_attention(s, dtype, spread=0.5)
    s.cache.scales[1].copy_(_dev((s.pool.scale * 8).astype(np.float32)))
    s.pool.scale = s.pool.scale * 8
    _check_attention(s, dtype, spread=0.5)


def test_attention_scales_far_apart():
    """Blocks whose scales differ by 2^40 in one sequence, and scales that are no powers of two."""
    s = Setup(4, 2, 64, 16, 4, [300], [3], seed=4)
    s.fill()
    scales = s.pool.scale * np.exp2(s.rng.integers(-30, 10, s.pool.scale.shape))
    scales[:, 0] = s.pool.scale[:, 0] * 1.37
    s.cache.scales[1].copy_(_dev(scales.astype(np.float32)))
    s.pool.scale = scales.astype(np.float32).astype(np.float64)
    _check_attention(s, "bfloat16")


@pytest.mark.parametrize("length, zeros", [(1000, 1000), (1000, 700), (40000, 39000)])
@pytest.mark.parametrize("scale", [2.0 ** -126, 0.0])
def test_attention_after_keys_without_a_value(length, zeros, scale):
    """Long runs of keys whose V rows are all zero: they weigh like any other key, with scores up to hundreds of units."""
    s = Setup(4, 2, 64, 16, 16, [length], [2], seed=14)
    s.fill()
    for p in range(zeros // 16):
        page = int(s.table[0, p])
        s.cache.codes[1, page, 1] = 0
        s.cache.scales[1, page, 1] = scale
        s.pool.val[page, 1], s.pool.scale[page, 1] = 0.0, scale
    _check_attention(s, "bfloat16", spread=0.5)
    _check_attention(s, "float16", spread=2.0)


@pytest.mark.parametrize("ps, window", [(1, 5), (4, 130), (16, 20), (16, 300), (7, 40)])
def test_pages_before_the_window_may_be_gone(ps, window):
    """A sliding window's caller gives old pages back: their entries are -1, their contents anybody's."""
    s = Setup(4, 2, 64, ps, ps, [700, 129], [3, 2], seed=15)
    s.fill()
    for b in range(s.B):
        gone = max(0, s.lengths[b] - window + 1) // ps
        s.table[b, :gone] = -1
    s.d_table = _i32(s.table)
    _check_attention(s, "bfloat16", window)
    assert s.cache.get_status() == 0


def test_attention_strides_and_second_device_buffers():
    """q inside a fused projection's rows and off a 16-byte boundary; the same results as dense rows."""
    import torch
    s = Setup(4, 2, 64, 16, 16, [200, 33], [3, 4], seed=6)
    s.fill()
    wide = torch.zeros(s.rows * 515 + 1, dtype=torch.bfloat16, device="cuda")[1:].view(s.rows, 515)
    strided = wide[:, 130:386].unflatten(1, (4, 64))
    out, _ = _check_attention(s, "bfloat16", q_tensor=strided)
    dense = torch.empty(s.rows, 4, 64, dtype=torch.bfloat16, device="cuda")
    s.cache.attention(1, strided.contiguous(), *s.args(), dense)
    assert torch.equal(dense, out)
    odd = torch.zeros(s.rows * 257 + 1, dtype=torch.bfloat16, device="cuda")[1:].view(s.rows, 257)[:, :256].unflatten(1, (4, 64))
    s.cache.attention(1, strided, *s.args(), odd)
    assert torch.equal(odd, dense)


def test_rows_do_not_depend_on_other_sequences():
    """A sequence's rows are the same bits whatever the others hold, and however long they are."""
    import torch
    rows = []
    for other in (5, 900, 2500):
        s = Setup(8, 2, 128, 16, 16, [1500, 2500], [4, 4], seed=8)
        s.fill()
        qt, _ = s.values((s.rows, 8, 128), "bfloat16", 0.5)
        base = _i32([1500, other])
        out = torch.empty_like(qt)
        s.cache.attention(1, qt, s.d_table, s.d_off, base, 2, 4, out)
        rows.append(out[:4].clone())
    assert torch.equal(rows[0], rows[1]) and torch.equal(rows[0], rows[2])


def test_values_of_dead_and_later_slots_do_not_matter():
    """NaN codes behind the sequence's end, in pages it does not own and in unused table slots' pages, change nothing."""
    import torch
    s = Setup(8, 2, 128, 16, 16, [100], [3], seed=3, room=200)
    s.fill()
    qt, _ = s.values((3, 8, 128), "bfloat16", 0.5)
    a, b = torch.empty_like(qt), torch.empty_like(qt)
    s.cache.attention(1, qt, *s.args(), a)
    codes = s.cache.codes[1]
    keep = torch.zeros(codes.shape[0], 16, dtype=torch.bool, device="cuda")
    for p in range(103):
        keep[s.table[0, p // 16], p % 16] = True
    codes.masked_fill_(~keep[:, None, None, :, None], 0x7f)
    table = s.d_table.clone()
    table[0, 7:] = -1
    s.cache.attention(1, qt, table, s.d_off, s.d_base, 1, 3, b)
    assert torch.equal(a, b) and s.cache.get_status() == 0


def test_device_errors_are_caught_and_bounded():
    """Spans past the limits and page ids outside the pool: the status word, NaN or zeros, nothing else touched."""
    import torch
    s = Setup(4, 2, 64, 16, 16, [40, 60], [3, 4], seed=7, room=0)
    s.fill()
    codes, scales = s.cache.codes.clone(), s.cache.scales.clone()
    qt, _ = s.values((s.rows, 4, 64), "bfloat16")
    kt, _ = s.values((s.rows, 2, 64), "bfloat16")
    ok = torch.empty_like(qt)
    s.cache.attention(1, qt, *s.args(), ok)
    assert s.cache.get_status() == 0
    far = _i32([40, 61])                                              # the second passes max_context = 64
    out = torch.zeros_like(qt)
    s.cache.attention(1, qt, s.d_table, s.d_off, far, 2, 4, out)
    assert s.cache.get_status() == -2 and out[3:].isnan().all() and torch.equal(out[:3], ok[:3])
    s.cache.write(1, kt, kt, s.d_table, s.d_off, _i32([-1, 61]), 2, 4)
    assert s.cache.get_status() == -2
    long = _i32([0, 3, 8])                                            # the second span is longer than max_span
    s.cache.write(1, kt, kt, s.d_table, _i32([0, 0, 7]), _i32([40, 20]), 2, 4)
    assert s.cache.get_status() == -1
    s.cache.write(1, kt, kt, s.d_table, long, _i32([0, 0]), 2, 4)     # and outside the call's rows
    assert s.cache.get_status() == -1
    bad = s.d_table.clone()
    bad[1, 1], bad[1, 3] = s.n_pages, -5
    # row tensors that hold fewer rows than the offsets name: the second span is refused, nothing past them is touched
    s.cache.attention(1, qt[:5], s.d_table, s.d_off, s.d_base, 2, 4, out[:5])
    assert s.cache.get_status() == -1
    s.cache.codes.copy_(codes)                                        # what the first of those spans wrote, taken back
    s.cache.scales.copy_(scales)
    s.cache.read(1, bad, s.d_off, s.d_base, 2, 4, kt, kt.clone())
    assert s.cache.get_status() == -2 and (kt[3:] == 0).all() and not (kt[:3] == 0).all()
    s.cache.attention(1, qt, bad, s.d_off, s.d_base, 2, 4, out)
    assert s.cache.get_status() == -2 and torch.equal(out[:3], ok[:3]) and out.isfinite().all()
    s.cache.codes.copy_(codes)
    s.cache.scales.copy_(scales)
    s.cache.write(1, kt, kt, bad, s.d_off, _i32([45, 60]), 2, 4)
    assert s.cache.get_status() == -2
    same = torch.ones(s.n_pages, dtype=torch.bool, device="cuda")
    same[torch.as_tensor(s.table[0, 2:3].copy()).cuda()] = False      # positions 45..47 are in one page
    assert torch.equal(s.cache.codes[1][same], codes[1][same]) and torch.equal(s.cache.codes[0], codes[0])


def test_binding_refusals_on_device():
    import torch
    s = Setup(4, 2, 64, 16, 16, [40], [3])
    k = torch.zeros(3, 2, 64, dtype=torch.bfloat16, device="cuda")
    q = torch.zeros(3, 4, 64, dtype=torch.bfloat16, device="cuda")
    bad = [lambda: s.cache.write(1, k, k.half(), *s.args()), lambda: s.cache.write(1, k, k[:2], *s.args()),
           lambda: s.cache.write(1, k.transpose(1, 2), k, *s.args()), lambda: s.cache.write(1, k[:, :1], k, *s.args()),
           lambda: s.cache.attention(1, q.float(), *s.args(), q.float()), lambda: s.cache.attention(1, q, *s.args(), q.half()),
           lambda: s.cache.attention(1, q, s.d_table.long(), *s.args()[1:], q),
           lambda: s.cache.attention(1, q, s.d_table[:, :1].contiguous(), *s.args()[1:], q)]
    for f in bad:
        with pytest.raises(ValueError):
            f()
    from speculative_decoding_verify_02_gb300 import SdvError
    for f in (lambda: s.cache.write(2, k, k, *s.args()), lambda: s.cache.attention(-1, q, *s.args(), q),
              lambda: s.cache.attention(1, q, *s.args()[:4], 4, q), lambda: s.cache.attention(1, q, *s.args(), q, window=-1)):
        with pytest.raises(SdvError):
            f()
    assert s.cache.get_status() == 0


def test_tensors_on_another_device_are_refused(monkeypatch):
    import torch
    import speculative_decoding_verify_02_gb300 as sdv
    s = Setup(2, 1, 64, 16, 16, [3], [1])
    q = torch.zeros(1, 2, 64, dtype=torch.bfloat16, device="cuda")
    s.cache.attention(1, q, *s.args(), q)
    monkeypatch.setattr(sdv, "_many", True)
    s.cache.attention(1, q, *s.args(), q)                             # all of them where the kernels run
    monkeypatch.setattr(sdv, "_elsewhere", lambda t: t is s.d_base)
    with pytest.raises(ValueError, match="base"):
        s.cache.attention(1, q, *s.args(), q)
    monkeypatch.setattr(sdv, "_elsewhere", lambda t: t is q)
    with pytest.raises(ValueError, match="q: a device tensor"):
        s.cache.attention(1, q, *s.args(), q)
    monkeypatch.undo()
    assert not sdv._elsewhere(q)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    assert sdv._elsewhere(q)


def test_captured_graph_follows_lengths_and_streams():
    """Write and attention captured once and replayed at other lengths give what eager calls give, on another stream
    than the current one, too."""
    import torch
    s = Setup(8, 2, 128, 16, 16, [100, 700], [4, 4], seed=12, room=900)
    s.fill()
    kv, _ = s.values((s.rows, 2, 2, 128), "bfloat16")
    qt, _ = s.values((s.rows, 8, 128), "bfloat16", 0.5)
    out = torch.zeros_like(qt)

    def step(stream=None):
        s.cache.write(1, kv[:, 0], kv[:, 1], *s.args(), stream=stream)
        s.cache.attention(1, qt, *s.args(), out, stream=stream)

    step()                                                            # warm-up outside the capture
    codes, scales = s.cache.codes.clone(), s.cache.scales.clone()
    g = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side), torch.cuda.graph(g, stream=side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    for base in ([100, 700], [1500, 3], [0, 1203]):
        s.d_base.copy_(_i32(base))
        res = []
        for how in ("graph", "eager", "stream"):
            s.cache.codes.copy_(codes)
            s.cache.scales.copy_(scales)
            out.zero_()
            torch.cuda.synchronize()
            if how == "graph":
                g.replay()
            elif how == "eager":
                step()
            else:
                step(side)
            torch.cuda.synchronize()
            res.append((out.clone(), s.cache.codes.clone(), s.cache.scales.clone()))
        for other in res[1:]:
            assert all(torch.equal(x, y) for x, y in zip(res[0], other))
    assert s.cache.get_status() == 0


def test_cache_on_the_verifiers_pages():
    """The run of them together: a Verifier reserves and rewinds pages, and an 8-bit cache of the same page table takes
    the K/V that its forward wrote, answers a verify span's queries, and follows a rewind."""
    import synth
    import torch
    from speculative_decoding_verify_02_gb300 import QuantCache
    from tests.helpers import upload_weights
    from speculative_decoding_verify_02_gb300 import Verifier
    shape = synth.TINY
    _, dev = upload_weights(shape, 1)
    v = Verifier(shape, dev, page_size=16, n_pages=32, max_batch=1, max_rows=128, max_span=128, max_context=256)
    nkv, D, ps = shape.n_kv_heads, shape.head_dim, 16
    cache = QuantCache(shape.n_layers, shape.n_q_heads, nkv, D, page_size=ps, n_pages=32, max_batch=1, max_rows=128,
                       max_span=128, max_context=256)
    pool = oracle.QuantPool(32, nkv, ps, D, 16)
    prompt = synth.tokens(3, "qcache.prompt", 100, shape.vocab)
    table, npg, top = _i32(np.zeros((1, 16))), _i32([0]), _i32([0])
    length, rng = 0, np.random.default_rng(0)
    for n, keep in ((100, 100), (8, 3), (8, 8)):
        toks = prompt[:n]
        v.ensure_capacity(_i32([length + n]), 1)
        v.spec_forward(_i32(toks), _i32([0, n]), 1, 128, 128, _i32(np.zeros(128)))
        v.page_table(table, npg, top)
        pages = table[0].long()
        kv = v.pool.view(torch.bfloat16).view(shape.n_layers, 32, 2, nkv, ps, D)[1]
        pos = torch.arange(length, length + n, device="cuda")
        rows = kv[pages[pos // ps], :, :, pos % ps]                   # [n, 2, nkv, D], as the forward wrote them
        cache.write(1, rows[:, 0], rows[:, 1], table, _i32([0, n]), _i32([length]), 1, 128)
        host = table[0].cpu().numpy()
        r64 = rows.double().cpu().numpy()
        pool.write(host, length, r64[:, 0], r64[:, 1])
        qt = _dev(rng.normal(size=(n, shape.n_q_heads, D)).astype(np.float32)).bfloat16()
        out, exact16 = torch.empty_like(qt), torch.empty(n, shape.n_q_heads * D, dtype=torch.bfloat16, device="cuda")
        cache.attention(1, qt, table, _i32([0, n]), _i32([length]), 1, 128, out)
        ref, mag, topq = pool.attention(host, length, qt.double().cpu().numpy())
        assert (np.abs(out.double().cpu().numpy() - ref) <= _tolerance(ref, mag, topq, D, "bfloat16")).all()
        # and next to the 16-bit cache's own answer: codes are within 2^-4 of each key and value
        v.op_attention(1, qt, _i32([0, n]), _i32([length]), 1, 128, exact16)
        rel = (out.reshape(n, -1).float() - exact16.float()).norm() / exact16.float().norm()
        assert float(rel) < 2.0 ** -4
        length += keep
        v.rewind_cache(_i32([length]), 1)
    assert v.get_status() == 0 and cache.get_status() == 0
    v.close()
