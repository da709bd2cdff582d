"""Sampled acceptance on the GPU against the float64 oracle (oracle.accept_sampled): every output equal.

Decisions are compared exactly: a draft's test u q(d) < p(d) and the race argmax w / e come out alike unless the two sides
are within rounding of each other (about 2^-20 relative), which a few hundred seeded decisions are not."""
import numpy as np
import pytest

import oracle
import synth
from tests.helpers import upload_weights

pytestmark = pytest.mark.gpu


def _i32(a):
    import torch
    return torch.as_tensor(np.asarray(a, dtype=np.int32)).cuda()


def _f32(a):
    import torch
    return torch.as_tensor(np.asarray(a, dtype=np.float32)).cuda()


def _verifier(vocab, max_batch, max_span, max_rows=128):
    """A context of any vocabulary: zero weights, one layer of the smallest shape."""
    import torch
    from speculative_decoding_verify_02_gb300 import Verifier
    shape = synth.Shape("accept", 1, 128, 2, 2, 64, 128, vocab)
    w = {n: torch.zeros(d, dtype=torch.bfloat16, device="cuda") for n, d in shape.tensor_shapes().items()}
    return Verifier(shape, w, page_size=16, n_pages=max_batch * 16, max_batch=max_batch, max_rows=max_rows,
                    max_span=max_span, max_context=256)


def _inputs(rng, spans, V, probs, temps, peak=8.0):
    R = int(sum(spans))
    logits = (2 * rng.normal(size=(R, V))).astype(np.float32)
    logits[np.arange(R), rng.integers(0, V, R)] += peak
    q = np.exp(logits.astype(np.float64) + 0.7 * rng.normal(size=(R, V)))
    q = (q / q.sum(-1, keepdims=True)).astype(np.float32)
    tokens = np.zeros(R, dtype=np.int64)
    for r in range(1, R):
        tokens[r] = rng.choice(V, p=q[r - 1].astype(np.float64) / q[r - 1].astype(np.float64).sum())
    return dict(spans=spans, V=V, logits=logits, probs=q if probs else None, tokens=tokens, u=rng.random(R).astype(np.float32),
                noise=rng.exponential(size=(len(spans), V)).astype(np.float32), temps=np.asarray(temps, dtype=np.float32))


def _run(v, x, max_commit=None, logits=None, probs=None, noise=None):
    import torch
    B, off = len(x["spans"]), np.concatenate([[0], np.cumsum(x["spans"])])
    mc = max_commit or max(x["spans"])
    n_acc, n_com, new = _i32(np.full(B, -7)), _i32(np.full(B, -7)), _i32(np.full(B, -7))
    com = _i32(np.full((B, mc), -9))
    if logits is None:
        logits = _f32(x["logits"])
    if probs is None and x["probs"] is not None:
        probs = _f32(x["probs"])
    v.accept_sampled(_i32(x["tokens"]), _i32(off), logits, _f32(x["temps"]), _f32(x["u"]),
                     _f32(x["noise"]) if noise is None else noise, B, mc, n_acc, com, n_com, new, draft_probs=probs)
    torch.cuda.synchronize()
    return [t.cpu().numpy() for t in (n_acc, com, n_com, new)]


def _ref(x, lengths, max_commit=None):
    B, off = len(x["spans"]), np.concatenate([[0], np.cumsum(x["spans"])])
    mc = max_commit or max(x["spans"])
    n_acc, n_com, new = np.full(B, -1), np.zeros(B, dtype=int), np.full(B, -1)
    com = np.full((B, mc), -9)
    for b, S in enumerate(x["spans"]):
        if S:
            r = slice(off[b], off[b + 1])
            m, toks = oracle.accept_sampled(x["tokens"][r], x["logits"][r], x["temps"][b], x["u"][r], x["noise"][b],
                                            None if x["probs"] is None else x["probs"][r])
            n_acc[b], n_com[b], new[b] = m, m + 1, lengths[b] - S + m + 1
            com[b, :m + 1] = toks
    return [n_acc, com, n_com, new]


def _lengths(v, B):
    import torch
    t = _i32(np.zeros(v.ccfg.max_batch))
    v.cache_seq_len(t)
    torch.cuda.synchronize()
    return t.cpu().numpy()[:B]


def _forward(v, spans):
    """Run the spans through the forward so that the lengths are those after a verify."""
    off = np.concatenate([[0], np.cumsum(spans)])
    v.ensure_capacity(_i32(spans), len(spans))
    v.spec_forward(_i32(np.zeros(off[-1])), _i32(off), len(spans), v.ccfg.max_rows, v.ccfg.max_span,
                   _i32(np.zeros(off[-1])))


CASES = [
    # spans, vocab, probs
    ([1], 5, False), ([2], 1, True), ([8], 4096, True), ([8], 4097, False), ([17, 1, 0, 5], 2048, True),
    ([3, 3, 0, 9], 4095, False), ([8] * 16, 10007, True), ([1] * 32, 3001, False), ([128], 257, True), ([8], 151936, True),
]


@pytest.mark.parametrize("spans, V, probs", CASES)
def test_accept_sampled_matches_oracle(spans, V, probs):
    rng = np.random.default_rng(V + len(spans))
    v = _verifier(V, len(spans), max(spans))
    _forward(v, spans)
    lengths = _lengths(v, len(spans))
    np.testing.assert_array_equal(lengths, spans)
    total = 0
    for seed in range(3):
        temps = rng.choice([0.0, 0.3, 0.8, 1.0, 2.0], len(spans))
        x = _inputs(rng, spans, V, probs, temps)
        for got, ref in zip(_run(v, x), _ref(x, lengths)):
            np.testing.assert_array_equal(got, ref)
            total += 1
    assert v.get_status() == 0
    v.close()


def test_strides_and_alignment():
    """Rows inside wider matrices and off a 16-byte boundary give the same answers."""
    import torch
    rng = np.random.default_rng(5)
    V, spans = 5000, [6, 4]
    v = _verifier(V, 2, 6)
    _forward(v, spans)
    x = _inputs(rng, spans, V, True, [0.9, 1.3])
    ref = _ref(x, _lengths(v, 2))

    def wide(a, extra, off):
        t = torch.full((a.shape[0], V + extra), float("nan"), device="cuda")
        t[:, off:off + V] = _f32(a)
        return t[:, off:off + V]

    for extra, off in ((8, 4), (7, 3)):
        got = _run(v, x, logits=wide(x["logits"], extra, off), probs=wide(x["probs"], extra, off),
                   noise=wide(x["noise"], extra, off))
        for a, b in zip(got, ref):
            np.testing.assert_array_equal(a, b)
    v.close()


def test_masked_and_extreme_logits():
    """-inf masks tokens, +inf shares the row, NaN is passed over, huge and tiny temperatures stay finite."""
    rng = np.random.default_rng(6)
    V, spans = 1500, [4, 4, 4, 4, 4]
    v = _verifier(V, 5, 4)
    _forward(v, spans)
    x = _inputs(rng, spans, V, True, [1.0, 1.0, 1e-30, 1e30, 0.0])
    x["logits"][:, ::3] = -np.inf
    x["logits"][5, 7] = np.inf
    x["logits"][9:11, 4] = np.nan
    x["logits"][16:, 11] = x["logits"][16:, 100] = 90.0               # greedy ties: the lowest index
    for got, ref in zip(_run(v, x), _ref(x, _lengths(v, 5))):
        np.testing.assert_array_equal(got, ref)
    assert v.get_status() == 0
    x["logits"][0] = -np.inf                                          # nothing to draw in the first row
    x["tokens"][5] = V                                                # and a draft outside the vocabulary
    for got, ref in zip(_run(v, x), _ref(x, _lengths(v, 5))):
        np.testing.assert_array_equal(got, ref)
    assert v.get_status() == -4
    v.close()


def test_identical_distributions_accept_everything():
    """q = p up to rounding: with u < 1 - 2^-10 every draft is accepted."""
    import torch
    rng = np.random.default_rng(7)
    V, spans = 3000, [16]
    v = _verifier(V, 1, 16)
    _forward(v, spans)
    x = _inputs(rng, spans, V, True, [0.7])
    x["probs"] = torch.softmax(_f32(x["logits"]).double() / float(x["temps"][0]), -1).float().cpu().numpy()
    x["tokens"][1:] = [rng.choice(V, p=q.astype(np.float64) / q.sum(dtype=np.float64)) for q in x["probs"][:-1]]
    x["u"] *= 1 - 2.0 ** -10
    n_acc, com, _, _ = _run(v, x)
    assert n_acc[0] == 15
    np.testing.assert_array_equal(com[0, :15], x["tokens"][1:])
    v.close()


def test_refused_spans():
    import torch
    rng = np.random.default_rng(8)
    v = _verifier(700, 3, 6)
    x = _inputs(rng, [3, 6, 2], 700, False, [1.0, 1.0, 1.0])
    _forward(v, [3, 6, 2])
    lengths = _lengths(v, 3)
    got, ref = _run(v, x, max_commit=4), None
    assert v.get_status() == -1 and got[0][1] == -1 and got[2][1] == 0 and got[3][1] == -1 and (got[1][1] == -9).all()
    y = dict(x, spans=[3, 0, 2])
    keep = np.r_[0:3, 9:11]
    y.update(logits=x["logits"][keep], tokens=x["tokens"][keep], u=x["u"][keep])
    ref = _ref(y, lengths, max_commit=4)
    for b in (0, 2):
        for a, r in zip(got, ref):
            np.testing.assert_array_equal(a[b], r[b])
    short = dict(x, logits=x["logits"][:10])                          # fewer rows than the offsets name: the last span
    got = _run(v, short)                                              # is refused
    assert v.get_status() == -1 and got[0].tolist()[2] == -1
    for a, r in zip(got, _ref(x, lengths)):
        np.testing.assert_array_equal(a[:2], r[:2])
    z = torch.zeros
    f, i = dict(device="cuda"), dict(device="cuda", dtype=torch.int32)
    good = dict(tokens=z(11, **i), row_off=z(4, **i), logits=z(11, 700, **f), temperature=z(3, **f), uniforms=z(11, **f),
                noise=z(3, 700, **f), B=3, max_commit=6, n_accept=z(3, **i), committed=z(3, 6, **i), n_commit=z(3, **i),
                new_len=z(3, **i))
    for bad in (dict(logits=z(11, 699, **f)), dict(logits=z(11, 700, **f).half()), dict(noise=z(2, 700, **f)),
                dict(uniforms=z(10, **f)), dict(temperature=z(3)), dict(committed=z(3, 5, **i)),
                dict(row_off=z(4, device="cuda", dtype=torch.int64)), dict(draft_probs=z(4, 700, **f)),
                dict(logits=z(700, 11, **f).T)):
        with pytest.raises(ValueError):
            v.accept_sampled(**{**good, **bad})
    from speculative_decoding_verify_02_gb300 import SdvError
    with pytest.raises(SdvError):
        v.accept_sampled(**{**good, "B": 4, "row_off": z(5, **i), "temperature": z(4, **f), "noise": z(4, 700, **f),
                            "n_accept": z(4, **i), "committed": z(4, 6, **i), "n_commit": z(4, **i), "new_len": z(4, **i)})
    v.close()


def test_offsets_at_the_ends_of_32_bits():
    rng = np.random.default_rng(12)
    v = _verifier(700, 1, 6)
    x = _inputs(rng, [2], 700, False, [1.0])
    _forward(v, [2])
    import torch
    n_acc, com, n_com, new = (torch.full((k,), -9, dtype=torch.int32, device="cuda") for k in (1, 6, 1, 1))
    for off in ([2**31 - 1, -2**31], [-2**31, 2**31 - 1], [2**31 - 2, 2**31 - 1], [-1, 1], [0, 2**31 - 1]):
        v.accept_sampled(_i32(x["tokens"]), _i32(off), _f32(x["logits"]), _f32(x["temps"]), _f32(x["u"]),
                         _f32(x["noise"]), 1, 6, n_acc, com, n_com, new)
        assert v.get_status() == -1 and n_acc.item() == -1 and n_com.item() == 0 and (com == -9).all()
    v.close()


def test_certain_drafts_at_temperature_zero_are_greedy_acceptance():
    """Temperature 0 and certain drafts: the same outputs and loop state as accept_greedy on the argmax."""
    rng = np.random.default_rng(9)
    V, spans = 600, [5, 7, 1]
    a, b = _verifier(V, 3, 7), _verifier(V, 3, 7)
    x = _inputs(rng, spans, V, False, [0.0, -1.0, 0.0])
    am = x["logits"].argmax(-1)
    x["tokens"][1:4] = am[:3]                                         # some accepted drafts
    x["tokens"][6:12] = am[5:11]
    outs = []
    for v in (a, b):
        _forward(v, spans)
        v.gen_init(_i32([1, 2, 3]), _i32([50, 50, 50]), 3, 2, True, 7)
    got = _run(a, x)
    off = _i32(np.concatenate([[0], np.cumsum(spans)]))
    n_acc, n_com, new, com = _i32([0] * 3), _i32([0] * 3), _i32([0] * 3), _i32(np.full((3, 7), -9))
    b.accept_greedy(_i32(x["tokens"]), off, _i32(am), 3, 7, n_acc, com, n_com, new)
    for g, r in zip(got, (n_acc, com, n_com, new)):
        np.testing.assert_array_equal(g, r.cpu().numpy())
    table = _i32(np.arange(3 * 60).reshape(3, 60) % V)
    for v in (a, b):                                                  # the next span: current token, count and K
        tok, ro, req = _i32(np.zeros(21)), _i32(np.zeros(4)), _i32(np.zeros(3))
        v.propose(2, table, 60, 3, 7, tok, ro, req)
        outs.append((tok.cpu().numpy(), ro.cpu().numpy(), req.cpu().numpy()))
        v.close()
    for p, q in zip(*outs):
        np.testing.assert_array_equal(p, q)


def test_loop_accepts_against_probabilities():
    """SpecLoop.step with uniforms and noise, eager and as a replayed graph: each step's committed tokens are the
    oracle's on the logits that the step's forward left, and the cache follows the accepted lengths."""
    import torch
    from synth import workloads
    from speculative_decoding_verify_02_gb300 import SDV_DRAFT_TABLE, Verifier
    from speculative_decoding_verify_02_gb300.runner import SpecLoop
    shape = synth.TINY
    _, dev = upload_weights(shape, 1)
    B, S, V = 2, 6, shape.vocab
    prompts = [workloads.motif_prompt(1), workloads.uniform_context(2, 40, V)]
    streams = []
    for graph in (False, True):
        v = Verifier(shape, dev, page_size=16, n_pages=64, max_batch=B, max_rows=128, max_span=128, max_context=512)
        loop = SpecLoop(v, B, S)
        first = loop.prefill(prompts)
        loop.start([40, 40], k_init=S - 1)
        rng = np.random.default_rng(13)
        table = _i32(rng.integers(0, 40, (B, 64)))
        temp, u, noise = _f32([0.05, 0.0]), _f32(np.zeros(B * S)), _f32(np.ones((B, V)))
        probs = torch.full((B * S, V), 1.0 / 40, device="cuda")       # the drafter: uniform over the first 40 tokens
        probs[:, 40:] = 0
        kw = dict(drafter=SDV_DRAFT_TABLE, table=table, table_stride=64, ngram=False, temperature=temp, uniforms=u,
                  noise=noise, draft_probs=probs)
        if graph:
            state = v.workspace.clone()
            loop.step(**kw)                                           # warm-up, taken back
            torch.cuda.synchronize()
            v.workspace.copy_(state)
            loop.capture(**kw)
        out = [[int(t)] for t in first]
        for _ in range(12):
            u.copy_(_f32(rng.random(B * S)))
            noise.copy_(_f32(rng.exponential(size=(B, V))))
            before = _lengths(v, B)
            loop.replay() if graph else loop.step(**kw)
            torch.cuda.synchronize()
            off = loop.row_off.cpu().numpy()
            lg, toks = loop.logits.cpu().numpy(), loop.tokens.cpu().numpy()
            for b in range(B):
                r = slice(off[b], off[b + 1])
                if r.start == r.stop:
                    continue
                m, com = oracle.accept_sampled(toks[r], lg[r], float(temp[b]), u.cpu().numpy()[r], noise[b].cpu().numpy(),
                                               probs[r.start:r.stop].cpu().numpy())
                assert int(loop.n_accept[b]) == m and loop.committed.view(B, S)[b, :m + 1].tolist() == com
                assert _lengths(v, B)[b] == before[b] + m + 1
                out[b] += com
        assert v.get_status() == 0
        streams.append(out)
        v.close()
    assert streams[0] == streams[1]
