"""Forked sequences on the GPU: the page bookkeeping against oracle.SharedPool, the copied rows bit by bit, and whole runs of
continuations against sequences that were prefilled one by one."""
import numpy as np
import pytest

import oracle
import synth
from tests.helpers import page_tables, upload_weights

pytestmark = pytest.mark.gpu


def _i32(a):
    import torch
    return torch.as_tensor(np.asarray(a, dtype=np.int32)).cuda()


def _f32(a):
    import torch
    return torch.as_tensor(np.asarray(a, dtype=np.float32)).cuda()


class Pair:
    """A context over zero weights and the oracle's pool, kept alike."""

    def __init__(self, n_pages=24, ps=16, B=6, context=128, layers=3, nkv=2, D=64, ngram=0):
        import torch
        from speculative_decoding_verify_02_gb300 import Verifier
        shape = synth.Shape("fork", layers, 128, nkv, nkv, D, 128, 256)
        w = {n: torch.zeros(d, dtype=torch.bfloat16, device="cuda") for n, d in shape.tensor_shapes().items()}
        self.v = Verifier(shape, w, page_size=ps, n_pages=n_pages, max_batch=B, max_rows=128, max_span=128, max_context=context,
                          ngram_capacity=ngram)
        self.o = oracle.SharedPool(n_pages, ps, B, -(-context // ps))
        self.B, self.ps = B, ps
        self.pool = self.v.pool.view(torch.bfloat16).view(layers, n_pages, 2, nkv, ps, D)

    def grow(self, lengths):
        """Reserve and write up to these lengths (-1: leave alone)."""
        import torch
        self.v.ensure_capacity(_i32(lengths), self.B)
        self.o.ensure_capacity(lengths)
        for b, n in enumerate(lengths):
            while n > self.o.length[b]:
                rows = min(128, n - self.o.length[b])
                off = np.zeros(self.B + 1, dtype=np.int32)
                off[b + 1:] = rows
                self.v.spec_forward(torch.zeros(128, dtype=torch.int32, device="cuda"), _i32(off), self.B, rows, rows, _i32([0] * 128))
                self.o.set_length(b, self.o.length[b] + rows)

    def same(self, status=0):
        import torch
        table, held, top = page_tables(self.v)
        lens = torch.zeros(self.B, dtype=torch.int32, device="cuda")
        self.v.cache_seq_len(lens)
        assert lens.tolist() == self.o.length and top == len(self.o.free)
        for b in range(self.B):
            assert held[b] == len(self.o.table[b]) and table[b, :held[b]].tolist() == self.o.table[b], b
            assert (table[b, held[b]:] == -1).all()
        assert self.v.get_status() == status

    def fork(self, src, dst):
        self.v.fork_seq(_i32(src), _i32(dst), len(src))
        return self.o.fork(src, dst)

    def rewind(self, lengths):
        self.v.rewind_cache(_i32(lengths), len(lengths))
        self.o.rewind(lengths)


@pytest.mark.parametrize("ps", [1, 7, 16, 32])
@pytest.mark.parametrize("L", [0, 1, 16, 31, 33, 64])
def test_tables_and_copied_rows(L, ps):
    import torch
    t = Pair(n_pages=100, ps=ps, B=5)
    t.grow([L, 20, -1, -1, -1])
    t.same()
    t.pool.copy_(torch.randn(t.pool.shape, device="cuda"))
    before = t.pool.clone()
    for s, d, fill in (c for c in t.fork([0, 0, 1], [3, 2, 4]) if c):
        before[:, d, :, :, :fill] = before[:, s, :, :, :fill]
    t.same()
    assert torch.equal(t.pool, before)       # filled slots copied, nothing else touched
    t.rewind([-1, -1, 0, 0, 0])
    t.same()


@pytest.mark.parametrize("seed", range(6))
def test_random_runs(seed):
    """Reservations, forks, rewinds and resets in any order: tables, free stack and lengths as the oracle's, refusals too."""
    from speculative_decoding_verify_02_gb300 import SDV_ERR_ARG, SDV_ERR_CAPACITY
    rng = np.random.default_rng(seed)
    t = Pair(n_pages=int(rng.integers(8, 30)), ps=int(rng.choice([4, 16])), B=6, context=96, layers=1)
    done = set()
    for _ in range(60):
        kind = rng.choice(["grow", "fork", "rewind", "reset"])
        code = 0
        try:
            if kind == "grow":
                b = int(rng.integers(t.B))
                want = [-1] * t.B
                want[b] = min(96, t.o.length[b] + int(rng.integers(1, 40)))
                t.grow(want)
            elif kind == "fork":
                n = int(rng.integers(1, 4))
                t.fork(rng.integers(0, t.B, n).tolist(), rng.integers(0, t.B, n).tolist())
            elif kind == "rewind":
                t.rewind([int(rng.integers(-1, t.o.length[b] + 2)) if rng.random() < 0.4 else -1 for b in range(t.B)])
            else:
                b = int(rng.integers(t.B))
                t.v.reset_seq(b)
                t.o.reset(b)
        except oracle.CapacityError:
            code = SDV_ERR_CAPACITY
        except ValueError:
            code = SDV_ERR_ARG
        done.add((kind, code))
        t.same(code)
    assert len(done) > 4


@pytest.mark.parametrize("seed", range(4))
def test_random_runs_of_forks(seed):
    """Forks of random sequences into empty ones, rewinds to page borders and resets."""
    rng = np.random.default_rng(100 + seed)
    t = Pair(n_pages=60, ps=int(rng.choice([4, 16])), B=12, context=96, layers=1)
    t.grow([int(rng.integers(1, 70)), int(rng.integers(1, 70))] + [-1] * 10)
    shared = 0
    for _ in range(40):
        empty = [b for b in range(t.B) if not t.o.table[b]]
        full = [b for b in range(t.B) if t.o.length[b] > 0]
        kind = rng.choice(["fork", "grow", "rewind", "reset"], p=[0.5, 0.2, 0.2, 0.1])
        try:
            if kind == "fork" and empty and full:
                n = int(rng.integers(1, len(empty) + 1))
                t.fork(rng.choice(full, n).tolist(), rng.permutation(empty)[:n].tolist())
            elif kind == "grow" and full:
                want = [-1] * t.B
                b = int(rng.choice(full))
                want[b] = min(96, t.o.length[b] + int(rng.integers(1, 9)))
                t.grow(want)
            elif kind == "rewind":
                t.rewind([int(rng.integers(0, t.o.length[b] // t.ps + 1)) * t.ps if t.o.length[b] and rng.random() < 0.4 else -1 for b in range(t.B)])
            elif kind == "reset" and full:
                b = int(rng.choice(full))
                t.v.reset_seq(b)
                t.o.reset(b)
        except oracle.CapacityError:
            t.v.get_status()
        pages = [x for table in t.o.table for x in table]
        shared += len(pages) - len(set(pages))
        t.same()
    assert shared > 20


def test_refusals_change_nothing():
    from speculative_decoding_verify_02_gb300 import SDV_ERR_ARG, SDV_ERR_CAPACITY, SdvError
    t = Pair(n_pages=4, B=4)
    t.grow([20, 0, -1, -1])
    for src, dst in (([0], [0]), ([0, 0], [1, 1]), ([0], [4]), ([0], [-1]), ([9], [1]), ([-1], [1]), ([1], [0]), ([2, 0], [3, 2])):
        t.v.fork_seq(_i32(src), _i32(dst), len(src))
        t.same(SDV_ERR_ARG)
    t.v.fork_seq(_i32([0, 0, 0]), _i32([1, 2, 3]), 3)      # three partial pages, two left
    t.same(SDV_ERR_CAPACITY)
    t.fork([0, 0], [1, 2])
    t.same()
    t.v.rewind_cache(_i32([-1, 5]), 2)                     # into the shared first page
    t.same(SDV_ERR_ARG)
    t.rewind([-1, 18, 17])                                 # inside of their own
    t.same()
    t.rewind([-1, 16])
    t.same()
    for n in (0, 5):
        with pytest.raises(SdvError):
            t.v.fork_seq(_i32([0] * 5), _i32([1] * 5), n)
    with pytest.raises(ValueError):
        t.v.fork_seq(_i32([0]), _i32([3]), 2)


def test_sliding_window_models_are_refused():
    import torch
    from dataclasses import replace
    from speculative_decoding_verify_02_gb300 import SDV_ERR_UNSUPPORTED, SdvError, Verifier
    shape = synth.Shape("fork", 2, 128, 2, 2, 64, 128, 256)
    w = {n: torch.zeros(d, dtype=torch.bfloat16, device="cuda") for n, d in shape.tensor_shapes().items()}
    try:
        shape = replace(shape, swa_window=32)
    except TypeError:
        object.__setattr__(shape, "swa_window", 32)
    v = Verifier(shape, w, page_size=16, n_pages=8, max_batch=2, max_rows=16, max_span=16, max_context=64)
    with pytest.raises(SdvError) as e:
        v.fork_seq(_i32([0]), _i32([1]), 1)
    assert e.value.code == SDV_ERR_UNSUPPORTED


def test_a_rewind_captured_before_the_first_fork():
    """A graph's rewind, made while nothing was shared, releases shared pages and refuses lengths inside of them all the same."""
    import torch
    from speculative_decoding_verify_02_gb300 import SDV_ERR_ARG
    t = Pair(n_pages=60, B=9)
    t.grow([70, 33] + [-1] * 7)
    lengths = _i32([-1] * 9)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        t.v.rewind_cache(lengths, 9)
    t.fork([0, 0, 1, 0, 1, 0, 0], [2, 3, 4, 5, 6, 7, 8])
    for n, ok in (([-1, -1, 0, 64, 32, -1, 0, 70, 16], True), ([20] + [-1] * 8, False), ([0, 0] + [-1] * 7, True), ([-1] * 9, True),
                  ([0] * 9, True)):
        lengths.copy_(_i32(n))
        g.replay()
        if ok:
            t.o.rewind(n)
        t.same(0 if ok else SDV_ERR_ARG)
    assert len(t.o.free) == 60


def test_a_page_goes_back_with_its_last_holder():
    t = Pair(n_pages=40, B=6)
    t.grow([70, -1, -1, -1, -1, -1])
    t.fork([0] * 5, [1, 2, 3, 4, 5])
    for b in (0, 3):
        t.v.reset_seq(b)
        t.o.reset(b)
        t.same()
    t.rewind([-1, 64, 70, -1, 32, 48])                     # part by part
    t.same()
    t.fork([1], [0])                                       # a fork of a fork
    t.same()
    t.rewind([0] * 6)
    t.same()
    assert t.o.table == [[]] * 6 and len(t.o.free) == 40


def _tiny(B, spans=8, ngram=0, n_pages=64):
    from speculative_decoding_verify_02_gb300 import Verifier
    shape = synth.TINY
    host, dev = upload_weights(shape, 1)
    return Verifier(shape, dev, page_size=16, n_pages=n_pages, max_batch=B, max_rows=128, max_span=128, max_context=256,
                    ngram_capacity=ngram), shape


def test_continuations_equal_prompts_of_their_own():
    """Spans after a fork give the same logits, bit by bit, as after a prefill of each sequence, and the pages of the prompt are
    held once."""
    import torch
    B = 4
    prompt = synth.tokens(3, "fork.prompt", 77, synth.TINY.vocab)
    spans = [synth.tokens(4 + b, "fork.span", 3 + b, synth.TINY.vocab) for b in range(B)]
    got = []
    for shared in (False, True):
        v, shape = _tiny(B)
        toks = _i32(prompt)
        for b in range(1 if shared else B):
            off = np.zeros(B + 1)
            off[b + 1:] = 77
            need = np.full(B, -1)
            need[b] = 77
            v.ensure_capacity(_i32(need), B)
            v.spec_forward(toks, _i32(off), B, 77, 77, _i32([0] * 77))
        if shared:
            v.fork_seq(_i32([0] * (B - 1)), _i32(range(1, B)), B - 1)
            assert page_tables(v)[2] == 64 - 5 - (B - 1)
        off = np.concatenate([[0], np.cumsum([len(s) for s in spans])])
        v.ensure_capacity(_i32([77 + len(s) for s in spans]), B)
        lg = torch.zeros(int(off[-1]), shape.vocab, device="cuda")
        v.spec_forward(_i32(np.concatenate(spans)), _i32(off), B, int(off[-1]), 8, _i32([0] * int(off[-1])), lg)
        torch.cuda.synchronize()
        assert v.get_status() == 0
        got.append(lg.clone())
    assert torch.equal(got[0], got[1])


@pytest.mark.parametrize("graph", [False, True])
def test_loops_equal_prompts_of_their_own(graph):
    """prefill_shared and greedy n-gram steps: the committed tokens are those of a batch of equal prompts, the n-gram index and
    the loop state having gone along."""
    import torch
    from speculative_decoding_verify_02_gb300.runner import SpecLoop
    from synth import workloads
    prompt = workloads.motif_prompt(1)
    B, runs = 3, []
    for shared in (False, True):
        v, _ = _tiny(B, ngram=256)
        loop = SpecLoop(v, B, 5)
        first = loop.prefill_shared(prompt, ngram=True) if shared else loop.prefill([prompt] * B, ngram=True)
        loop.start([20] * B, 2, adaptive=True, k_max=4)
        if graph:
            loop.step()
            loop.capture()
        text = [[int(f)] for f in first]

        def take():
            com, n = loop.committed.view(B, 5).cpu().numpy(), loop.n_commit.cpu().numpy()
            for b in range(B):
                text[b] += com[b, :n[b]].tolist()

        if graph:
            take()
        for _ in range(9):
            loop.replay() if graph else loop.step()
            torch.cuda.synchronize()
            take()
        assert v.get_status() == 0
        runs.append(text)
        v.close()
    assert runs[0] == runs[1]


def test_sampled_continuations_with_cuts_follow_the_oracle():
    """The run as it is used: one prompt, continuations whose first tokens are drawn from it, then steps of drafts verified
    against the cut distribution. Each decision is the oracle's for the logits that the forward gave."""
    import torch
    from speculative_decoding_verify_02_gb300 import SDV_DRAFT_NGRAM
    from speculative_decoding_verify_02_gb300.runner import SpecLoop
    from synth import workloads
    B, S = 4, 5
    prompt = workloads.motif_prompt(1)
    v, shape = _tiny(B, ngram=256)
    V = shape.vocab
    rng = np.random.default_rng(11)
    T, k, p, m = np.float32([0.7, 1.0, 1.3, 0.0]), [20, 0, 7, 3], np.float32([0.9, 0.8, 1.0, 0.5]), np.float32([0.0, 0.02, 0.05, 0.0])
    noise = rng.exponential(size=(B, V)).astype(np.float32)
    loop = SpecLoop(v, B, S)
    cuts = dict(top_k=_i32(k), top_p=_f32(p), min_p=_f32(m))
    first = loop.prefill_shared(prompt, ngram=True, temperature=_f32(T), noise=_f32(noise), **cuts)
    # the prompt's last row again, from a context of its own
    w, _ = _tiny(1)
    w.ensure_capacity(_i32([len(prompt)]), 1)
    lg = torch.zeros(len(prompt), V, device="cuda")
    w.spec_forward(_i32(prompt), _i32([0, len(prompt)]), 1, len(prompt), len(prompt), _i32([0] * len(prompt)), lg)
    last = lg[-1].cpu().numpy()
    for b in range(B):
        assert first[b] == oracle.draw_kept(*oracle.kept_tokens(last, T[b], k[b], p[b], m[b]), noise[b])
    loop.start([40] * B, 3)
    raw = torch.zeros(B * S, V, device="cuda")
    real = v.filter_logits

    def spy(logits, *a, **kw):
        raw.copy_(logits)
        real(logits, *a, **kw)

    v.filter_logits = spy
    for _ in range(6):
        u, e = rng.random(B * S).astype(np.float32), rng.exponential(size=(B, V)).astype(np.float32)
        loop.step(drafter=SDV_DRAFT_NGRAM, temperature=_f32(T), uniforms=_f32(u), noise=_f32(e), **cuts)
        torch.cuda.synchronize()
        off, toks = loop.row_off.cpu().numpy(), loop.tokens.cpu().numpy()
        com, n = loop.committed.view(B, S).cpu().numpy(), loop.n_commit.cpu().numpy()
        x = raw.cpu().numpy()
        for b in range(B):
            rows = slice(off[b], off[b + 1])
            cut = np.full((off[b + 1] - off[b], V), -np.inf, dtype=np.float32)
            for i, row in enumerate(x[rows]):
                keep = oracle.kept_tokens(row, T[b], k[b], p[b], m[b])[0]
                cut[i, keep] = row[keep]
            j, want = oracle.accept_sampled(toks[rows].tolist(), cut, T[b], u[rows], e[b])
            assert n[b] == j + 1 and com[b, :n[b]].tolist() == want
        assert v.get_status() == 0


def test_shared_attention_over_a_verifiers_pages():
    """The pool and the tables of forked sequences, read by the attention for a group: as the context's own attention, whose
    rows are those of a batch without groups."""
    import torch
    from speculative_decoding_verify_02_gb300 import SharedAttention
    B, S, L = 5, 4, 100
    t = Pair(n_pages=64, B=B, context=256, layers=2, nkv=2, D=64)
    t.grow([L] + [-1] * (B - 1))
    t.fork([0] * (B - 1), list(range(1, B)))
    t.v.ensure_capacity(_i32([L + S + b for b in range(B)]), B)
    t.o.ensure_capacity([L + S + b for b in range(B)])
    live = torch.randn(t.pool.shape, device="cuda").to(torch.bfloat16)
    for s_, d_ in ((t.o.table[0][6], t.o.table[b][6]) for b in range(1, B)):
        live[:, d_, :, :, :L % 16] = live[:, s_, :, :, :L % 16]
    t.pool.copy_(live)
    table = torch.zeros(B, t.v.pages_per_seq, dtype=torch.int32, device="cuda")
    t.v.page_table(table, None, None)
    q = torch.randn(B * S, 2, 64, device="cuda").to(torch.bfloat16)
    off, base = _i32(np.arange(B + 1) * S), _i32([L + b for b in range(B)])
    plan = SharedAttention(2, 2, 2, 64, n_pages=64, max_batch=B, max_rows=B * S, max_span=S, max_context=256, pool=t.v.pool)
    out, ref = torch.zeros_like(q), torch.zeros(B * S, 128, dtype=torch.bfloat16, device="cuda")
    plan.attention(1, q, table, off, base, B, S, out, group_off=_i32([0, B]), prefix_len=_i32([L]), G=1)
    t.v.op_attention(1, q, off, base, B, S, ref)
    torch.cuda.synchronize()
    assert plan.get_status() == 0 and t.v.get_status() == 0
    # both round a result of magnitude up to max |v| < 8 once: a step of bf16 apart at most, and each is near the exact one
    d = (out.view(B * S, 128).double() - ref.double()).abs()
    assert (d <= 2.0 ** -7 * ref.double().abs() + 2.0 ** -9).all()
