"""Cases, plain forms and 64-bit forms of the operators for many continuations of one prompt.

Four operators, selected by a case's "op":
  attention  paged attention for groups of sequences that share a prefix, with a window, a tanh cap or a distance bias
  fork       sequences that take over a prompt's pages, and their release
  filter     logits outside a row's top-k, top-p and min-p set masked
  sample     a token drawn from that set with given random numbers

With `own` false, run() computes a pass in elementary torch operations; with `own` true it makes the package's calls.
"""
import math
import types

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ---------------------------------------------------------------- cases

def _attention(name, batch, groups, prefix, own_lo, own_hi, span, **kw):
    c = dict(name=name, op="attention", batch=batch, groups=groups, prefix=prefix, own_lo=own_lo, own_hi=own_hi, span=span,
             ragged=False, nq=32, nkv=8, dim=128, page=16, window=0, cap=0.0, slopes=False, dtype="bf16")
    c.update(kw)
    return c


def _fork(name, sources, copies, lo, hi, **kw):
    c = dict(name=name, op="fork", sources=sources, copies=copies, lo=lo, hi=hi, layers=36, nkv=8, dim=128, page=16)
    c.update(kw)
    return c


def _draw_case(name, op, batch, span, vocab, **kw):
    c = dict(name=name, op=op, batch=batch, span=span, ragged=False, vocab=vocab, top_k=True, top_p=True, min_p=True,
             ties=False)
    c.update(kw)
    return c


def listed():
    return [
        # eight continuations of a prompt at the headline context, each verifying seven drafts
        _attention("verify 8 of 848", 8, 1, 848, 0, 64, 8),
        # many samples of one long document, decoding a token each
        _attention("decode 64 of 32k", 64, 1, 32768, 1, 512, 1),
        # sixteen continuations of the long context with spans of eight rows: tensor cores count
        _attention("verify 16 of 32k", 16, 1, 32768, 0, 256, 8),
        # several prompts of different lengths, small heads in fp16 behind a sliding window, pages of an odd size
        _attention("three prompts window fp16", 21, 3, 2900, 0, 300, 5, ragged=True, nq=12, nkv=2, dim=64, page=24,
                   window=1024, dtype="fp16"),
        # the batch workload of unrelated sequences, for a model that caps its scores
        _attention("b16 ragged cap", 16, 0, 0, 512, 4096, 8, ragged=True, cap=50.0),
        # two prompts for a model with a distance bias
        _attention("two prompts bias", 12, 2, 4000, 0, 800, 3, ragged=True, slopes=True),
        # best of eight after a verify step at the headline context: tails copied, pages shared, and given back
        _fork("fork 1 to 8", 1, 7, 855, 855),
        # a batch of prompts, each continued sixteen times
        _fork("fork 4 to 64", 4, 15, 512, 4096),
        # the headline verify step's rows, filtered before acceptance
        _draw_case("filter 8 rows", "filter", 1, 8, 151936),
        # the batch verify step
        _draw_case("filter 128 rows", "filter", 16, 8, 151936, min_p=False),
        # one token of one sequence
        _draw_case("sample 1 row", "sample", 1, 1, 151936),
        # a decoding batch, logits rounded to bf16 by the head
        _draw_case("sample 64 rows", "sample", 64, 1, 151936, ties=True, min_p=False),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attention", "attention", "attention", "fork", "filter", "sample"])
    if op in ("filter", "sample"):
        batch = _log_int(rng, 1, 64)
        span = rng.randint(1, max(1, min(17, 128 // batch)))
        return dict(op=op, batch=batch, span=span, ragged=rng.random() < 0.5, vocab=_log_int(rng, 1000, 151936),
                    top_k=rng.random() < 0.6, top_p=rng.random() < 0.7, min_p=rng.random() < 0.4, ties=rng.random() < 0.4)
    if op == "fork":
        sources = rng.randint(1, 4)
        hi = _log_int(rng, 16, 4096)
        return dict(op=op, sources=sources, copies=rng.randint(1, 60 // sources), lo=rng.choice([hi, hi // 2, 1]), hi=hi,
                    layers=rng.randint(1, 36), nkv=rng.choice([1, 2, 8]), dim=rng.choice([64, 128, 128]),
                    page=rng.choice([8, 16, 16, 24, 32, 64]))
    nq, nkv, dim = rng.choice([(32, 8, 128), (32, 8, 128), (4, 2, 64), (8, 1, 128), (6, 6, 64), (20, 4, 128), (12, 2, 64)])
    span = rng.choice([1, 1, rng.randint(2, 17), rng.randint(2, 17), rng.randint(18, 64)])
    batch = _log_int(rng, 1, min(128, max(1, 512 // span)))
    groups = rng.choice([0, 1, 1, rng.randint(1, max(1, min(4, batch)))])
    # never more than the largest listed case
    most = 128 * 33024 * 32 // (batch * span * nq)
    own_hi = _log_int(rng, 1, max(1, min(4096, most // 2, 16 * 4096 * 8 * 128 // (batch * nkv * dim))))
    prefix = _log_int(rng, 16, max(16, min(32768, most // 2))) if groups else 0
    return dict(op="attention", batch=batch, groups=groups, prefix=prefix, own_lo=rng.choice([own_hi, own_hi // 2, 0]),
                own_hi=own_hi, span=span, ragged=rng.random() < 0.5, nq=nq, nkv=nkv, dim=dim,
                page=rng.choice([8, 16, 16, 24, 32, 64, 128, 10]), window=rng.choice([0, 0, rng.randint(1, prefix + own_hi + 1)]),
                cap=rng.choice([0.0, 0.0, 30.0, 50.0]), slopes=rng.random() < 0.25, dtype=rng.choice(["bf16", "bf16", "fp16"]))


# ---------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 29)


def _spans(case, g):
    """Span lengths and their offsets: all of the full length, or from that down to half of it in any order."""
    n = torch.full((case["batch"],), case["span"], device="cuda", dtype=torch.int32)
    if case["ragged"]:
        cut = torch.arange(case["batch"], device="cuda") * (case["span"] // 2) // max(1, case["batch"] - 1)
        n -= cut[torch.randperm(case["batch"], device="cuda", generator=g)].to(torch.int32)
    off = torch.zeros(case["batch"] + 1, device="cuda", dtype=torch.int32)
    off[1:] = n.cumsum(0)
    return n, off


def _group_bounds(case):
    """Sequence bounds of the groups: later groups are larger."""
    G, B = case["groups"], case["batch"]
    return [max(i, B * i * (i + 1) // (G * (G + 1))) for i in range(G)] + [B] if G else []


def _attention_inputs(case, seed):
    """Spans, lengths, page tables whose groups share their prefix's whole pages, the pool and the queries."""
    g = _gen(seed)
    B, G, ps, nkv, D, P = case["batch"], case["groups"], case["page"], case["nkv"], case["dim"], case["prefix"]
    dt = DTYPES[case["dtype"]]
    n, off = _spans(case, g)
    bounds = _group_bounds(case)
    i32 = dict(device="cuda", dtype=torch.int32)
    prefix = torch.zeros(max(G, 1), **i32)
    group_of = torch.zeros(B, device="cuda", dtype=torch.long)
    if G:
        # a group's prompt has the full length or down to half of it
        prefix[:] = torch.tensor([P - (P // 2) * i // G for i in range(G)], **i32)
        group_of = torch.repeat_interleave(torch.arange(G, device="cuda"), torch.diff(torch.tensor(bounds, device="cuda")))
    base = prefix[group_of] + torch.randint(case["own_lo"], case["own_hi"] + 1, (B,), device="cuda", generator=g,
                                            dtype=torch.int32)
    context = P + case["own_hi"] + case["span"]
    per_seq = -(-context // ps)
    own_pages = -(-(case["own_hi"] + case["span"]) // ps) + 1
    shared_pages = P // ps
    n_pages = max(1, G * shared_pages + B * own_pages)
    perm = torch.randperm(n_pages, device="cuda", generator=g).to(torch.int32)
    mine = perm[G * shared_pages:].view(B, own_pages)
    full = (prefix[group_of] // ps).long()[:, None]            # whole pages of the prefix
    j = torch.arange(per_seq, device="cuda")[None]
    table = mine.gather(1, (j - full).clamp(0, own_pages - 1))
    if G and shared_pages:
        shared = perm[:G * shared_pages].view(G, shared_pages)
        table = torch.where(j < full, shared[group_of][:, j[0].clamp_max(shared_pages - 1)], table)
    table = table.contiguous()
    pool = torch.empty(n_pages, 2, nkv, ps, D, device="cuda", dtype=dt)
    step = max(1, (1 << 26) // (2 * nkv * ps * D))
    for p in range(0, n_pages, step):
        m = min(step, n_pages - p)
        x = torch.randn(m, 2, nkv, ps, D, device="cuda", generator=g)
        # a few channels of every key are several times larger than the rest
        x[:, 0] *= 1 + 3 * (torch.arange(D, device="cuda") % 37 == 5)
        pool[p:p + m] = x
    if G:
        # the page that a prefix ends in: every sequence has a copy of its filled slots
        first = torch.tensor(bounds[:-1], device="cuda")[group_of]
        tail = table.gather(1, full.clamp_max(per_seq - 1))[:, 0].long()
        source = pool[tail[first]]
        filled = torch.arange(ps, device="cuda") < (prefix[group_of] % ps)[:, None]
        pool[tail] = torch.where(filled[:, None, None, :, None], source, pool[tail])
    rows = int(off[-1])
    q = (1.5 * torch.randn(rows, case["nq"], D, device="cuda", generator=g)).to(dt)
    slopes = None
    if case["slopes"]:  # a geometric series over the heads
        slopes = torch.exp2(-8.0 * torch.arange(1, case["nq"] + 1, device="cuda") / case["nq"]).float()
    return types.SimpleNamespace(n=n, off=off, base=base, table=table, pool=pool, q=q, rows=rows, context=context,
                                 n_pages=n_pages, prefix=prefix, bounds=bounds, group_of=group_of, slopes=slopes,
                                 group_off=torch.tensor(bounds, **i32) if G else None)


def _fork_inputs(case, seed):
    """Lengths of the prompts, and the pool as their prefill leaves it (page 0 up, prompt by prompt)."""
    g = _gen(seed)
    A, ps = case["sources"], case["page"]
    length = torch.randint(case["lo"], case["hi"] + 1, (A,), device="cuda", generator=g, dtype=torch.int32)
    held = [-(-x // ps) for x in length.tolist()]
    per_seq = -(-case["hi"] // ps) + 1
    batch = A * (1 + case["copies"])
    # rounded up so that seeds share a size; one free page for each continuation
    n_pages = A * per_seq + batch
    pool = torch.empty(case["layers"], n_pages, 2, case["nkv"], ps, case["dim"], device="cuda", dtype=torch.bfloat16)
    for layer in range(case["layers"]):
        pool[layer] = torch.randn(pool.shape[1:], device="cuda", generator=g)
    i32 = dict(device="cuda", dtype=torch.int32)
    src = torch.arange(A, **i32).repeat_interleave(case["copies"])
    dst = torch.arange(A, batch, **i32)
    return types.SimpleNamespace(length=length, held=held, per_seq=per_seq, batch=batch, n_pages=n_pages, pool=pool, src=src,
                                 dst=dst)


def _draw_inputs(case, seed):
    """Logits with a few likely tokens, each sequence's settings, and the random numbers."""
    g = _gen(seed)
    B, V = case["batch"], case["vocab"]
    n, off = _spans(case, g)
    rows = int(off[-1])
    logits = 2.0 * torch.randn(rows, V, device="cuda", generator=g)
    top = torch.randint(0, V, (rows, 40), device="cuda", generator=g)
    logits.scatter_add_(1, top, 4 + 12 * torch.rand(rows, 40, device="cuda", generator=g))
    if case["ties"]:
        logits = logits.to(torch.bfloat16).float()
    u = torch.rand(B, 4, device="cuda", generator=g)
    temperature = 0.5 + u[:, 0]
    temperature[torch.rand(B, device="cuda", generator=g) < 0.1] = 0.0
    top_k = torch.exp(u[:, 1] * math.log(min(V, 1000))).to(torch.int32)
    top_p = (0.7 + 0.3 * u[:, 2]).contiguous()
    min_p = (0.1 * u[:, 3]).contiguous()
    s = types.SimpleNamespace(n=n, off=off, rows=rows, logits=logits, temperature=temperature.contiguous(),
                              top_k=top_k if case["top_k"] else None, top_p=top_p if case["top_p"] else None,
                              min_p=min_p if case["min_p"] else None, noise=None)
    if case["op"] == "sample":
        s.noise = torch.empty(rows, V, device="cuda").exponential_(generator=g)
    return s


def _verifier(vocab, layers, nkv, dim, **limits):
    """A context of a small decoder with the case's cache or vocabulary."""
    from speculative_decoding_verify_02_gb300 import Verifier
    nkv = max(nkv, 128 // dim)
    wide = nkv * dim
    shape = types.SimpleNamespace(n_layers=layers, hidden=128, n_q_heads=nkv, n_kv_heads=nkv, head_dim=dim, ffn=128,
                                  vocab=vocab, rms_eps=1e-6, rope_theta=1e6, qk_norm=True)
    z = lambda *d: torch.zeros(*d, device="cuda", dtype=torch.bfloat16)  # noqa: E731
    w = {"embed": z(vocab, 128), "lm_head": z(vocab, 128), "final_norm": z(128)}
    for layer in range(layers):
        for name, dims in dict(attn_norm=(128,), wq=(wide, 128), wk=(wide, 128), wv=(wide, 128), q_norm=(dim,), k_norm=(dim,),
                               wo=(128, wide), ffn_norm=(128,), w_gate=(128, 128), w_up=(128, 128),
                               w_down=(128, 128)).items():
            w[f"layers.{layer}.{name}"] = z(*dims)
    return Verifier(shape, w, **limits)


def prepare(case, seed):
    if case["op"] == "attention":
        s = _attention_inputs(case, seed)
        s.out = torch.empty_like(s.q)
        if own:
            from speculative_decoding_verify_02_gb300 import SharedAttention
            s.plan = SharedAttention(1, case["nq"], case["nkv"], case["dim"], page_size=case["page"], n_pages=s.n_pages,
                                     max_batch=case["batch"], max_rows=s.rows, max_span=case["span"], max_context=s.context,
                                     dtype=s.q.dtype, pool=s.pool)
    elif case["op"] == "fork":
        case = dict(case, nkv=max(case["nkv"], 128 // case["dim"]))
        s = _fork_inputs(case, seed)
        i32 = dict(device="cuda", dtype=torch.int32)
        s.out_table = torch.zeros(s.batch, s.per_seq, **i32)
        s.out_held, s.out_len, s.out_free = torch.zeros(s.batch, **i32), torch.zeros(s.batch, **i32), torch.zeros(1, **i32)
        s.release = torch.full((s.batch,), -1, **i32)
        s.release[case["sources"]:] = 0
        if own:
            s.verifier = _prefilled(case, s)
    else:
        s = _draw_inputs(case, seed)
        s.tokens = torch.zeros(s.rows, device="cuda", dtype=torch.int32)
        s.kept = torch.zeros(s.rows, device="cuda", dtype=torch.int32)
        s.out = torch.empty_like(s.logits) if case["op"] == "filter" else None
        if own:
            s.verifier = _verifier(case["vocab"], 1, 2, 64, page_size=16, n_pages=1, max_batch=case["batch"],
                                   max_rows=s.rows, max_span=case["span"], max_context=case["span"])
    s.case = dict(case)
    return s


def _prefilled(case, s):
    """A context that holds the prompts, and the pool's values in place of what its zero weights wrote."""
    A = case["sources"]
    v = _verifier(1024, case["layers"], case["nkv"], case["dim"], page_size=case["page"], n_pages=s.n_pages,
                  max_batch=s.batch, max_rows=128, max_span=128, max_context=s.per_seq * case["page"])
    tokens = torch.zeros(128, device="cuda", dtype=torch.int32)
    argmax = torch.zeros_like(tokens)
    v.ensure_capacity(s.length, A)
    for a, n in enumerate(s.length.tolist()):
        for at in range(0, n, 128):
            rows = min(128, n - at)
            off = torch.zeros(A + 1, device="cuda", dtype=torch.int32)
            off[a + 1:] = rows
            v.spec_forward(tokens, off, A, rows, rows, argmax)
    pool = v.pool.view(torch.bfloat16).view_as(s.pool)
    pool.copy_(s.pool)
    s.pool = pool
    return v


# ---------------------------------------------------------------- a pass

def run(state):
    return {"attention": _run_attention, "fork": _run_fork, "filter": _run_filter, "sample": _run_sample}[state.case["op"]](state)


def _pages(pool, ids):
    """K and V [2, n, nkv, tokens, D] in 32 bits of the pages ids [n, pages]."""
    kv = pool[ids.long()].float()
    return kv.permute(2, 0, 3, 1, 4, 5).flatten(3, 4)


def _run_attention(s):
    c = s.case
    B, G, S, D, nq, nkv, W = c["batch"], c["groups"], c["span"], c["dim"], c["nq"], c["nkv"], c["window"]
    if own:
        s.plan.attention(0, s.q, s.table, s.off, s.base, B, S, s.out, group_off=s.group_off,
                         prefix_len=s.prefix if G else None, G=G, window=W, softcap=c["cap"], slopes=s.slopes)
        return s.out
    grp, ps = nq // nkv, c["page"]
    out = torch.empty_like(s.q)
    bounds = s.bounds if G else list(range(0, B, 16)) + [B]
    for g, (b0, b1) in enumerate(zip(bounds[:-1], bounds[1:])):
        n = b1 - b0
        if n == 0:
            continue
        i = torch.arange(S, device="cuda")
        rows = (s.off[b0:b1, None] + i).clamp_max(s.rows - 1).long()                  # [n, S], padded
        pos = s.base[b0:b1, None] + i                                                 # [n, S]
        q = s.q[rows].float().view(n, S, nkv, grp, D).permute(2, 0, 3, 1, 4)          # [nkv, n, grp, S, D]
        pre = s.prefix[g].long() if G else torch.zeros((), device="cuda", dtype=torch.long)
        scores, keys = [], []
        if G:
            kp, vp = _pages(s.pool, s.table[b0:b0 + 1, :-(-c["prefix"] // ps)])       # [1, nkv, tokens, D]
            t = torch.arange(kp.shape[2], device="cuda")
            scores.append((q.reshape(nkv, -1, D) @ kp[0].transpose(-1, -2)).view(nkv, n, grp, S, -1))
            keys.append(torch.where(t < pre, t, 1 << 30).expand(n, -1))               # position of each key; beyond all: hidden
        slots = -(-(c["own_hi"] + S) // ps) + 1
        at = (pre // ps + torch.arange(slots, device="cuda")).clamp_max(s.table.shape[1] - 1)
        ko, vo = _pages(s.pool, s.table[b0:b1, at])                                   # [n, nkv, tokens, D]
        t = pre // ps * ps + torch.arange(slots * ps, device="cuda")
        scores.append((q.transpose(0, 1).reshape(n, nkv, grp * S, D) @ ko.transpose(-1, -2)).view(n, nkv, grp, S, -1).transpose(0, 1))
        keys.append(torch.where(t >= pre, t, 1 << 30).expand(n, -1))
        z = torch.cat(scores, -1) / math.sqrt(D)
        del scores
        if c["cap"] > 0:
            z = c["cap"] * torch.tanh(z / c["cap"])
        t = torch.cat(keys, -1)[:, None, :]                                           # [n, 1, keys]
        if s.slopes is not None:
            z += s.slopes.view(nkv, 1, grp, 1, 1) * (t - pos[..., None])[None, :, None].float()
        seen = t <= pos[..., None]
        if W:
            seen &= t > pos[..., None] - W
        z.masked_fill_(~seen[None, :, None], -math.inf)
        z -= z.amax(-1, keepdim=True)
        z = torch.exp_(z)
        z /= z.sum(-1, keepdim=True)
        o = torch.zeros(nkv, n, grp, S, D, device="cuda")
        if G:
            o += (z[..., :vp.shape[2]].reshape(nkv, n * grp * S, -1) @ vp[0]).view_as(o)
            z = z[..., vp.shape[2]:]
        o += (z.transpose(0, 1).reshape(n, nkv, grp * S, -1) @ vo).view(n, nkv, grp, S, D).transpose(0, 1)
        live = i < s.n[b0:b1, None]
        o = o.permute(1, 3, 0, 2, 4).reshape(n * S, nq, D).to(out.dtype)
        # padded rows go where a row of the call lies anyway: keep the live ones
        out[rows.view(-1)[live.view(-1)]] = o[live.view(-1)]
    return out


def _run_fork(s):
    c = s.case
    A, n, ps = c["sources"], s.batch - c["sources"], c["page"]
    if own:
        v = s.verifier
        v.fork_seq(s.src, s.dst, n)
        v.page_table(s.out_table, s.out_held, s.out_free)
        v.cache_seq_len(s.out_len)
        v.rewind_cache(s.release, s.batch)
        return {"pool": s.pool, "table": s.out_table, "held": s.out_held, "free": s.out_free, "length": s.out_len}
    L = s.length.long()
    held = -(-L // ps)
    first = held.cumsum(0) - held
    j = torch.arange(s.per_seq, device="cuda")
    table = torch.where(j < held[:, None], first[:, None] + j, -1)                    # the prompts' pages
    src = s.src.long()
    fill = L % ps
    part = fill[src] > 0
    fresh = held.sum() + part.long().cumsum(0) - 1                                    # pages taken from the stack in order
    child = torch.where(j < (L // ps)[src][:, None], table[src], -1)
    child = torch.where((j == (L // ps)[src][:, None]) & part[:, None], fresh[:, None], child)
    tail = table[src].gather(1, (L // ps)[src][:, None].clamp_max(s.per_seq - 1))[:, 0].clamp_min(0)
    to = torch.where(part, fresh, tail)                                               # nothing to copy: onto itself
    filled = torch.arange(ps, device="cuda") < fill[src][:, None]
    pool = s.pool
    pool[:, to] = torch.where(filled[None, :, None, None, :, None], pool[:, tail], pool[:, to])
    s.out_table.copy_(torch.cat([table, child]))
    s.out_held.copy_(torch.cat([held, held[src]]))
    s.out_free.copy_(s.n_pages - held.sum() - part.sum())
    s.out_len.copy_(torch.cat([L, L[src]]))
    return {"pool": pool, "table": s.out_table, "held": s.out_held, "free": s.out_free, "length": s.out_len}


def _kept_set(s):
    """Weights of the logits over the largest and which of them are kept, in 64 bits: decisions lie next to borders."""
    V = s.logits.shape[1]
    r = torch.arange(s.rows, device="cuda")
    seq = torch.searchsorted(s.off, r.to(torch.int32), right=True) - 1
    x, order = torch.sort(s.logits, dim=-1, descending=True, stable=True)                 # equal logits by ascending index
    x = x.double()
    t = s.temperature[seq].double()[:, None]
    rank = torch.arange(V, device="cuda")
    w = torch.exp((x - x[:, :1]) / torch.where(t > 0, t, 1.0))
    keep = torch.ones_like(w, dtype=torch.bool)
    if s.top_k is not None:
        k = s.top_k[seq].long()[:, None]
        keep &= (rank < k) | (k <= 0)
    if s.top_p is not None:
        mass = (w * keep).cumsum(-1)
        before = torch.cat([torch.zeros_like(mass[:, :1]), mass[:, :-1]], -1)
        keep &= before < s.top_p[seq].double()[:, None] * mass[:, -1:]
    if s.min_p is not None:
        keep &= w >= s.min_p[seq].double()[:, None]
    keep &= (t > 0) | (rank == 0)
    keep[:, 0] = True
    return torch.zeros_like(w).scatter_(1, order, w), torch.zeros_like(keep).scatter_(1, order, keep)


def _run_filter(s):
    if own:
        s.verifier.filter_logits(s.logits, s.off, s.case["batch"], s.out, s.kept, s.temperature, top_k=s.top_k, top_p=s.top_p,
                                 min_p=s.min_p)
        return {"logits": s.out, "kept": s.kept}
    _, keep = _kept_set(s)
    return {"logits": torch.where(keep, s.logits, -math.inf), "kept": keep.sum(-1).to(torch.int32)}


def _run_sample(s):
    if own:
        s.verifier.sample(s.logits, s.off, s.noise, s.case["batch"], s.tokens, s.temperature, top_k=s.top_k, top_p=s.top_p,
                          min_p=s.min_p, n_kept=s.kept)
        return {"token": s.tokens, "kept": s.kept}
    V = s.logits.shape[1]
    w, keep = _kept_set(s)
    race = torch.where(keep, w / s.noise.double(), -1.0)  # the largest is a draw in proportion to the weights
    won = race == race.amax(-1, keepdim=True)
    token = torch.where(won, torch.arange(V, device="cuda"), V).amin(-1)
    return {"token": token.to(torch.int32), "kept": keep.sum(-1).to(torch.int32)}


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    if case["op"] == "fork":
        nkv = max(case["nkv"], 128 // case["dim"])
        token = case["layers"] * 2 * nkv * case["dim"] * 2.0
        fill = (case["lo"] % case["page"]) if case["lo"] == case["hi"] else case["page"] / 2
        return {"bytes": case["sources"] * (1 + case["copies"]) * fill * token + 64.0, "flops": 0.0}
    rows = case["batch"] * case["span"] * (0.75 if case["ragged"] and case["batch"] > 1 else 1.0)
    if case["op"] in ("filter", "sample"):
        return {"bytes": 4.0 * case["vocab"] * rows * (2 if case["op"] == "filter" else 1), "flops": 6.0 * case["vocab"] * rows}
    mid = (case["own_lo"] + case["own_hi"]) / 2
    G = case["groups"]
    prefix = case["prefix"] * (1 - (G - 1) / (4 * G)) if G else 0.0
    tokens, keys = G * prefix + case["batch"] * (mid + case["span"]), prefix + mid + case["span"] / 2
    if case["window"]:
        seen = min(keys, case["window"])
        tokens, keys = tokens * min(1.0, (seen + case["span"]) / (keys + case["span"])), seen
    size = DTYPES[case["dtype"]].itemsize
    return {"bytes": (tokens * 2 * case["nkv"] + 2 * rows * case["nq"]) * case["dim"] * size,
            "flops": 4.0 * rows * case["nq"] * case["dim"] * keys}


# ---------------------------------------------------------------- 64 bits

def exact(case, seed):
    if case["op"] == "attention":
        return _exact_attention(case, seed)
    if case["op"] == "fork":
        return _exact_fork(dict(case, nkv=max(case["nkv"], 128 // case["dim"])), seed)
    return _exact_draw(case, seed)


def _exact_attention(case, seed):
    s = _attention_inputs(case, seed)
    D, ps, grp = case["dim"], case["page"], case["nq"] // case["nkv"]
    off, base = s.off.tolist(), s.base.tolist()
    out = torch.empty(s.q.shape, device="cuda", dtype=torch.float64)
    for b in range(case["batch"]):
        S = off[b + 1] - off[b]
        if S == 0:
            continue
        end = base[b] + S
        kv = s.pool[s.table[b, :-(-end // ps)].long()]                                # [pages, 2, nkv, ps, D]
        pos = base[b] + torch.arange(S, device="cuda")[:, None]
        key = torch.arange(end, device="cuda")[None]
        hidden = key > pos
        if case["window"]:
            hidden |= pos - key >= case["window"]
        for h in range(case["nkv"]):
            k = kv[:, 0, h].reshape(-1, D)[:end].double()
            v = kv[:, 1, h].reshape(-1, D)[:end].double()
            for e in range(h * grp, (h + 1) * grp):
                z = s.q[off[b]:off[b + 1], e].double() @ k.T * D ** -0.5
                if case["cap"]:
                    z = torch.tanh(z / case["cap"]) * case["cap"]
                if s.slopes is not None:
                    z = z - s.slopes[e].double() * (pos - key)
                out[off[b]:off[b + 1], e] = torch.softmax(z.masked_fill(hidden, -math.inf), -1) @ v
    return out


def _exact_fork(case, seed):
    s = _fork_inputs(case, seed)
    A, ps = case["sources"], case["page"]
    lengths = s.length.tolist()
    free = list(range(s.n_pages - 1, -1, -1))
    tables = [[free.pop() for _ in range(-(-n // ps))] for n in lengths]
    pool = s.pool.double()
    for a in s.src.tolist():
        n = lengths[a]
        pages = tables[a][:n // ps]
        if n % ps:
            page = free.pop()
            pool[:, page, :, :, :n % ps] = pool[:, tables[a][n // ps], :, :, :n % ps]
            pages = pages + [page]
        tables.append(pages)
        lengths.append(n)
    table = torch.full((s.batch, s.per_seq), -1, dtype=torch.int32)
    for b, pages in enumerate(tables):
        table[b, :len(pages)] = torch.tensor(pages, dtype=torch.int32)
    i32 = dict(dtype=torch.int32)
    return {"pool": pool, "table": table, "held": torch.tensor([len(p) for p in tables], **i32),
            "free": torch.tensor([len(free)], **i32), "length": torch.tensor(lengths, **i32)}


def _exact_draw(case, seed):
    s = _draw_inputs(case, seed)
    off, V = s.off.tolist(), case["vocab"]
    kept = torch.zeros(s.rows, dtype=torch.int32)
    token = torch.zeros(s.rows, dtype=torch.int32)
    logits = torch.full((s.rows, V), -math.inf, dtype=torch.float64)
    for b in range(case["batch"]):
        T = float(s.temperature[b].double())
        k = int(s.top_k[b]) if s.top_k is not None else V
        p = float(s.top_p[b].double()) if s.top_p is not None else 2.0
        m = float(s.min_p[b].double()) if s.min_p is not None else 0.0
        for r in range(off[b], off[b + 1]):
            x = s.logits[r].double().cpu()
            order = torch.argsort(-x, stable=True)
            best = float(x[order[0]])
            if T <= 0:
                live = order[:1]
                w = torch.ones(1, dtype=torch.float64)
            else:
                live = order[:min(V, k)]
                w = torch.exp((x[live] - best) / T)
                total = float(w.sum())
                before = w.cumsum(0) - w
                ok = (before < p * total) & (w >= m)
                ok[0] = True
                live, w = live[ok], w[ok]
            kept[r] = len(live)
            logits[r, live] = x[live]
            if s.noise is not None:
                score = torch.log(w) - torch.log(s.noise[r].double().cpu()[live])
                token[r] = int(live[score == score.max()].min())
    if case["op"] == "filter":
        return {"logits": logits, "kept": kept}
    return {"token": token, "kept": kept}
