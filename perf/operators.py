"""Cases, plain forms and 64-bit forms of the 8-bit cache operators and the sampled acceptance.

Four operators, selected by a case's "op":
  attention  paged attention over a cache held in e4m3 with a power-of-two scale for each block of tokens and head
  write      quantising K/V rows into that cache as they are written
  read       reading rows of the cache back
  accept     verification of drafted tokens against the target's probabilities from given random numbers

With `own` false, run() computes a pass in elementary torch operations; with `own` true it makes the package's calls.
"""
import math
import types

import torch

own = False

E4M3 = torch.float8_e4m3fn
E4M3_MAX = 448.0
MIN_EXP = -126  # the smallest scale is 2^-126
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ---------------------------------------------------------------- cases

def _attention(name, batch, lo, hi, span, **kw):
    c = dict(name=name, op="attention", batch=batch, lo=lo, hi=hi, span=span, ragged=False, nq=32, nkv=8, dim=128,
             page=16, block=16, window=0, dtype="bf16")
    c.update(kw)
    return c


def _cache(name, op, batch, lo, hi, span, **kw):
    c = dict(name=name, op=op, batch=batch, lo=lo, hi=hi, span=span, ragged=False, nkv=8, dim=128, page=16, block=16,
             dtype="bf16")
    c.update(kw)
    return c


def _accept(name, batch, span, vocab, probs, **kw):
    c = dict(name=name, op="accept", batch=batch, span=span, ragged=False, vocab=vocab, probs=probs)
    c.update(kw)
    return c


def listed():
    return [
        # plain decoding of one sequence at the headline context: one row a head, latency counts
        _attention("decode 848", 1, 848, 848, 1),
        # the headline verify step: 7 drafts and the current token
        _attention("verify 848 x8", 1, 848, 848, 8),
        # the batch workload: ragged contexts and spans, one scale a token
        _attention("verify b16 ragged", 16, 512, 4096, 8, ragged=True, block=1),
        # the long-context workload
        _attention("verify 32k x8", 1, 32768, 32768, 8),
        # a prefill chunk deep in a long prompt
        _attention("prefill 128 at 32k", 1, 32640, 32640, 128, page=64, block=64),
        # small heads in fp16 behind a sliding window, pages of an odd size
        _attention("window fp16 d64", 7, 900, 5000, 5, ragged=True, nq=12, nkv=2, dim=64, page=24, block=8, window=1024,
                   dtype="fp16"),
        # one layer's K/V of a batch verify step, most spans starting inside a block
        _cache("write b16 x8", "write", 16, 512, 4096, 8, ragged=True),
        # prompts quantised in one go when a sequence moves into the 8-bit cache
        _cache("write prompts", "write", 16, 0, 0, 4096, ragged=True),
        # a whole batch's rows read back, as for moving sequences out of the cache
        _cache("read prompts", "read", 16, 0, 0, 4096, ragged=True, page=32, block=8),
        # one sequence's recent rows
        _cache("read 509", "read", 1, 339, 339, 509, dtype="fp32"),
        # the headline verify step with prompt-lookup drafts (each draft certain)
        _accept("accept x8", 1, 8, 151936, False),
        # the batch verify step with a drafter that gives its distribution
        _accept("accept b16 x8 probs", 16, 8, 151936, True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attention", "attention", "write", "read", "accept"])
    if op == "accept":
        batch = _log_int(rng, 1, 16)
        return dict(op=op, batch=batch, span=rng.randint(1, max(1, min(17, 128 // batch))), ragged=rng.random() < 0.5,
                    vocab=_log_int(rng, 1000, 151936), probs=rng.random() < 0.6)
    page = rng.choice([8, 16, 16, 24, 32, 64, 128])
    block = rng.choice([b for b in (1, 4, 8, 16, 32, page) if page % b == 0])
    batch = _log_int(rng, 1, 32)
    if op == "attention":
        nq, nkv, dim = rng.choice([(32, 8, 128), (32, 8, 128), (4, 2, 64), (8, 1, 128), (6, 6, 64), (20, 4, 128)])
        span = rng.choice([1, rng.randint(2, 17), rng.randint(2, 17), rng.randint(18, 128)])
        hi = _log_int(rng, 16, max(32, min(32768, 16 * 4096 * 8 * 128 // (batch * nkv * dim),
                                           128 * 32768 * 32 // (batch * span * nq))))
        lo = rng.choice([hi, hi // 2, 0])
        window = rng.choice([0, 0, rng.randint(1, 2 * hi)])
        return dict(op=op, batch=batch, lo=lo, hi=hi, span=span, ragged=rng.random() < 0.5, nq=nq, nkv=nkv, dim=dim,
                    page=page, block=block, window=window, dtype=rng.choice(["bf16", "bf16", "fp16"]))
    nkv, dim = rng.choice([(8, 128), (2, 64), (1, 128), (5, 64)])
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    span = _log_int(rng, 1, 12 * 4096 // batch // (2 if dtype == "fp32" else 1))
    hi = rng.randint(0, 4096)
    return dict(op=op, batch=batch, lo=hi // 2, hi=hi, span=span, ragged=rng.random() < 0.5, nkv=nkv, dim=dim, page=page,
                block=block, dtype=dtype)


# ---------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 17)


def _spans(case, g):
    """Span lengths and their offsets: all of the full length, or from that down to half of it in any order."""
    n = torch.full((case["batch"],), case["span"], device="cuda", dtype=torch.int32)
    if case["ragged"]:
        cut = torch.arange(case["batch"], device="cuda") * (case["span"] // 2) // max(1, case["batch"] - 1)
        n -= cut[torch.randperm(case["batch"], device="cuda", generator=g)].to(torch.int32)
    off = torch.zeros(case["batch"] + 1, device="cuda", dtype=torch.int32)
    off[1:] = n.cumsum(0)
    return n, off


def _cache_inputs(case, seed):
    """Spans, lengths, page tables in a random page order and a filled pool."""
    g = _gen(seed)
    B, ps, sb, nkv, D = case["batch"], case["page"], case["block"], case["nkv"], case["dim"]
    n, off = _spans(case, g)
    base = torch.randint(case["lo"], case["hi"] + 1, (B,), device="cuda", generator=g, dtype=torch.int32)
    context = case["hi"] + case["span"]
    per_seq = -(-context // ps)
    n_pages = B * per_seq
    table = torch.randperm(n_pages, device="cuda", generator=g).to(torch.int32).view(B, per_seq).contiguous()
    codes = torch.empty(n_pages, 2, nkv, ps, D, device="cuda", dtype=torch.uint8)
    scales = torch.empty(n_pages, 2, nkv, ps // sb, device="cuda", dtype=torch.float32)
    step = max(1, (1 << 26) // (2 * nkv * ps * D))
    for p in range(0, n_pages, step):
        m = min(step, n_pages - p)
        x = torch.randn(m, 2, nkv, ps // sb, sb, D, device="cuda", generator=g)
        # a few channels of every head are several times larger than the rest, as keys are
        x *= 1 + 6 * (torch.arange(D, device="cuda") % 37 == 5)
        s = torch.exp2((x.abs().amax((-1, -2)) / E4M3_MAX).log2().ceil())
        codes[p:p + m] = (x / s[..., None, None]).to(E4M3).view(torch.uint8).view(m, 2, nkv, ps, D)
        scales[p:p + m] = s
    rows = int(off[-1])
    return types.SimpleNamespace(g=g, n=n, off=off, base=base, table=table, codes=codes, scales=scales, rows=rows,
                                 context=context, n_pages=n_pages)


def _accept_inputs(case, seed):
    """Logits with a few likely tokens, drafts drawn from the drafter's distribution, and the random numbers."""
    g = _gen(seed)
    B, S, V = case["batch"], case["span"], case["vocab"]
    n, off = _spans(case, g)
    rows = int(off[-1])
    logits = 2.0 * torch.randn(rows, V, device="cuda", generator=g)
    top = torch.randint(0, V, (rows, 8), device="cuda", generator=g)
    logits.scatter_add_(1, top, 9 + 3 * torch.rand(rows, 8, device="cuda", generator=g))
    temperature = 0.5 + torch.rand(B, device="cuda", generator=g)
    temperature[torch.rand(B, device="cuda", generator=g) < 0.15] = 0.0
    seq = torch.repeat_interleave(torch.arange(B, device="cuda"), n.long(), output_size=rows)
    t = temperature[seq].clamp_min(0.3)[:, None]
    probs = torch.softmax(logits / t + 0.7 * torch.randn(rows, V, device="cuda", generator=g), -1)
    drafts = torch.multinomial(probs, 1, generator=g)[:, 0].to(torch.int32)
    tokens = torch.zeros(rows, device="cuda", dtype=torch.int32)
    tokens[1:] = drafts[:-1]  # the token of a row was drawn from the row before it
    uniforms = torch.rand(rows, device="cuda", generator=g)
    noise = torch.empty(B, V, device="cuda").exponential_(generator=g)
    return types.SimpleNamespace(n=n, off=off, rows=rows, logits=logits, temperature=temperature, tokens=tokens,
                                 probs=probs if case["probs"] else None, uniforms=uniforms, noise=noise)


def _rows_of(case, s):
    """The K/V or query rows of a cache case."""
    dt = DTYPES[case["dtype"]]
    if case["op"] == "write":
        # K and V lie side by side in the projection's output row, as a fused projection leaves them
        kv = torch.randn(s.rows, 2, case["nkv"], case["dim"], device="cuda", generator=s.g)
        kv *= torch.exp(0.5 * torch.randn(s.rows, 1, case["nkv"], 1, device="cuda", generator=s.g))
        kv *= 1 + 6 * (torch.arange(case["dim"], device="cuda") % 37 == 5)
        return kv.to(dt)
    return (1.5 * torch.randn(s.rows, case["nq"], case["dim"], device="cuda", generator=s.g)).to(dt)


def prepare(case, seed):
    if case["op"] == "accept":
        s = _accept_inputs(case, seed)
        B, S = case["batch"], case["span"]
        s.length = s.n.clone()  # the forward of the span is all that the cache holds
        i32 = dict(device="cuda", dtype=torch.int32)
        s.n_accept, s.n_commit, s.new_len = (torch.zeros(B, **i32) for _ in range(3))
        s.committed = torch.zeros(B, S, **i32)
        if own:
            s.verifier = _verifier(case, s)
    else:
        s = _cache_inputs(case, seed)
        dt = DTYPES[case["dtype"]]
        if case["op"] == "attention":
            s.q = _rows_of(case, s)
            s.out = torch.empty_like(s.q)
        elif case["op"] == "write":
            s.kv = _rows_of(case, s)
        else:
            s.k, s.v = (torch.empty(s.rows, case["nkv"], case["dim"], device="cuda", dtype=dt) for _ in range(2))
        if own:
            from speculative_decoding_verify_02_gb300 import QuantCache
            s.cache = QuantCache(1, case.get("nq", case["nkv"]), case["nkv"], case["dim"], page_size=case["page"],
                                 n_pages=s.n_pages, max_batch=case["batch"], max_rows=s.rows, max_span=case["span"],
                                 max_context=s.context, scale_block=case["block"])
            s.cache.codes[0].copy_(s.codes)
            s.cache.scales[0].copy_(s.scales)
            s.codes, s.scales = s.cache.codes[0], s.cache.scales[0]
    s.case = dict(case)
    return s


def _verifier(case, s):
    """A context of the case's vocabulary whose cache holds each span, as after its forward."""
    from speculative_decoding_verify_02_gb300 import Verifier
    B, S, V = case["batch"], case["span"], case["vocab"]
    shape = types.SimpleNamespace(n_layers=1, hidden=128, n_q_heads=2, n_kv_heads=2, head_dim=64, ffn=128, vocab=V,
                                  rms_eps=1e-6, rope_theta=1e6, qk_norm=True)
    z = lambda *d: torch.zeros(*d, device="cuda", dtype=torch.bfloat16)  # noqa: E731
    w = {"embed": z(V, 128), "lm_head": z(V, 128), "final_norm": z(128)}
    for name, dims in dict(attn_norm=(128,), wq=(128, 128), wk=(128, 128), wv=(128, 128), q_norm=(64,), k_norm=(64,),
                           wo=(128, 128), ffn_norm=(128,), w_gate=(128, 128), w_up=(128, 128),
                           w_down=(128, 128)).items():
        w["layers.0." + name] = z(*dims)
    v = Verifier(shape, w, page_size=16, n_pages=B * (-(-S // 16)), max_batch=B, max_rows=max(s.rows, S), max_span=S,
                 max_context=S)
    v.ensure_capacity(s.n, B)
    v.spec_forward(torch.zeros_like(s.tokens), s.off, B, max(s.rows, S), S, torch.zeros_like(s.tokens))
    return v


# ---------------------------------------------------------------- a pass

def run(state):
    return {"attention": _run_attention, "write": _run_write, "read": _run_read, "accept": _run_accept}[state.case["op"]](state)


def _where(s):
    """The sequence, span index and position of each row."""
    r = torch.arange(s.rows, device="cuda", dtype=torch.int32)
    seq = torch.searchsorted(s.off, r, right=True) - 1
    i = r - s.off[seq]
    return seq, i, (s.base[seq] + i).long()


def _run_attention(s):
    c = s.case
    if own:
        s.cache.attention(0, s.q, s.table, s.off, s.base, c["batch"], c["span"], s.out, window=c["window"])
        return s.out
    B, S, ps, sb, D = c["batch"], c["span"], c["page"], c["block"], c["dim"]
    nq, nkv, grp = c["nq"], c["nkv"], c["nq"] // c["nkv"]
    at = s.table.long()
    scale = s.scales[at].repeat_interleave(sb, -1)[..., None]
    kv = s.codes[at].view(E4M3).float() * scale                      # [B, pages, 2, nkv, ps, D]
    k, v = kv.permute(2, 0, 3, 1, 4, 5).reshape(2, B, nkv, -1, D)
    seq, i, pos = _where(s)
    rows = (s.off[:-1, None] + torch.arange(S, device="cuda")).clamp_max(s.rows - 1).long()  # [B, S], padded
    q = s.q[rows].float().view(B, S, nkv, grp, D).permute(0, 2, 3, 1, 4).reshape(B, nkv, grp * S, D)
    scores = (q @ k.transpose(-1, -2) / math.sqrt(D)).view(B, nkv, grp, S, -1)
    qpos = s.base[:, None] + torch.arange(S, device="cuda")
    key = torch.arange(k.shape[2], device="cuda")
    seen = key <= qpos[..., None]
    if c["window"]:
        seen &= key > qpos[..., None] - c["window"]
    scores.masked_fill_(~seen[:, None, None], -math.inf)
    p = torch.exp(scores - scores.amax(-1, keepdim=True))
    p /= p.sum(-1, keepdim=True)
    o = (p.view(B, nkv, grp * S, -1) @ v).view(B, nkv, grp, S, D).permute(0, 3, 1, 2, 4).reshape(B, S, nq, D)
    return o[seq, i.long()].to(s.q.dtype)


def _needed_scale(amax):
    m, e = torch.frexp(amax)
    e = torch.where(m <= 0.875, e - 9, e - 8)  # 448 = 0.875 * 2^9
    e = torch.where(amax > 0, e, MIN_EXP).clamp_min(MIN_EXP)
    return torch.exp2(e.double()).float()


def _run_write(s):
    c = s.case
    if own:
        s.cache.write(0, s.kv[:, 0], s.kv[:, 1], s.table, s.off, s.base, c["batch"], c["span"])
        return {"codes": s.codes.view(E4M3), "scales": s.scales}
    ps, sb, nkv, D = c["page"], c["block"], c["nkv"], c["dim"]
    nblk = ps // sb
    seq, i, pos = _where(s)
    x = s.kv.float()
    page, slot = s.table[seq, pos // ps].long(), pos % ps
    block = page * nblk + slot // sb
    flat = s.scales.permute(0, 3, 1, 2).reshape(-1, 2, nkv)          # [page x block, 2, nkv]
    peak = x.abs().amax(-1)
    amax = torch.zeros_like(flat).scatter_reduce_(0, block[:, None, None].expand_as(peak), peak, "amax")
    scale = _needed_scale(amax)
    # the block that a span starts in keeps the rows below the span: its scale can only grow
    first = s.base.long()
    page0 = s.table.gather(1, (first // ps).clamp_max(s.table.shape[1] - 1)[:, None])[:, 0].long()
    block0 = page0 * nblk + (first % ps) // sb
    inside = ((first % sb > 0) & (s.n > 0))[:, None, None]
    old = flat[block0]
    grown = torch.where(inside, torch.maximum(old, scale[block0]), scale[block0])
    scale[block0] = grown
    touched = torch.zeros(flat.shape[0], device="cuda", dtype=torch.bool).index_fill_(0, block, True)
    flat = torch.where(touched[:, None, None], scale, flat)
    slots = ((first % ps) // sb * sb)[:, None] + torch.arange(sb, device="cuda")
    live = (slots < (first % ps)[:, None]) & inside[:, 0]
    kept = s.codes[page0[:, None], :, :, slots]                      # [B, sb, 2, nkv, D]
    again = (kept.view(E4M3).float() * (old / grown)[:, None, :, :, None]).to(E4M3).view(torch.uint8)
    s.codes[page0[:, None], :, :, slots] = torch.where(live[:, :, None, None, None], again, kept)
    s.codes[page, :, :, slot] = (x / flat[block][..., None]).to(E4M3).view(torch.uint8)
    s.scales.copy_(flat.view(-1, nblk, 2, nkv).permute(0, 2, 3, 1))
    return {"codes": s.codes.view(E4M3), "scales": s.scales}


def _run_read(s):
    c = s.case
    if own:
        s.cache.read(0, s.table, s.off, s.base, c["batch"], c["span"], s.k, s.v)
        return {"k": s.k, "v": s.v}
    ps, sb = c["page"], c["block"]
    seq, i, pos = _where(s)
    page, slot = s.table[seq, pos // ps].long(), pos % ps
    x = s.codes[page, :, :, slot].view(E4M3).float() * s.scales[page, :, :, slot // sb][..., None]
    return {"k": x[:, 0].to(s.k.dtype), "v": x[:, 1].to(s.v.dtype)}


def _run_accept(s):
    c = s.case
    B, S, V = c["batch"], c["span"], c["vocab"]
    if own:
        s.verifier.accept_sampled(s.tokens, s.off, s.logits, s.temperature, s.uniforms, s.noise, B, S, s.n_accept,
                                  s.committed, s.n_commit, s.new_len, draft_probs=s.probs)
        return {"n_accept": s.n_accept, "committed": s.committed, "n_commit": s.n_commit, "new_len": s.new_len}
    r = torch.arange(s.rows, device="cuda")
    seq = torch.searchsorted(s.off, r.to(torch.int32), right=True) - 1
    x = s.logits.double()  # decisions next to a border need more than 32 bits
    t = s.temperature[seq].double()[:, None]
    top = x.amax(-1, keepdim=True)
    best = torch.where(x == top, torch.arange(V, device="cuda"), V).amin(-1, keepdim=True)
    p = torch.exp((x - top) / torch.where(t > 0, t, 1.0))
    p /= p.sum(-1, keepdim=True)
    p = torch.where(t > 0, p, (torch.arange(V, device="cuda") == best).double())
    draft = s.tokens.roll(-1).long()[:, None]
    last = r == s.off[seq + 1] - 1
    q_draft = s.probs.gather(1, draft)[:, 0].double() if s.probs is not None else 1.0
    ok = (s.uniforms.double() * q_draft < p.gather(1, draft)[:, 0]) & ~last
    span = torch.arange(S, device="cuda")
    rows = (s.off[:-1, None] + span).clamp_max(s.rows - 1).long()
    m = (ok[rows] & (span < s.n[:, None] - 1)).int().cumprod(1).sum(1)
    at = (s.off[:-1] + m).clamp_max(s.rows - 1).long()               # the row that ends each span
    w = p[at]
    if s.probs is not None:
        other = s.probs[at].double()
    else:
        other = (torch.arange(V, device="cuda") == draft[at]).double()
    rest = (w - other).clamp_min(0)
    w = torch.where(((m < s.n - 1)[:, None]) & (rest.sum(-1, keepdim=True) > 0), rest, w)
    race = w / s.noise.double()  # the largest weight over exponential noise is a draw in proportion to the weights
    race = torch.where(w > 0, race, -1.0)
    won = race == race.amax(-1, keepdim=True)
    token = torch.where(won, torch.arange(V, device="cuda"), V).amin(-1).to(torch.int32)
    some = s.n > 0
    drafts = s.tokens[(rows + 1).clamp_max(s.rows - 1)]
    j, mm = span[None], m[:, None]
    s.committed.copy_(torch.where(some[:, None] & (j < mm), drafts, torch.where(some[:, None] & (j == mm), token[:, None],
                                                                              s.committed)))
    s.n_accept.copy_(torch.where(some, m, -1))
    s.n_commit.copy_(torch.where(some, m + 1, 0))
    s.new_len.copy_(torch.where(some, s.length - s.n + m + 1, -1))
    return {"n_accept": s.n_accept, "committed": s.committed, "n_commit": s.n_commit, "new_len": s.new_len}


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    B, S = case["batch"], case["span"]
    rows = B * S * (0.75 if case["ragged"] and B > 1 else 1.0)
    if case["op"] == "accept":
        return {"bytes": 4.0 * case["vocab"] * (rows + (2 if case["probs"] else 1) * B), "flops": 6.0 * case["vocab"] * rows}
    mid = (case["lo"] + case["hi"]) / 2
    per_token = 2 * case["nkv"] * (case["dim"] + 4.0 / case["block"])
    size = DTYPES[case["dtype"]].itemsize
    if case["op"] == "attention":
        keys = mid + S / 2
        tokens = B * (mid + S)
        if case["window"]:
            tokens, keys = min(tokens, B * (case["window"] + S)), min(keys, case["window"])
        return {"bytes": tokens * per_token + 2 * rows * case["nq"] * case["dim"] * size,
                "flops": 4.0 * rows * case["nq"] * case["dim"] * keys}
    return {"bytes": rows * (per_token + 2 * case["nkv"] * case["dim"] * size), "flops": 2.0 * rows * case["nkv"] * case["dim"]}


# ---------------------------------------------------------------- 64 bits

def _tokens64(codes, scales, table, n, ps, sb):
    """K and V of the first n tokens of one sequence, [2, nkv, n, D] in 64 bits."""
    pages = table[: -(-n // ps)].long()
    x = codes[pages].view(E4M3).double()
    x = x.view(*x.shape[:3], ps // sb, sb, x.shape[-1]) * scales[pages].double()[..., None, None]
    x = x.flatten(3, 4)
    return x.permute(1, 2, 0, 3, 4).flatten(2, 3)[:, :, :n]


def _to_e4m3_64(x):
    """x rounded to the nearest e4m3 value, ties to even, in 64 bits."""
    e = torch.frexp(x)[1].clamp_min(-5) - 4          # 4 significant bits; below 2^-6 the step stays 2^-9
    step = torch.exp2(e.double())
    return (x / step).round() * step


def exact(case, seed):
    if case["op"] == "accept":
        return _exact_accept(case, seed)
    s = _cache_inputs(case, seed)
    ps, sb = case["page"], case["block"]
    off, base = s.off.tolist(), s.base.tolist()
    if case["op"] == "attention":
        q = _rows_of(case, s)
        grp = case["nq"] // case["nkv"]
        out = torch.empty(q.shape, device="cuda", dtype=torch.float64)
        for b in range(case["batch"]):
            S = off[b + 1] - off[b]
            if S == 0:
                continue
            kv = _tokens64(s.codes, s.scales, s.table[b], base[b] + S, ps, sb)
            pos = base[b] + torch.arange(S, device="cuda")[:, None]
            key = torch.arange(base[b] + S, device="cuda")[None]
            hidden = key > pos
            if case["window"]:
                hidden |= key <= pos - case["window"]
            for h in range(case["nq"]):
                z = q[off[b]:off[b + 1], h].double() @ kv[0, h // grp].T * case["dim"] ** -0.5
                out[off[b]:off[b + 1], h] = torch.softmax(z.masked_fill(hidden, -math.inf), -1) @ kv[1, h // grp]
        return out
    if case["op"] == "read":
        k, v = [], []
        for b in range(case["batch"]):
            kv = _tokens64(s.codes, s.scales, s.table[b], base[b] + off[b + 1] - off[b], ps, sb)[:, :, base[b]:]
            k.append(kv[0].transpose(0, 1))
            v.append(kv[1].transpose(0, 1))
        return {"k": torch.cat(k), "v": torch.cat(v)}
    rows = _rows_of(case, s).double()
    codes, scales = s.codes.view(E4M3).double(), s.scales.double()
    for b in range(case["batch"]):
        p, end = base[b], base[b] + off[b + 1] - off[b]
        while p < end:
            stop = min(end, (p // sb + 1) * sb)
            page, a, blk = int(s.table[b, p // ps]), p % ps, p % ps // sb
            x = rows[off[b] + p - base[b]:off[b] + stop - base[b]].permute(1, 2, 0, 3)    # [2, nkv, rows, D]
            peak = x.abs().amax((-1, -2))
            need = torch.exp2(torch.log2((peak / E4M3_MAX).clamp_min(2.0 ** MIN_EXP)).round())
            need = torch.where(peak > E4M3_MAX * need, 2 * need, need)  # the nearest power, or its double
            if p % sb:
                was = scales[page, :, :, blk]
                need = torch.maximum(need, was)
                lower = codes[page, :, :, blk * sb:a]
                codes[page, :, :, blk * sb:a] = _to_e4m3_64(lower * (was / need)[..., None, None])
            scales[page, :, :, blk] = need
            codes[page, :, :, a:a + stop - p] = _to_e4m3_64(x / need[..., None, None])
            p = stop
    return {"codes": codes, "scales": scales}


def _exact_accept(case, seed):
    s = _accept_inputs(case, seed)
    off, temps = s.off.tolist(), s.temperature.tolist()
    B, V = case["batch"], case["vocab"]
    out = {k: torch.zeros(B, dtype=torch.int32) for k in ("n_accept", "n_commit", "new_len")}
    out["committed"] = torch.zeros(B, case["span"], dtype=torch.int32)
    for b in range(B):
        m, S = 0, off[b + 1] - off[b]
        while True:
            r = off[b] + m
            x = s.logits[r].double().cpu()
            if temps[b] > 0:
                p = torch.softmax(x / s.temperature[b].double().cpu(), 0)
            else:
                p = torch.zeros(V, dtype=torch.float64)
                p[int(torch.nonzero(x == x.max())[0])] = 1.0
            u = float(s.uniforms[r].double())
            if m == S - 1:
                break
            d = int(s.tokens[r + 1])
            if s.probs is not None:
                q = s.probs[r].double().cpu()
            else:
                q = torch.zeros(V, dtype=torch.float64)
                q[d] = 1.0
            if not u * float(q[d]) < float(p[d]):
                left = (p - q).clamp_min(0)
                p = left if float(left.sum()) > 0 else p
                break
            out["committed"][b, m] = d
            m += 1
        race = torch.log(p) - torch.log(s.noise[b].double().cpu())
        out["committed"][b, m] = int(torch.nonzero(race == race.max())[0])
        out["n_accept"][b], out["n_commit"][b], out["new_len"][b] = m, m + 1, m + 1
    return out
