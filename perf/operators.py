"""The operators of the target's verification pass, measured: one case of work at a time.

A drafted block is answered by the target model in one pass over its own cache: the block's keys and values are
rotated and appended to the paged cache, the block's rows attend to it, and the target's logits decide which drafts
stay.  Three operators, each in its plain form (elementary torch operations) and, with `own` set, as a user calls the
framework's kernels:

  append     q, k normed and rotated by their positions, k and v written into their pages
  attention  every new row over the cached keys up to its own, split over the length and joined
  verify     drafts kept while u q(x) < p(x), then one token from what p leaves over q

A case is a dict of plain values; sizes are those of the Qwen3-8B-shaped workloads (32 heads, 8 key/value heads of
128, a vocabulary of 151936, blocks of 16 rows, contexts of 2048 to 32768, 32 sequences, prompts of 8192 rows) and of
the small test geometries (heads of 64, a vocabulary of 5003).
"""
import math
import random

import numpy as np
import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn}
BYTES = {"bf16": 2, "f16": 2, "f32": 4, "e4m3": 1}


# ------------------------------------------------------------------ the cases
def _append(name, **kw):
    c = dict(name=name, op="append", n=1, rows=1, ragged=False, heads=32, kv_heads=8, head_dim=128, page=16,
             dtype="bf16", cache="bf16", ctx=4096, rotary=128, interleaved=False, scaling="none", norm=False)
    return {**c, **kw}


def _attention(name, **kw):
    c = dict(name=name, op="attention", n=1, rows=1, ragged=False, heads=32, kv_heads=8, head_dim=128, page=16,
             dtype="bf16", cache="bf16", ctx=4096, window=0, lse=False)
    return {**c, **kw}


def _verify(name, **kw):
    c = dict(name=name, op="verify", n=1, drafts=15, ragged=False, vocab=151936, dtype="f32", draft="logits",
             temperature=0.8)
    return {**c, **kw}


def listed():
    return [
        # plain decoding of one stream: the smallest call, one row a layer
        _append("append_token"),
        # 32 streams, each with a drafted block; Qwen3's head norms; an 8-bit cache with scales
        _append("append_blocks_e4m3", n=32, rows=16, cache="e4m3", page=64, norm=True),
        # a prompt's rows in one call; half of each head rotated, interleaved pairs, frequencies scaled for long contexts
        _append("append_prompt", rows=8192, ctx=32768, page=64, rotary=64, interleaved=True, scaling="yarn"),
        # small heads, drafts of different lengths, float16
        _append("append_ragged_hd64", n=9, rows=8, ragged=True, heads=12, kv_heads=4, head_dim=64, rotary=64,
                dtype="f16", cache="f16", page=32, ctx=1024),
        # one stream, one new token: latency
        _attention("token_ctx2048", ctx=2048),
        # 32 streams of different lengths, one new token each: the everyday decoding step
        _attention("tokens_batch32", n=32, ragged=True),
        # a drafted block against a long context
        _attention("block_ctx32768", rows=16, ctx=32768, page=64, lse=True),
        # 32 streams, a drafted block each, an 8-bit cache
        _attention("blocks_batch32_e4m3", n=32, rows=16, ragged=True, cache="e4m3", page=64),
        # many long streams, one new token each: the largest cache
        _attention("tokens_long", n=16, ctx=32768, page=64),
        # greedy verification of one block: drafts against the target's own top tokens
        _verify("verify_one_greedy", draft="tokens", temperature=0.0),
        # sampled verification of one block against the drafter's probabilities
        _verify("verify_one"),
        # 32 blocks of different lengths, the target's logits in 16 bits
        _verify("verify_batch32", n=32, ragged=True, dtype="bf16"),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(("append", "attention", "attention", "verify"))
    if op == "verify":
        drafts = rng.randint(0, 16)
        vocab = _log_int(rng, 1000, 160000)
        n = _log_int(rng, 1, max(1, min(48, 73_000_000 // (vocab * (drafts + 1)))))
        return dict(op=op, n=n, drafts=drafts, ragged=rng.random() < 0.5, vocab=vocab,
                    dtype=rng.choice(("f32", "bf16", "f16")), draft=rng.choice(("logits", "tokens")),
                    temperature=rng.choice((0.0, 0.6, 0.8, 1.0, 1.3)))
    kv_heads = rng.choice((1, 2, 4, 8))
    heads = kv_heads * rng.choice((1, 2, 3, 4, 5, 8))
    dtype = rng.choice(("bf16", "f16"))
    c = dict(op=op, n=_log_int(rng, 1, 48), ragged=rng.random() < 0.6, heads=heads, kv_heads=kv_heads,
             head_dim=rng.choice((64, 128)), page=rng.choice((1, 7, 16, 32, 48, 64, 128)), dtype=dtype,
             cache=rng.choice((dtype, dtype, "e4m3")))
    if op == "append":
        c["rows"] = _log_int(rng, 1, max(1, 8192 // c["n"]))
        c["ctx"] = _log_int(rng, max(64, c["rows"]), 131072)
        c["rotary"] = c["head_dim"] // rng.choice((1, 1, 2, 4))
        c["interleaved"] = rng.random() < 0.4
        c["scaling"] = rng.choice(("none", "linear", "yarn"))
        c["norm"] = rng.random() < 0.5
    else:
        c["rows"] = _log_int(rng, 1, 16)
        # up to the largest listed cache, and up to the scores that the largest listed block has
        most = min(131072, 16 * 32768 * 8 * 128 // (c["n"] * kv_heads * c["head_dim"]),
                   32 * 16 * 4096 * 32 // (c["n"] * c["rows"] * heads))
        c["ctx"] = _log_int(rng, 16, max(16, most))
        c["window"] = rng.choice((0, 0, 0, _log_int(rng, 8, 4096)))
        c["lse"] = rng.random() < 0.3
    return c


# ------------------------------------------------------------------ what a case's sequences hold
def _spread(case, key, lo, hi):
    """One whole number of [lo, hi] a sequence: the same for every seed, so that the work is the case's."""
    r = random.Random("%s %s %s %s" % (key, case["n"], lo, hi))
    return [r.randint(lo, hi) for _ in range(case["n"])] if case["ragged"] else [hi] * case["n"]


def _rows_of(case):
    return _spread(case, "rows", 1, case["rows"])


def _lens_of(case):
    """Tokens in each sequence's cache once its new rows are in."""
    rows = _rows_of(case)
    return [max(r, l) for r, l in zip(rows, _spread(case, "ctx", max(1, case["ctx"] // 4), case["ctx"]))]


def _drafts_of(case):
    return _spread(case, "drafts", case["drafts"] // 3, case["drafts"])


def _starts(counts):
    return [0] + list(np.cumsum(counts))


def _visible(case):
    """Sum over the new rows of the keys each sees."""
    w = case["window"]
    tot = 0
    for r, l in zip(_rows_of(case), _lens_of(case)):
        for p in range(l - r, l):
            tot += min(p + 1, w) if w else p + 1
    return tot


def work(case):
    n = case["n"]
    if case["op"] == "verify":
        d = sum(_drafts_of(case))
        b = (d + n) * case["vocab"] * BYTES[case["dtype"]] + 12 * d + 16 * n
        if case["draft"] == "logits" and case["temperature"] > 0:
            b += d * case["vocab"] * 4
        return {"bytes": b, "flops": 4 * (d + n) * case["vocab"]}
    rows, hd, kvh = sum(_rows_of(case)), case["head_dim"], case["kv_heads"]
    e, ec = BYTES[case["dtype"]], BYTES[case["cache"]]
    if case["op"] == "append":
        b = rows * hd * (2 * case["heads"] * e + 2 * kvh * (e + ec))
        return {"bytes": b, "flops": 6 * rows * hd * (case["heads"] + kvh)}
    w = case["window"]
    keys = sum(min(l, w + r - 1) if w else l for r, l in zip(_rows_of(case), _lens_of(case)))
    b = keys * kvh * hd * 2 * ec + 2 * rows * case["heads"] * hd * e + (rows * case["heads"] * 4 if case["lse"] else 0)
    return {"bytes": b, "flops": 4 * _visible(case) * case["heads"] * hd}


# ------------------------------------------------------------------ inputs
def _inv_freq(case):
    """Rotation frequencies in 64 bits: theta^(-2i/d), unscaled, slowed by a factor, or slowed where a context of the
    trained length turns less than once (with the matching growth of the rotated length)."""
    d, theta, factor, trained = case["rotary"], 1e6, 4.0, 8192
    f = theta ** (-np.arange(0, d, 2, dtype=np.float64) / d)
    if case["scaling"] == "linear":
        return f / factor, 1.0
    if case["scaling"] == "yarn":
        at = lambda turns: d * math.log(trained / (turns * 2 * math.pi)) / (2 * math.log(theta))  # noqa: E731
        lo, hi = max(math.floor(at(32)), 0), min(math.ceil(at(1)), d - 1)
        ramp = np.clip((np.arange(d // 2, dtype=np.float64) - lo) / max(hi - lo, 1e-3), 0, 1)
        return f / factor * ramp + f * (1 - ramp), 0.1 * math.log(factor) + 1.0
    return f, 1.0


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(dev).manual_seed(seed)
    randn = lambda *s, dtype=torch.float32: torch.randn(*s, device=dev, generator=gen, dtype=dtype)  # noqa: E731
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
    st = {"case": case}
    if case["op"] == "verify":
        n, V, counts = case["n"], case["vocab"], _drafts_of(case)
        d = sum(counts)
        # the target's logits and a drafter's that mostly agrees with them; drafts sampled from the drafter's
        target = 2.5 * randn(d + n, V)
        seq = np.repeat(np.arange(n), counts)
        rows = torch.tensor(np.arange(d) + seq, device=dev, dtype=torch.int64)
        draft = target[rows] + 0.7 * randn(d, V)
        T = case["temperature"] or 0.5
        gumbel = -torch.log(-torch.log(torch.rand(d, V, device=dev, generator=gen).clamp_(1e-9, 1 - 1e-7)))
        st["draft_tokens"] = (draft / T + gumbel).argmax(-1).to(torch.int32) if d else ints([])
        st["target_logits"] = target.to(TYPES[case["dtype"]])
        st["draft_logits"] = draft if case["draft"] == "logits" else None
        st["accept_u"] = torch.rand(d, device=dev, generator=gen)
        st["sample_u"] = torch.rand(n, device=dev, generator=gen)
        st["draft_start"] = ints(_starts(counts)) if case["ragged"] else None
        st["temperature"] = torch.full((n,), case["temperature"], device=dev)
        return st
    rows, lens = _rows_of(case), _lens_of(case)
    n, R, page, kvh, hd = case["n"], sum(rows), case["page"], case["kv_heads"], case["head_dim"]
    dt, cd = TYPES[case["dtype"]], TYPES[case["cache"]]
    # pages are dealt out of a shuffled pool.  An append touches only the pages of its new rows: there the pages of
    # earlier tokens are no longer held (-1), as in a layer whose window has moved past them.
    first = [max(0, (l - r) // page) if case["op"] == "append" else 0 for r, l in zip(rows, lens)]
    held = [-(-l // page) - f for f, l in zip(first, lens)]
    width = max(f + h for f, h in zip(first, held))
    pool = torch.randperm(sum(held) + 3, generator=torch.Generator().manual_seed(seed)).tolist()
    table = np.full((n, width), -1, dtype=np.int32)
    at = 0
    for s in range(n):
        table[s, first[s]:first[s] + held[s]] = pool[at:at + held[s]]
        at += held[s]
    st["table"] = torch.from_numpy(table).to(dev)
    st["kv_len"] = ints(lens)
    st["row_start"] = ints(_starts(rows)) if case["ragged"] else None
    shape = (sum(held) + 3, page, kvh, hd)
    if case["cache"] == "e4m3":
        st["k_cache"], st["v_cache"] = (randn(*shape, dtype=torch.bfloat16).mul_(32).to(cd) for _ in range(2))
        st["k_scale"], st["v_scale"] = ((0.5 + torch.rand(kvh, device=dev, generator=gen)) / 32 for _ in range(2))
    else:
        st["k_cache"], st["v_cache"] = (randn(*shape, dtype=cd) for _ in range(2))
        st["k_scale"] = st["v_scale"] = None
    if case["op"] == "append":
        # q, k and v as a fused projection leaves them: slices of one row
        qkv = randn(R, case["heads"] + 2 * kvh, hd).to(dt)
        st["q"], st["k"], st["v"] = qkv.split((case["heads"], kvh, kvh), 1)
        f, scale = _inv_freq(case)
        st["inv_freq"], st["rope_scale"] = torch.from_numpy(f).to(dev), scale
        st["q_norm"], st["k_norm"] = ((1 + 0.1 * randn(hd) for _ in range(2)) if case["norm"] else (None, None))
    else:
        st["q"] = randn(R, case["heads"], hd).to(dt)
    return st


# ------------------------------------------------------------------ one pass
def run(state):
    return {"append": _run_append, "attention": _run_attention, "verify": _run_verify}[state["case"]["op"]](state)


def _positions(st, R):
    """Each row's sequence, place in its sequence and position."""
    n, dev = st["case"]["n"], st["kv_len"].device
    r = torch.arange(R, device=dev)
    if st["row_start"] is None:
        per = R // n
        seq, i, rows = r // per, r % per, torch.full_like(st["kv_len"], per)
    else:
        start = st["row_start"].long()
        seq = torch.searchsorted(start[1:].contiguous(), r, right=True)
        i, rows = r - start[seq], start[1:] - start[:-1]
    return seq, i, (st["kv_len"] - rows)[seq].long() + i


def _run_append(st):
    case = st["case"]
    if own:
        import block_speculative_drafting_gb300 as dfl
        q = dfl.paged_append(st["k_cache"], st["v_cache"], st["k"], st["v"], st["table"], st["kv_len"],
                             row_start=st["row_start"], q=st["q"], inv_freq=st["inv_freq"],
                             interleaved=case["interleaved"], rope_scale=st["rope_scale"], q_norm=st["q_norm"],
                             k_norm=st["k_norm"], k_scale=st["k_scale"], v_scale=st["v_scale"])
        return [q, st["k_cache"], st["v_cache"]]
    R = st["k"].shape[0]
    seq, _, pos = _positions(st, R)
    angle = pos[:, None].double() * st["inv_freq"]  # far positions turn many times: 64 bits
    cos, sin = ((f(angle) * st["rope_scale"]).float()[:, None] for f in (torch.cos, torch.sin))
    rot = case["rotary"]

    def turned(x, gain):
        x = x.float()
        if gain is not None:
            x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * gain
        a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if case["interleaved"] else (x[..., :rot // 2], x[..., rot // 2:rot])
        y = (a * cos - b * sin, a * sin + b * cos)
        y = torch.stack(y, -1).flatten(-2) if case["interleaved"] else torch.cat(y, -1)
        return torch.cat((y, x[..., rot:]), -1)

    page = st["table"][seq, pos // case["page"]].long()
    slot = pos % case["page"]
    for cache, x, scale in ((st["k_cache"], turned(st["k"], st["k_norm"]), st["k_scale"]),
                            (st["v_cache"], st["v"].float(), st["v_scale"])):
        if scale is not None:
            x = (x / scale[:, None]).clamp(-448, 448)
        x = x.to(cache.dtype)
        if scale is not None:
            cache, x = cache.view(torch.uint8), x.view(torch.uint8)
        cache[page, slot] = x
    return [turned(st["q"], st["q_norm"]).to(st["q"].dtype), st["k_cache"], st["v_cache"]]


def _run_attention(st):
    case, q = st["case"], st["q"]
    if own:
        import block_speculative_drafting_gb300 as dfl
        lse = torch.empty(q.shape[:2], dtype=torch.float32, device=q.device) if case["lse"] else None
        out = dfl.paged_attention(q, st["k_cache"], st["v_cache"], st["table"], st["kv_len"],
                                  row_start=st["row_start"], window=case["window"], k_scale=st["k_scale"],
                                  v_scale=st["v_scale"], lse=lse)
        return [out, lse] if case["lse"] else [out]
    n, kvh, hd = case["n"], case["kv_heads"], case["head_dim"]
    g = case["heads"] // kvh
    seq, i, pos = _positions(st, q.shape[0])
    held = st["table"].clamp(min=0).long()

    def gathered(cache, scale):  # every sequence's cache, padded: [n][keys][kv_heads][head_dim]
        if scale is None:
            return cache[held].flatten(1, 2).float()
        return cache.view(torch.uint8)[held].view(cache.dtype).flatten(1, 2).float() * scale[:, None]

    rows = case["rows"]
    qs = torch.zeros(n, rows, case["heads"], hd, device=q.device)
    qs[seq, i] = q.float()
    at = torch.full((n, rows), -1, device=q.device, dtype=torch.int64)
    at[seq, i] = pos
    qs = qs.view(n, rows, kvh, g, hd).permute(0, 2, 1, 3, 4).reshape(n, kvh, rows * g, hd)
    s = torch.matmul(qs, gathered(st["k_cache"], st["k_scale"]).permute(0, 2, 3, 1)) / math.sqrt(hd)
    key = torch.arange(s.shape[-1], device=q.device)
    seen = key <= at[..., None]
    if case["window"]:
        seen &= key > at[..., None] - case["window"]
    s.masked_fill_(~seen[:, None, :, None].expand(n, 1, rows, g, -1).reshape(n, 1, rows * g, -1), -math.inf)
    m = s.amax(-1, keepdim=True).clamp(min=-1e30)
    p = torch.exp(s - m)
    total = p.sum(-1, keepdim=True)
    y = torch.matmul(p / total.clamp(min=1e-30), gathered(st["v_cache"], st["v_scale"]).transpose(1, 2))
    back = lambda x: x.view(n, kvh, rows, g, -1).permute(0, 2, 1, 3, 4).flatten(2, 3)[seq, i]  # noqa: E731
    out = back(y).to(q.dtype)
    return [out, back(m + torch.log(total)).squeeze(-1)] if case["lse"] else [out]


def _run_verify(st):
    case = st["case"]
    if own:
        import block_speculative_drafting_gb300 as dfl
        return list(dfl.verify_drafts(st["target_logits"], st["draft_tokens"], st["accept_u"], st["sample_u"],
                                      draft_logits=st["draft_logits"], draft_start=st["draft_start"],
                                      temperature=st["temperature"]))
    n, V, d = case["n"], case["vocab"], st["draft_tokens"].shape[0]
    dev = st["sample_u"].device
    j = torch.arange(d, device=dev)
    if st["draft_start"] is None:
        per = d // n
        seq, first = (j // max(per, 1)), torch.arange(n, device=dev) * per
        count = torch.full((n,), per, device=dev)
    else:
        start = st["draft_start"].long()
        seq, first, count = torch.searchsorted(start[1:].contiguous(), j, right=True), start[:-1], start[1:] - start[:-1]
    logits, tok = st["target_logits"].float(), st["draft_tokens"].long()
    T = st["temperature"].double()

    def probabilities(x, t):  # 64 bits: a sum over the vocabulary, and borders that decide whole numbers
        x = x.double()
        if case["temperature"] == 0:
            return torch.zeros_like(x).scatter_(1, x.argmax(-1, keepdim=True), 1.0)
        e = torch.exp((x - x.amax(-1, keepdim=True)) / t[:, None])
        return e / e.sum(-1, keepdim=True)

    row_seq = torch.searchsorted((first + torch.arange(n, device=dev)).contiguous(), torch.arange(d + n, device=dev),
                                 right=True) - 1
    p = probabilities(logits, T[row_seq])
    px = p[j + seq, tok]
    sampled = st["draft_logits"] is not None and case["temperature"] > 0
    qp = probabilities(st["draft_logits"], T[seq]) if sampled else None
    qx = qp[j, tok] if sampled else torch.ones_like(px)
    kept = st["accept_u"].double() * qx < px
    # the drafts of a sequence before its first refusal
    refused = torch.full((n,), d, device=dev).scatter_reduce(0, seq, torch.where(kept, d, j - first[seq]), "amin")
    accepted = torch.minimum(refused, count)
    row = first + torch.arange(n, device=dev) + accepted
    rest = p[row]
    if d:
        jd = (first + accepted).clamp(max=d - 1)
        if sampled:
            q_row = qp[jd]
        else:
            q_row = torch.zeros_like(rest).scatter_(1, tok[jd][:, None], 1.0)
        over = (rest - q_row).clamp(min=0) if case["temperature"] > 0 else rest
        rest = torch.where((accepted < count)[:, None], over, rest)
    c = rest.cumsum(-1)
    token = (c <= st["sample_u"].double()[:, None] * c[:, -1:]).sum(-1)
    prob = torch.minimum(px / qx, torch.ones_like(px))
    return [accepted.to(torch.int32), token.to(torch.int32), prob.float()]


# ------------------------------------------------------------------ the definition in 64 bits
def exact(case, seed):
    """The definition, one sequence at a time, in 64 bits."""
    st = prepare(case, seed)
    if case["op"] == "verify":
        return _exact_verify(case, st)
    rows, lens = _rows_of(case), _lens_of(case)
    at = _starts(rows)
    table, page = st["table"].tolist(), case["page"]
    if case["op"] == "append":
        return _exact_append(case, st, rows, lens, at, table, page)
    kvh, g, hd = case["kv_heads"], case["heads"] // case["kv_heads"], case["head_dim"]
    out, lses = [], []
    for s in range(case["n"]):
        L, r = lens[s], rows[s]
        pages = torch.tensor(table[s][:-(-L // page)], device="cuda")

        def read(cache, scale):
            x = (cache.view(torch.uint8)[pages].view(cache.dtype) if scale is not None else cache[pages])
            x = x.reshape(-1, kvh, hd)[:L].double()
            return x * scale.double()[None, :, None] if scale is not None else x

        k, v = read(st["k_cache"], st["k_scale"]), read(st["v_cache"], st["v_scale"])
        q = st["q"][at[s]:at[s + 1]].double().view(r, kvh, g, hd)
        sc = torch.einsum("rkgd,lkd->kgrl", q, k) * hd ** -0.5
        pos = torch.arange(L - r, L, device="cuda")[:, None]
        key = torch.arange(L, device="cuda")[None]
        hide = key > pos
        if case["window"]:
            hide = hide | (key <= pos - case["window"])
        sc = sc.masked_fill(hide, -math.inf)
        lse = torch.logsumexp(sc, -1)
        out.append(torch.einsum("kgrl,lkd->rkgd", torch.exp(sc - lse[..., None]), v).reshape(r, kvh * g, hd))
        lses.append(lse.permute(2, 0, 1).reshape(r, kvh * g))
    return [torch.cat(out), torch.cat(lses)] if case["lse"] else [torch.cat(out)]


def _exact_append(case, st, rows, lens, at, table, page):
    f, scale = _inv_freq(case)
    f = torch.from_numpy(f).cuda()
    rot, h = case["rotary"], case["rotary"] // 2
    caches = [st[c].double() for c in ("k_cache", "v_cache")]
    qs = []
    for s in range(case["n"]):
        r, part = rows[s], slice(at[s], at[s + 1])
        pos = torch.arange(lens[s] - r, lens[s], device="cuda", dtype=torch.float64)
        turn = torch.polar(torch.full((r, 1, h), scale, dtype=torch.float64, device="cuda"),
                           (pos[:, None] * f)[:, None])
        done = []
        for x, gain in ((st["q"], st["q_norm"]), (st["k"], st["k_norm"])):
            x = x[part].double()
            if gain is not None:
                x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / case["head_dim"] + 1e-6) * gain.double()
            head = x[..., :rot].unflatten(-1, (h, 2) if case["interleaved"] else (2, h))
            if not case["interleaved"]:
                head = head.transpose(-1, -2)
            z = torch.view_as_real(torch.view_as_complex(head.contiguous()) * turn)
            if not case["interleaved"]:
                z = z.transpose(-1, -2)
            done.append(torch.cat((z.flatten(-2), x[..., rot:]), -1))
        qs.append(done[0])
        slots = [(table[s][p // page], p % page) for p in range(lens[s] - r, lens[s])]
        pg, sl = (torch.tensor(x, device="cuda") for x in zip(*slots))
        for cache, x, sc in ((caches[0], done[1], st["k_scale"]), (caches[1], st["v"][part].double(), st["v_scale"])):
            if sc is not None:
                x = (x / sc.double()[None, :, None]).clamp(-448, 448)
            cache[pg, sl] = x
    return [torch.cat(qs)] + caches


def _exact_verify(case, st):
    counts = _drafts_of(case)
    at, T = _starts(counts), float(st["temperature"][0])
    accepted, token, prob = [], [], []

    def softmax(x):
        if T == 0:
            y = torch.zeros_like(x, dtype=torch.float64)
            y[int((x == x.max()).nonzero()[0])] = 1.0
            return y
        return torch.softmax(x.double() / T, -1)

    for s in range(case["n"]):
        d, row0, a = counts[s], at[s] + s, None
        for i in range(d):
            p = softmax(st["target_logits"][row0 + i].float())
            x = int(st["draft_tokens"][at[s] + i])
            q = None
            if st["draft_logits"] is not None and T > 0:
                q = softmax(st["draft_logits"][at[s] + i])
            qx = float(q[x]) if q is not None else 1.0
            prob.append(min(1.0, float(p[x]) / qx))
            if a is None and not float(st["accept_u"][at[s] + i]) * qx < float(p[x]):
                a = i
                if T > 0:
                    if q is None:
                        p[x] = 0.0
                        rest = p
                    else:
                        rest = torch.relu(p - q)
                else:
                    rest = p
        if a is None:
            a, rest = d, softmax(st["target_logits"][row0 + d].float())
        c = torch.cumsum(rest, 0)
        accepted.append(a)
        token.append(int((c > float(st["sample_u"][s]) * c[-1]).nonzero()[0]))
    return [torch.tensor(accepted, dtype=torch.int32), torch.tensor(token, dtype=torch.int32),
            torch.tensor(prob, dtype=torch.float64)]
