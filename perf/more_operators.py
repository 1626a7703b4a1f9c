"""The operators that keep the target's cache small, measured: one case of work at a time.

The target's keys and values can be held in 4 bits, and a cache that has grown long can be cut back to the tokens that
its queries look at.  Each operator in its plain form (elementary torch operations) and, with `own` set, as a user
calls the framework's kernels:

  append     keys and values rounded into the 4-bit paged cache (e2m1 codes, an e4m3 scale for 16 columns, one f32
             scale a head), and the new rows read back as what the cache now holds
  attention  every new row over the 4-bit cached keys up to its own
  weights    what attention weight each cached key has received, added up over rows and the heads that share it
  evict      of a cache over its budget, the heaviest keys kept, first and recent ones always, and moved together

A case is a dict of plain values; sizes are those of the Qwen3-8B-shaped workloads (32 heads, 8 key/value heads of
128, blocks of 16 rows, contexts of 2048 to 32768, 32 sequences, prompts of 8192 rows) and of the small test
geometries (heads of 64).
"""
import math
import random

import numpy as np
import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn}
BYTES = {"bf16": 2, "f16": 2, "f32": 4, "e4m3": 1, "e2m1": 0.5 + 1 / 16}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------ the cases
def _case(name, op, **kw):
    c = dict(name=name, op=op, n=1, rows=1, ragged=False, kv_heads=8, head_dim=128, page=16, ctx=4096)
    if op == "append":
        c.update(dtype="bf16")
    elif op == "attention":
        c.update(heads=32, dtype="bf16", window=0, lse=False)
    elif op == "weights":
        c.update(heads=32, dtype="bf16", cache="bf16", window=0)
    else:
        c.update(cache="bf16", keep=2048, first=4, recent=128)
    return {**c, **kw}


def listed():
    return [
        # plain decoding of one stream: the smallest call, one row a layer
        _case("append4_token", "append"),
        # 32 streams, each with a drafted block
        _case("append4_blocks", "append", n=32, rows=16, page=64),
        # a prompt's rows in one call
        _case("append4_prompt", "append", rows=8192, ctx=32768, page=64),
        # one stream, one new token: latency
        _case("token4_ctx2048", "attention", ctx=2048),
        # 32 streams of different lengths, one new token each: the everyday decoding step
        _case("tokens4_batch32", "attention", n=32, ragged=True, lse=True),
        # 32 streams, a drafted block each
        _case("blocks4_batch32", "attention", n=32, rows=16, ragged=True, page=64),
        # many long streams, one new token each: what 4 bits are for
        _case("tokens4_long", "attention", n=16, ctx=32768, page=64),
        # 32 streams, one new token each: the weights beside an everyday decoding step
        _case("weights_batch32", "weights", n=32, ragged=True),
        # a drafted block over a long 4-bit cache
        _case("weights_block", "weights", rows=16, ctx=32768, cache="e2m1", page=64),
        # a prompt's last part over the whole prompt
        _case("weights_prompt", "weights", rows=2048, ctx=16384, page=64),
        # one long stream cut to half
        _case("evict_long", "evict", ctx=32768, keep=16384, page=64),
        # 32 streams of different lengths cut to one budget, an 8-bit cache
        _case("evict_batch32", "evict", n=32, ragged=True, cache="e4m3", page=64),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(("append", "attention", "attention", "weights", "weights", "evict"))
    kv_heads = rng.choice((1, 2, 4, 8))
    heads = kv_heads * rng.choice((1, 2, 3, 4, 5, 8))
    c = dict(op=op, n=_log_int(rng, 1, 48), ragged=rng.random() < 0.6, kv_heads=kv_heads,
             head_dim=rng.choice((64, 128)), page=rng.choice((1, 7, 16, 32, 48, 64, 128)))
    if op == "append":
        c["rows"] = _log_int(rng, 1, max(1, 8192 // c["n"]))
        c["ctx"] = _log_int(rng, max(64, c["rows"]), 131072)
        c["dtype"] = rng.choice(("bf16", "f16", "f32"))
        return c
    # up to the largest listed cache
    most = min(131072, 16 * 32768 * 8 * 128 // (c["n"] * kv_heads * c["head_dim"]))
    if op == "evict":
        c["rows"] = 1
        c["cache"] = rng.choice(("bf16", "f16", "e4m3", "e2m1"))
        c["ctx"] = _log_int(rng, 64, max(64, most // 4))
        c["keep"] = _log_int(rng, 16, c["ctx"])
        c["first"] = rng.choice((0, 1, 4, 8))
        c["recent"] = rng.randint(0, c["keep"] - 8)
        return c
    c["heads"] = heads
    c["dtype"] = rng.choice(("bf16", "f16"))
    c["window"] = rng.choice((0, 0, 0, _log_int(rng, 8, 4096)))
    if op == "attention":
        c["rows"] = _log_int(rng, 1, 16)
        c["lse"] = rng.random() < 0.5
        scores = 32 * 16 * 4096 * 32
    else:
        c["rows"] = _log_int(rng, 1, max(1, 512 // c["n"]))
        c["cache"] = rng.choice((c["dtype"], "e4m3", "e2m1", "e2m1"))
        most = most // 2
        scores = 2048 * 16384 * 32 // 8
    c["ctx"] = _log_int(rng, max(16, c["rows"]), max(16, c["rows"], min(most, scores // (c["n"] * c["rows"] * heads))))
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
    rows, hd, kvh = sum(_rows_of(case)), case["head_dim"], case["kv_heads"]
    lens = _lens_of(case)
    if case["op"] == "append":  # keys and values in, codes and what they stand for out
        return {"bytes": 2 * rows * kvh * hd * (BYTES[case["dtype"]] + BYTES["e2m1"] + 2), "flops": 6 * rows * kvh * hd}
    if case["op"] == "evict":  # every weight in; the kept tokens of a cache over its budget read and written
        over = sum(l > case["keep"] for l in lens)
        b = kvh * (4 * sum(lens) + over * case["keep"] * (4 * hd * BYTES[case["cache"]] + 4) + 4 * case["n"] * case["keep"])
        return {"bytes": b, "flops": 2 * kvh * sum(lens)}
    w = case["window"]
    keys = sum(min(l, w + r - 1) if w else l for r, l in zip(_rows_of(case), lens))
    e, q = BYTES[case["dtype"]], rows * case["heads"] * hd
    if case["op"] == "attention":
        b = keys * kvh * hd * 2 * BYTES["e2m1"] + 2 * q * e + (rows * case["heads"] * 4 if case["lse"] else 0)
        return {"bytes": b, "flops": 4 * _visible(case) * case["heads"] * hd}
    b = keys * kvh * (hd * BYTES[case["cache"]] + 8) + q * e + rows * case["heads"] * 4
    return {"bytes": b, "flops": 2 * _visible(case) * case["heads"] * hd}


# ------------------------------------------------------------------ 4 bits in plain operations
def _e2m1_blocks(t):
    """[..][16 b] in units of the head's scale -> codes [..][8 b] uint8 (the first of two in the lower bits) and the
    blocks' e4m3 scales [..][b]."""
    t = t.unflatten(-1, (-1, 16))
    s = (t.abs().amax(-1) / 6).clamp(max=448).to(torch.float8_e4m3fn)
    u = t / s.float()[..., None].clamp(min=2.0 ** -9)
    a = u.abs()
    # a value between two codes goes to the nearer, half way to the even one
    c = torch.zeros_like(a, dtype=torch.uint8)
    for k, edge in enumerate((0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)):
        c += (a > edge) if k % 2 == 0 else (a >= edge)
    c = (c + 8 * (u < 0)).to(torch.uint8).flatten(-2)
    return c[..., 0::2] | (c[..., 1::2] << 4), s


def _e2m1_values(codes, blocks, scale):
    """Codes [..][kv_heads][8 b], block scales and the heads' scales as f32 values."""
    table = torch.tensor(E2M1 + tuple(-x for x in E2M1), device=codes.device)
    x = torch.stack((codes & 15, codes >> 4), -1).flatten(-2)
    return (table[x.int()].unflatten(-1, (-1, 16)) * blocks.float()[..., None]).flatten(-2) * scale[:, None]


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(dev).manual_seed(seed)
    randn = lambda *s, dtype=torch.float32: torch.randn(*s, device=dev, generator=gen, dtype=dtype)  # noqa: E731
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
    op, rows, lens = case["op"], _rows_of(case), _lens_of(case)
    n, R, page, kvh, hd = case["n"], sum(rows), case["page"], case["kv_heads"], case["head_dim"]
    kind = case.get("cache", "e2m1")
    # pages are dealt out of a shuffled pool.  An append touches only the pages of its new rows: there the pages of
    # earlier tokens are no longer held (-1).
    first = [max(0, (l - r) // page) if op == "append" else 0 for r, l in zip(rows, lens)]
    held = [-(-l // page) - f for f, l in zip(first, lens)]
    width = max(f + h for f, h in zip(first, held))
    pool = torch.randperm(sum(held) + 3, generator=torch.Generator().manual_seed(seed)).tolist()
    table = np.full((n, width), -1, dtype=np.int32)
    at = 0
    for s in range(n):
        table[s, first[s]:first[s] + held[s]] = pool[at:at + held[s]]
        at += held[s]
    st = {"case": case, "table": torch.from_numpy(table).to(dev), "kv_len": ints(lens),
          "row_start": ints(_starts(rows)) if case["ragged"] else None}
    shape = (sum(held) + 3, page, kvh, hd)
    for x in "kv":
        st[x + "_scale"] = st[x + "_block"] = None
        if kind == "e2m1":
            st[x + "_scale"] = (0.5 + torch.rand(kvh, device=dev, generator=gen)) / 64
            codes = torch.empty(*shape[:3], hd // 2, dtype=torch.uint8, device=dev)
            blocks = torch.empty(*shape[:3], hd // 16, dtype=torch.float8_e4m3fn, device=dev)
            step = max(1, (1 << 26) // (page * kvh * hd))
            for p in range(0, shape[0], step):
                m = min(step, shape[0] - p)
                c, b = _e2m1_blocks(randn(m, *shape[1:]) / st[x + "_scale"][:, None])
                codes[p:p + m] = c
                blocks.view(torch.uint8)[p:p + m] = b.view(torch.uint8)
            st[x + "_cache"], st[x + "_block"] = codes, blocks
        elif kind == "e4m3":
            st[x + "_cache"] = randn(*shape, dtype=torch.bfloat16).mul_(32).to(TYPES[kind])
            st[x + "_scale"] = (0.5 + torch.rand(kvh, device=dev, generator=gen)) / 32
        else:
            st[x + "_cache"] = randn(*shape, dtype=TYPES[kind])
    if op == "append":
        # k and v as a fused projection leaves them: slices of one row
        kv = randn(R, 2 * kvh, hd).to(TYPES[case["dtype"]])
        st["k"], st["v"] = kv.split((kvh, kvh), 1)
        return st
    if op == "evict":
        # a few heavy keys and many light ones, some of them equally heavy
        w = torch.exp(2 * randn(n, kvh, width * page))
        st["weights"] = torch.where(w < 0.25, torch.ceil(w * 64) / 64, w)
        st["weights_out"] = torch.zeros_like(st["weights"])
        st["kept"] = torch.zeros(n, kvh, case["keep"], dtype=torch.int32, device=dev)
        return st
    st["q"] = randn(R, case["heads"], hd).to(TYPES[case["dtype"]])
    if op == "weights":
        # what earlier passes have left, and the statistics that this pass's attention gave
        st["weights"] = torch.rand(n, kvh, width * page, device=dev, generator=gen)
        s, seq, i = _scores(st)
        st["lse"] = _rows_back(case, torch.logsumexp(s.double(), -1, keepdim=True).float(), seq, i).squeeze(-1).contiguous()
    return st


# ------------------------------------------------------------------ one pass
def run(state):
    return {"append": _run_append, "attention": _run_attention, "weights": _run_weights,
            "evict": _run_evict}[state["case"]["op"]](state)


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


def _gathered(st, x):
    """Every sequence's keys or values, padded, in f32: [n][positions][kv_heads][head_dim]."""
    held = st["table"].clamp(min=0).long()
    cache, block, scale = st[x + "_cache"], st[x + "_block"], st[x + "_scale"]
    if block is not None:
        b = block.view(torch.uint8)[held].view(block.dtype)
        return _e2m1_values(cache[held], b, scale).flatten(1, 2)
    if scale is not None:
        return cache.view(torch.uint8)[held].view(cache.dtype).flatten(1, 2).float() * scale[:, None]
    return cache[held].flatten(1, 2).float()


def _scores(st):
    """Scaled scores of all rows, -inf out of view: [n][kv_heads][rows x group][positions], and the rows' places."""
    case, q = st["case"], st["q"]
    n, kvh, hd, rows = case["n"], case["kv_heads"], case["head_dim"], case["rows"]
    g = case["heads"] // kvh
    seq, i, pos = _positions(st, q.shape[0])
    qs = torch.zeros(n, rows, case["heads"], hd, device=q.device)
    qs[seq, i] = q.float()
    at = torch.full((n, rows), -1, device=q.device, dtype=torch.int64)
    at[seq, i] = pos
    qs = qs.view(n, rows, kvh, g, hd).permute(0, 2, 1, 3, 4).reshape(n, kvh, rows * g, hd)
    s = torch.matmul(qs, _gathered(st, "k").permute(0, 2, 3, 1)) / math.sqrt(hd)
    key = torch.arange(s.shape[-1], device=q.device)
    seen = key <= at[..., None]
    if case["window"]:
        seen &= key > at[..., None] - case["window"]
    s.masked_fill_(~seen[:, None, :, None].expand(n, 1, rows, g, -1).reshape(n, 1, rows * g, -1), -math.inf)
    return s, seq, i


def _rows_back(case, x, seq, i):
    """[n][kv_heads][rows x group][c] as the call's rows: [R][heads][c]."""
    kvh = case["kv_heads"]
    return x.view(case["n"], kvh, case["rows"], case["heads"] // kvh, -1).permute(0, 2, 1, 3, 4).flatten(2, 3)[seq, i]


def _run_append(st):
    case, R = st["case"], st["k"].shape[0]
    if own:
        import block_speculative_drafting_gb300 as dfl
        held = dict(row_start=st["row_start"], k_scale=st["k_scale"], v_scale=st["v_scale"], k_block=st["k_block"],
                    v_block=st["v_block"])
        dfl.paged_append(st["k_cache"], st["v_cache"], st["k"], st["v"], st["table"], st["kv_len"], **held)
        k, v = dfl.paged_read(st["k_cache"], st["v_cache"], st["table"], st["kv_len"], R, dtype=torch.bfloat16, **held)
        return [k, v, st["k_block"], st["v_block"]]
    seq, _, pos = _positions(st, R)
    page, slot = st["table"][seq, pos // case["page"]].long(), pos % case["page"]
    back = []
    for x in "kv":
        scale, block = st[x + "_scale"], st[x + "_block"].view(torch.uint8)
        codes, s = _e2m1_blocks(st[x].float() / scale[:, None])
        st[x + "_cache"][page, slot] = codes
        block[page, slot] = s.view(torch.uint8)
        back.append(_e2m1_values(st[x + "_cache"][page, slot], block[page, slot].view(s.dtype), scale).bfloat16())
    return back + [st["k_block"], st["v_block"]]


def _run_attention(st):
    case, q = st["case"], st["q"]
    if own:
        import block_speculative_drafting_gb300 as dfl
        lse = torch.empty(q.shape[:2], dtype=torch.float32, device=q.device) if case["lse"] else None
        out = dfl.paged_attention(q, st["k_cache"], st["v_cache"], st["table"], st["kv_len"],
                                  row_start=st["row_start"], window=case["window"], k_scale=st["k_scale"],
                                  v_scale=st["v_scale"], k_block=st["k_block"], v_block=st["v_block"], lse=lse)
        return [out, lse] if case["lse"] else [out]
    s, seq, i = _scores(st)
    m = s.amax(-1, keepdim=True).clamp(min=-1e30)
    p = torch.exp(s - m)
    total = p.sum(-1, keepdim=True)
    y = torch.matmul(p / total.clamp(min=1e-30), _gathered(st, "v").transpose(1, 2))
    out = _rows_back(case, y, seq, i).to(q.dtype)
    return [out, _rows_back(case, m + torch.log(total), seq, i).squeeze(-1)] if case["lse"] else [out]


def _run_weights(st):
    case, W = st["case"], st["weights"]
    if own:
        import block_speculative_drafting_gb300 as dfl
        return [dfl.paged_key_weights(W, st["q"], st["k_cache"], st["table"], st["kv_len"], st["lse"],
                                      row_start=st["row_start"], window=case["window"], k_scale=st["k_scale"],
                                      k_block=st["k_block"])]
    n, kvh = case["n"], case["kv_heads"]
    s, seq, i = _scores(st)
    lse = torch.zeros(n, case["rows"], case["heads"], device=W.device)
    lse[seq, i] = st["lse"]
    lse = lse.view(n, case["rows"], kvh, -1).transpose(1, 2).reshape(n, kvh, -1, 1)
    got = torch.exp(s.sub_(lse)).sum(2)
    # a position that the call itself brings starts at nothing; positions past the last are left as they are
    key = torch.arange(W.shape[-1], device=W.device)
    count = torch.zeros_like(st["kv_len"]).index_add_(0, seq, torch.ones_like(seq, dtype=torch.int32))
    old = key < (st["kv_len"] - count)[:, None]
    held = key < st["kv_len"][:, None]
    W.copy_(torch.where(old[:, None], W + got, torch.where(held[:, None], got, W)))
    return [W]


def _run_evict(st):
    case, W, out = st["case"], st["weights"], st["weights_out"]
    keep, n, kvh = case["keep"], case["n"], case["kv_heads"]
    if own:
        import block_speculative_drafting_gb300 as dfl
        new_len = dfl.paged_evict(st["k_cache"], st["v_cache"], W, st["table"], st["kv_len"], keep, first=case["first"],
                                  recent=case["recent"], k_block=st["k_block"], v_block=st["v_block"], weights_out=out,
                                  kept=st["kept"])
        if case["cache"] != "e2m1":
            return [st["k_cache"], st["v_cache"], out, new_len, st["kept"]]
        start = torch.arange(n + 1, device=out.device, dtype=torch.int32) * keep
        k, v = dfl.paged_read(st["k_cache"], st["v_cache"], st["table"], torch.full_like(new_len, keep), n * keep,
                              row_start=start, k_scale=st["k_scale"], v_scale=st["v_scale"], k_block=st["k_block"],
                              v_block=st["v_block"], dtype=torch.bfloat16)
        return [k, v, out, new_len, st["kept"]]
    L = st["kv_len"].long()[:, None]
    slot = torch.arange(W.shape[-1], device=W.device)
    over = L > keep
    always = (slot < case["first"]) | (slot >= L - case["recent"])
    w = torch.where(always[:, None], math.inf, W)
    w = torch.where((slot < L)[:, None], w, -math.inf)
    best = torch.sort(w, dim=-1, descending=True, stable=True).indices[..., :keep].sort(-1).values
    at = torch.arange(best.shape[-1], device=W.device)
    src = torch.where(over[:, None], best, at.expand_as(best))  # [n][kv_heads][keep]
    live = (at < L)[:, None].expand_as(src)
    head = torch.arange(kvh, device=W.device)[:, None]
    seq = torch.arange(n, device=W.device)[:, None, None]

    def place(x):
        return st["table"][seq, x // case["page"]].clamp(min=0).long(), x % case["page"], head

    src = torch.where(live, src, at)
    dst = at.expand_as(src)
    for x in ("k_cache", "v_cache", "k_block", "v_block"):
        if st[x] is not None:
            c = st[x].view(torch.uint8) if st[x].element_size() == 1 else st[x]
            c[tuple(y[live] for y in torch.broadcast_tensors(*place(dst)))] = \
                c[tuple(y[live] for y in torch.broadcast_tensors(*place(src)))]
    k_len = best.shape[-1]
    out[..., :k_len] = torch.where(live, torch.gather(W, -1, src), out[..., :k_len])
    st["kept"].fill_(-1)
    st["kept"][..., :k_len] = torch.where(live, src, -1).to(torch.int32)
    new_len = torch.minimum(L[:, 0], torch.full_like(L[:, 0], keep)).to(torch.int32)
    if case["cache"] != "e2m1":
        return [st["k_cache"], st["v_cache"], out, new_len, st["kept"]]
    # the slots that the budget names, as values (0 where the table holds no page)
    s = torch.arange(keep, device=W.device)
    page = torch.full((n, keep), -1, device=W.device, dtype=torch.int64)
    width = min(keep, st["table"].shape[1] * case["page"])
    page[:, :width] = st["table"][:, s[:width] // case["page"]].long()
    back = []
    for x in "kv":
        c, b = st[x + "_cache"][page.clamp(min=0), s % case["page"]], st[x + "_block"].view(torch.uint8)[page.clamp(min=0), s % case["page"]]
        y = _e2m1_values(c, b.view(torch.float8_e4m3fn), st[x + "_scale"])
        back.append(torch.where((page >= 0)[..., None, None], y, 0.0).flatten(0, 1).bfloat16())
    return back + [out, new_len, st["kept"]]


# ------------------------------------------------------------------ the definition in 64 bits
def _round_to(x, bits, least):
    """x rounded to `bits` significant bits, not finer than `least` (ties to even)."""
    e = torch.floor(torch.log2(x.abs().clamp(min=1e-300)))
    e = torch.where(torch.exp2(e) > x.abs(), e - 1, e)
    step = torch.exp2(e - (bits - 1)).clamp(min=least)
    return torch.round(x / step) * step


def _value64(st, x, pages, slots=None):
    """Rows of a cache in 64 bits."""
    c, b, sc = st[x + "_cache"], st[x + "_block"], st[x + "_scale"]
    at = (lambda y: y[pages]) if slots is None else (lambda y: y[pages, slots])
    if b is None:
        y = at(c.view(torch.uint8)).view(c.dtype).double() if c.element_size() == 1 else at(c).double()
        return y * sc.double()[:, None] if sc is not None else y
    code = at(c).long()
    code = torch.stack((code % 16, code // 16), -1).flatten(-2)
    m = code % 8
    mag = torch.where(m < 2, m * 0.5, (1 + (m % 2) * 0.5) * torch.exp2((m // 2 - 1).double()))
    y = torch.where(code >= 8, -mag, mag) * at(b.view(torch.uint8)).view(b.dtype).double().repeat_interleave(16, -1)
    return y * sc.double()[:, None]


def exact(case, seed):
    """The definition, one sequence at a time, in 64 bits."""
    st = prepare(case, seed)
    rows, lens = _rows_of(case), _lens_of(case)
    at, page, table = _starts(rows), case["page"], st["table"].tolist()
    if case["op"] == "append":
        return _exact_append(case, st, rows, lens, table)
    if case["op"] == "evict":
        return _exact_evict(case, st, lens, table)
    kvh, g, hd = case["kv_heads"], case["heads"] // case["kv_heads"], case["head_dim"]
    if case["op"] == "weights" and sum(rows) * max(lens) * case["heads"] > 3e9:
        return None
    out, lses = [], []
    W = st["weights"].double() if case["op"] == "weights" else None
    for s in range(case["n"]):
        L, r = lens[s], rows[s]
        pages = torch.tensor(table[s][:-(-L // page)], device="cuda")
        k = _value64(st, "k", pages).reshape(-1, kvh, hd)[:L]
        q = st["q"][at[s]:at[s + 1]].double().view(r, kvh, g, hd)
        sc = torch.einsum("rkgd,lkd->kgrl", q, k) * hd ** -0.5
        pos = torch.arange(L - r, L, device="cuda")[:, None]
        key = torch.arange(L, device="cuda")[None]
        hide = key > pos
        if case["window"]:
            hide = hide | (key <= pos - case["window"])
        sc = sc.masked_fill(hide, -math.inf)
        if case["op"] == "weights":
            lse = st["lse"][at[s]:at[s + 1]].double().view(r, kvh, g).permute(1, 2, 0)
            W[s, :, L - r:L] = 0
            W[s, :, :L] += torch.exp(sc - lse[..., None]).sum((1, 2))
            continue
        v = _value64(st, "v", pages).reshape(-1, kvh, hd)[:L]
        lse = torch.logsumexp(sc, -1)
        out.append(torch.einsum("kgrl,lkd->rkgd", torch.exp(sc - lse[..., None]), v).reshape(r, kvh * g, hd))
        lses.append(lse.permute(2, 0, 1).reshape(r, kvh * g))
    if case["op"] == "weights":
        return [W]
    return [torch.cat(out), torch.cat(lses)] if case["lse"] else [torch.cat(out)]


def _exact_append(case, st, rows, lens, table):
    page = case["page"]
    slots = [(table[s][p // page], p % page) for s in range(case["n"]) for p in range(lens[s] - rows[s], lens[s])]
    pg, sl = (torch.tensor(x, device="cuda") for x in zip(*slots))
    back, blocks = [], []
    for x in "kv":
        t = (st[x].double() / st[x + "_scale"].double()[:, None]).unflatten(-1, (-1, 16))
        s = _round_to(torch.clamp(t.abs().amax(-1) / 6, max=448), 4, 2.0 ** -9)
        u = torch.where(s[..., None] > 0, t / s[..., None], 0.0)
        y = _round_to(u, 2, 0.5).clamp(-6, 6)
        back.append((y * s[..., None]).flatten(-2) * st[x + "_scale"].double()[:, None])
        b = st[x + "_block"].double()
        b[pg, sl] = s
        blocks.append(b)
    return back + blocks


def _exact_evict(case, st, lens, table):
    keep, page = case["keep"], case["page"]
    n, kvh = case["n"], case["kv_heads"]
    out, kept = st["weights_out"].double(), torch.full((n, kvh, keep), -1, dtype=torch.int32)
    flat = {x: _value64(st, x, slice(None)) if case["cache"] == "e2m1" else st[x + "_cache"].double() for x in "kv"}
    back = {x: torch.zeros(n, keep, kvh, case["head_dim"], dtype=torch.float64, device="cuda") for x in "kv"}
    new_len = []
    for s in range(n):
        L = lens[s]
        slot = np.arange(L)
        w = st["weights"][s, :, :L].cpu().numpy()
        pages = np.array(table[s])[slot // page]
        new_len.append(min(L, keep))
        took = np.tile(slot, (kvh, 1))
        if L > keep:
            must = (slot < case["first"]) | (slot >= L - case["recent"])
            for h in range(kvh):
                order = np.lexsort((slot, -w[h].astype(np.float64), ~must))
                took[h, :keep] = np.sort(order[:keep])
            took = took[:, :keep]
        m = took.shape[1]
        kept[s, :, :m] = torch.from_numpy(took).to(torch.int32)
        src = torch.from_numpy(took).cuda()
        out[s, :, :m] = torch.gather(st["weights"][s].double(), 1, src)
        h = torch.arange(kvh, device="cuda")[:, None]
        pg, sl = torch.from_numpy(pages).cuda().long(), torch.from_numpy(slot % page).cuda()
        for x in "kv":
            moved = flat[x][pg[src], sl[src], h]
            flat[x][pg[None, :m].expand(kvh, m), sl[None, :m].expand(kvh, m), h] = moved
            if case["cache"] == "e2m1":
                width = min(keep, len(table[s]) * page)
                every = np.arange(width)
                ids = np.array(table[s])[every // page]
                y = flat[x][torch.from_numpy(np.maximum(ids, 0)).cuda().long(), torch.from_numpy(every % page).cuda()]
                back[x][s, :width] = torch.where(torch.from_numpy(ids >= 0).cuda()[:, None, None], y, 0.0)
    head = [back["k"].flatten(0, 1), back["v"].flatten(0, 1)] if case["cache"] == "e2m1" else [flat["k"], flat["v"]]
    return head + [out, torch.tensor(new_len, dtype=torch.int32), kept]
