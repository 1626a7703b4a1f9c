"""Further cases of the target's verification pass: each test holds one behaviour that went wrong before, against
oracle/target.py or a plain 64-bit computation."""
import numpy as np
import pytest

from oracle import target as O
from test_paged_index import walk  # noqa: F401  (a fixture: the kernels' walk from rows to pages, on the host)

gpu = pytest.mark.gpu


def _dfl():
    import block_speculative_drafting_gb300 as dfl
    return dfl


def _torch():
    return pytest.importorskip("torch")


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def _i32(torch, x):
    return torch.tensor(np.asarray(x, np.int32), device="cuda")


# --------------------------------------------------------------------------- starts out of order
BAD_STARTS = [[0, 5, 3, 8], [6, 0, 6, 2], [0, 99, 99, 99], [-5, 2, 4, 99], [3, 1, 2, 5], [8, 8, 0, 8], [0, 8, 8, 1],
              [2, -2 ** 31, 2 ** 31 - 1, 3]]


def test_rows_of_starts_out_of_order_have_one_owner(walk):  # noqa: F811
    """Every row has the sequence that the oracle's ascending starts give it, or none."""
    text = ""
    for start in BAD_STARTS:
        text += f"3 8 1 16 4 0\n{' '.join(map(str, start))}\n9 9 9\n0 1 2\n"
    lines = iter(walk(text + "-1 0 0 0 0 0\n"))
    for start in BAD_STARTS:
        owner = {r: s for s, a, n in O.rows_of(3, 8, start) for r in range(a, a + n)}
        for r in range(8):
            assert int(next(lines).split()[0]) == owner.get(r, -1), (start, r)
        assert next(lines) == "end"


@gpu
@pytest.mark.parametrize("start", BAD_STARTS)
@pytest.mark.parametrize("heads", [4, 40])  # the warps' kernel, and the tensor memory's
def test_paged_calls_with_starts_out_of_order(start, heads):
    torch, dfl = _torch(), _dfl()
    rng = np.random.default_rng(0)
    R = lambda *s: torch.from_numpy(rng.standard_normal(s).astype(np.float32)).cuda().to(torch.bfloat16)  # noqa: E731
    kc, vc, q, k, v = R(6, 16, 2, 64), R(6, 16, 2, 64), R(8, heads, 64), R(8, 2, 64), R(8, 2, 64)
    table, lens = [[0, 1], [2, 3], [4, 5]], [20, 31, 9]
    args = (_i32(torch, table), _i32(torch, lens))
    k64, v64 = f64(kc), f64(vc)
    q_out = torch.full_like(q, 7.0)
    dfl.paged_append(kc, vc, k, v, *args, row_start=_i32(torch, start), q=q, q_out=q_out)
    slots, _, touched = O.paged_append(f64(k), f64(v), f64(q), table, lens, 16, 6, start)
    for at, (kk, vv) in slots.items():
        k64[at], v64[at] = kk, vv
    assert np.array_equal(f64(kc), k64) and np.array_equal(f64(vc), v64)
    rest = [r for r in range(8) if r not in touched]
    assert np.array_equal(f64(q_out)[touched], f64(q)[touched]) and (f64(q_out)[rest] == 7.0).all()
    ref, _, mag, touched = O.paged_attention(f64(q), k64, v64, table, lens, start)
    out = torch.full_like(q, 7.0)
    dfl.paged_attention(q, kc, vc, *args, row_start=_i32(torch, start), out=out)
    # bf16 outputs: half a step; scores: 64 f32 products of up to |q| |k| = 100, times the scale
    assert (np.abs(f64(out) - ref) <= 2.0 ** -8 * np.abs(ref) + 64 * 2.0 ** -24 * 100 * mag)[touched].all()
    assert (f64(out)[[r for r in range(8) if r not in touched]] == 7.0).all()


@gpu
@pytest.mark.parametrize("start", BAD_STARTS)
@pytest.mark.parametrize("drawn", [False, True])
def test_verify_with_starts_out_of_order(start, drawn):
    """What the oracle's ascending starts give, whatever the workspace held before: every output, and nothing else."""
    torch, dfl = _torch(), _dfl()
    for seed, temps in enumerate(([0.0, 0.0, 0.0], [0.9, 0.0, 1.4], [0.7, 1.0, 0.8])):
        rng = np.random.default_rng(seed)
        n, d, V = 3, 8, 100
        t = torch.from_numpy(rng.standard_normal((n + d, V)).astype(np.float32)).cuda()
        dl = torch.from_numpy(rng.standard_normal((d, V)).astype(np.float32)).cuda()
        tok = rng.integers(0, V, d)
        au, su = (torch.from_numpy(rng.random(m).astype(np.float32)).cuda() for m in (d, n))
        res, pref = O.verify(f64(t), tok, f64(au), f64(su), f64(dl) if drawn else None, start, temps)
        at = O.rows_of(n, d, start)
        owned = [j for _, a, m in at for j in range(a, a + m)]
        need = dfl.verify_workspace(n, d, V)
        for fill in (0x00, 0x7f, 0xff, 0x41):
            ws = torch.full((need,), fill, dtype=torch.uint8, device="cuda")
            prob = torch.full((d,), 7.0, device="cuda")
            acc, nxt, _ = dfl.verify_drafts(t, _i32(torch, tok), au, su, draft_logits=dl if drawn else None,
                                            draft_start=_i32(torch, start), prob=prob, workspace=ws,
                                            temperature=torch.tensor(temps, device="cuda"))
            for s, (a, x, margin) in enumerate(res):
                if margin > 1e-5:
                    assert (acc[s].item(), nxt[s].item()) == (a, x), (start, s, fill)
                assert -1 <= nxt[s].item() < V and 0 <= acc[s].item() <= at[s][2]
            p = f64(prob)
            assert (np.abs(p[owned] - pref[owned]) <= 2e-6 * np.abs(pref[owned])).all()
            assert all(p[j] == 7.0 for j in range(d) if j not in owned)


# --------------------------------------------------------------------------- verification
@gpu
def test_verify_of_many_short_sequences_in_clusters_that_start_late():
    """Thousands of clusters with next to nothing to read, behind work on another stream that keeps the SMs: a cluster's
    CTAs then start at different times, and none may be written to before it runs."""
    torch, dfl = _torch(), _dfl()
    rng = np.random.default_rng(0)
    n, V = 3000, 40
    t = torch.from_numpy(rng.standard_normal((n, V)).astype(np.float32)).cuda()
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    su = torch.from_numpy(rng.random(n).astype(np.float32)).cuda()
    temps = torch.from_numpy(np.where(np.arange(n) % 3 == 0, 0.0, 0.9).astype(np.float32)).cuda()  # greedy ones between
    res, _ = O.verify(f64(t), [], [], f64(su), None, None, temps.tolist())
    side, busy = torch.cuda.Stream(), torch.randn(2048, 2048, device="cuda")
    for _ in range(5):
        with torch.cuda.stream(side):
            for _ in range(4):
                busy = busy @ busy * 1e-3
        acc, nxt, _ = dfl.verify_drafts(t, none, torch.empty(0, device="cuda"), su, temperature=temps)
        got = nxt.tolist()
        assert acc.tolist() == [0] * n
        assert all(g == x for g, (_, x, margin) in zip(got, res) if margin > 1e-5)
        torch.cuda.synchronize()


def _define(torch, target, tok, au, su, draft=None, T=1.0):
    """One draft a sequence (none: tok None), verified by the definition in 64 bits: (kept, token, how far the numbers are
    from where the answer changes, relative to what is compared, what is left in all)."""
    soft = lambda x: torch.softmax(x.double() / T, -1)  # noqa: E731
    n = su.shape[0]
    rows = target.view(n, -1, target.shape[-1])
    kept = torch.ones(n, dtype=torch.bool, device="cuda")
    near = torch.full((n,), np.inf, dtype=torch.float64, device="cuda")
    rest = soft(rows[:, -1])
    if tok is not None:
        p, i = soft(rows[:, 0]), torch.arange(n, device="cuda")
        q = torch.zeros_like(p).scatter_(1, tok.long()[:, None], 1.0) if draft is None else soft(draft)
        px, uq = p[i, tok.long()], au.double() * q[i, tok.long()]
        kept, near = uq < px, (uq - px).abs() / torch.maximum(uq, px)
        rest = torch.where(kept[:, None], rest, (p - q).clamp(min=0))
    c = torch.cumsum(rest, -1)
    whole = c[:, -1:]
    want = su.double()[:, None] * whole
    token = (c <= want).sum(-1)
    near = torch.minimum(near, ((c - want).abs().amin(-1)) / whole[:, 0])
    return kept, token, near, whole[:, 0]


def _compare(torch, got, want):
    """(accepted, token) against _define's, wherever 64 bits decide: p and q there are off by their exponentials' and
    divisions' few 2^-53 and the exponents' 2^-53 of up to 40, 4e-15 in all, of what is left."""
    kept, token, near, whole = want
    sure = near > torch.maximum(4e-15 / whole, torch.full_like(whole, 1e-12))
    acc, nxt = got[0].bool(), got[1].long()
    assert torch.equal(acc[sure], kept[sure]) and torch.equal(nxt[sure], token[sure])
    return int(sure.sum())


@gpu
@pytest.mark.parametrize("kind", ["float32", "bfloat16"])
@pytest.mark.parametrize("noise", [0.7, 0.1, 0.01, 0.001, None])
def test_verify_draws_the_definitions_token(kind, noise):
    """Hundreds of refused drafts over a whole vocabulary, of drafters from far to very near the target (what is left to
    draw from is the refused mass, 0.3 down to 0.0003), and drafts that were chosen: every token is the definition's."""
    torch, dfl = _torch(), _dfl()
    n, V, T, sure, total, left = 256, 151936, float(np.float32(0.8)), 0, 0, []
    for seed in range(2):
        g = torch.Generator("cuda").manual_seed(seed)
        t = (2.5 * torch.randn(2 * n, V, device="cuda", generator=g)).to(getattr(torch, kind))
        first = t[0::2].float()
        d = None if noise is None else first + noise * torch.randn(n, V, device="cuda", generator=g)
        # a draft that the drafter likes better than the target does (chosen: a likely one), refused by a large number
        tok = (first if d is None else d.softmax(-1) - first.softmax(-1)).argmax(-1).int()
        au = torch.full((n,), 1 - 2.0 ** -24, device="cuda")
        su = torch.rand(n, device="cuda", generator=g)
        got = dfl.verify_drafts(t, tok, au, su, draft_logits=d, temperature=torch.full((n,), T, device="cuda"))
        want = _define(torch, t, tok, au, su, d, T)
        sure, total, left = sure + _compare(torch, got, want), total + n, left + want[3].tolist()
        assert not want[0].any()
    assert sure > 0.99 * total
    if noise is not None:
        assert 0.1 * noise < np.median(left) < noise


def _at_borders(torch, rest, least):
    """For every row a number in [0, 1) of 32 bits right at a border of the row's running sums: as near as it can be and
    still more than `least` of the whole away."""
    c = torch.cumsum(rest, -1)
    whole = c[:, -1:]
    share = c / whole
    u = share.float()
    away = ((u.double() * whole - c).abs() / whole).masked_fill((u >= 1) | (u <= 0), np.inf)
    away = away.masked_fill(away < least, np.inf)
    return u.gather(1, away.argmin(-1, keepdim=True))[:, 0]


@gpu
@pytest.mark.parametrize("kind", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("V", [1000, 151936, 700001])
@pytest.mark.parametrize("drawn", [None, False, True])
def test_verify_draws_at_the_borders(kind, V, drawn):
    """Numbers within 1e-9 to 1e-12 of a border of the running sums, where sums of 32-bit weights do not decide."""
    torch, dfl = _torch(), _dfl()
    T = float(np.float32(0.9))
    for n, seed in ((3, 0), (30, 1)):
        g = torch.Generator("cuda").manual_seed(seed)
        t = (2 * torch.randn(n * (1 if drawn is None else 2), V, device="cuda", generator=g)).to(getattr(torch, kind))
        su, au = torch.zeros(n, device="cuda"), torch.full((n,), 1 - 2.0 ** -24, device="cuda")
        temps = torch.full((n,), T, device="cuda")
        soft = lambda x: torch.softmax(x.double() / T, -1)  # noqa: E731
        d = tok = None
        if drawn is None:
            rest = soft(t)
            tok_in, au_in = torch.empty(0, dtype=torch.int32, device="cuda"), torch.empty(0, device="cuda")
        else:
            first = t[0::2].float()
            if drawn:
                d = first + 0.3 * torch.randn(n, V, device="cuda", generator=g)
                q = soft(d)
                tok = (q - soft(first)).argmax(-1).int()
            else:
                tok = first.argmax(-1).int()
                q = torch.zeros(n, V, dtype=torch.float64, device="cuda").scatter_(1, tok.long()[:, None], 1.0)
            rest = (soft(first) - q).clamp(min=0)
            tok_in, au_in = tok, au
        su = _at_borders(torch, rest, 2e-12)
        got = dfl.verify_drafts(t, tok_in, au_in, su, draft_logits=d, temperature=temps)
        want = _define(torch, t, tok, au, su, d, T)
        acc = (torch.ones(n, device="cuda") if drawn is None else got[0], got[1])
        assert _compare(torch, acc, want) == n


@gpu
@pytest.mark.parametrize("drawn", [False, True])
def test_verify_decides_drafts_at_the_border(drawn):
    """Numbers within 1e-8 to 1e-12 of p / q: kept or refused as 64 bits say."""
    torch, dfl = _torch(), _dfl()
    n, V, T = 64, 50000, float(np.float32(0.7))
    g = torch.Generator("cuda").manual_seed(0)
    t = 2 * torch.randn(2 * n, V, device="cuda", generator=g)
    first = t[0::2]
    d = first + 0.5 * torch.randn(n, V, device="cuda", generator=g) if drawn else None
    p = torch.softmax(first.double() / T, -1)
    q = torch.softmax(d.double() / T, -1) if drawn else torch.ones_like(p)
    ratio = p / q
    u = ratio.float()
    away = ((u.double() - ratio).abs() / ratio).masked_fill((u >= 1) | (u < 1e-6), np.inf)
    away = away.masked_fill(away < 1e-12, np.inf)
    tok = away.argmin(-1).int()
    au = u.gather(1, tok.long()[:, None])[:, 0]
    assert away.amin(-1).max() < 2e-8
    got = dfl.verify_drafts(t, tok, au, torch.rand(n, device="cuda", generator=g), draft_logits=d,
                            temperature=torch.full((n,), T, device="cuda"))
    want = _define(torch, t, tok, au, torch.rand(n, device="cuda", generator=g), d, T)
    assert torch.equal(got[0].bool(), want[0]) and 0 < got[0].sum() < n
    # probabilities: 32-bit sums of exponentials, within 2^-20
    px = (p / q).gather(1, tok.long()[:, None])[:, 0].clamp(max=1)
    assert ((got[2].double() - px).abs() <= 2.0 ** -20 * px).all()


@gpu
def test_verify_of_the_smallest_numbers_and_sharp_temperatures():
    torch, dfl = _torch(), _dfl()
    inf = float("inf")
    none, empty = torch.empty(0, dtype=torch.int32, device="cuda"), torch.empty(0, device="cuda")
    # a number of 0 takes the first entry with any probability in 64 bits: masked and vanishing ones come first
    t = torch.full((4, 3000), -inf, device="cuda")
    t[:, 2000] = 10.0
    t[0, 700], t[1, 700], t[2, 700], t[3, 700] = -500.0, -800.0, 9.0, -30.0
    _, nxt, _ = dfl.verify_drafts(t, none, empty, torch.zeros(4, device="cuda"))
    assert nxt.tolist() == [700, 2000, 700, 700]
    # after a refusal: the first entry that the target likes better, however little of either there is
    t = torch.full((2, 3000), -inf, device="cuda")
    t[:, 5], t[:, 40], t[:, 1000], t[:, 2000] = -59.0, -70.0, 3.0, 2.9
    d = t[:1].clone()
    d[0, 1000], d[0, 5], d[0, 40] = 3.5, -59.0, -75.0
    acc, nxt, _ = dfl.verify_drafts(t, _i32(torch, [1000]), torch.full((1,), 1 - 2.0 ** -24, device="cuda"),
                                    torch.zeros(1, device="cuda"), draft_logits=d)
    p, q = torch.softmax(t[0].double(), -1), torch.softmax(d[0].double(), -1)
    assert acc.tolist() == [0] and nxt.tolist() == [int((p > q).nonzero()[0])]
    # exponents past the 32-bit form's range, and at its end
    g = torch.Generator("cuda").manual_seed(0)
    for T in (1e-2, 3e-3, 1e-3, 1e-5, 1e-9):
        T = float(np.float32(T))
        t = (3 * torch.randn(40, 5000, device="cuda", generator=g)).to(torch.bfloat16)
        t[:, 3000] = t[:, 17] = t.amax(-1)  # (several entries share what there is)
        su = torch.rand(40, device="cuda", generator=g)
        _, nxt, _ = dfl.verify_drafts(t, none, empty, su, temperature=torch.full((40,), T, device="cuda"))
        x = t.double()
        c = torch.cumsum(torch.softmax((x - x.amax(-1, keepdim=True)) / T, -1), -1)
        want = su.double()[:, None] * c[:, -1:]
        sure = (c - want).abs().amin(-1) > 1e-12
        assert torch.equal(nxt.long()[sure], (c <= want).sum(-1)[sure]) and sure.sum() > 35


# --------------------------------------------------------------------------- append
@gpu
@pytest.mark.parametrize("src", ["float32", "bfloat16"])
def test_append_rounds_the_quotient(src):
    """An 8-bit cache's codes are those of the f32 quotient x / scale, rounded once each: values around every step of the
    codes and far beyond, scales over f32's range."""
    torch, dfl = _torch(), _dfl()
    rng = np.random.default_rng(0)
    scales = np.array([1.0, 0.1, 3.0, 1 / 3, 2.0 ** -126, 2.0 ** 126, 3.3e38, 0.07, 1e-10, 448.0, 1e20, 7e-7], np.float32)
    rows, kvh, hd = 64, len(scales), 128
    code = np.frombuffer(np.arange(256, dtype=np.uint8).tobytes(), np.uint8)
    steps = torch.from_numpy(code.copy()).view(torch.float8_e4m3fn).float().numpy()
    steps = np.sort(steps[np.isfinite(steps)])
    mids = np.concatenate((steps, (steps[1:] + steps[:-1]) / 2, [1e4, -1e9, 0.0]))
    x = (rng.choice(mids, (rows, kvh, hd)) * (1 + rng.integers(-2, 3, (rows, kvh, hd)) * 2.0 ** -23)).astype(np.float32)
    with np.errstate(all="ignore"):
        x = (x * scales[:, None]).astype(np.float32)
        x[~np.isfinite(x)] = 3.4e38
        x = torch.from_numpy(x).to(getattr(torch, src))
        want = torch.from_numpy(np.clip(x.float().numpy() / scales[:, None], -448, 448)).to(torch.float8_e4m3fn)
    kc = torch.zeros(rows, 1, kvh, hd, device="cuda").to(torch.float8_e4m3fn)
    vc, sc = kc.clone(), torch.from_numpy(scales).cuda()
    dfl.paged_append(kc, vc, x.cuda(), x.cuda(), torch.arange(rows, device="cuda", dtype=torch.int32)[None],
                     _i32(torch, [rows]), k_scale=sc, v_scale=sc)
    for c in (kc, vc):
        assert torch.equal(c.view(torch.uint8)[:, 0].cpu(), want.view(torch.uint8))


# --------------------------------------------------------------------------- attention
def _odd_values(torch, kc, vc, table):
    """Values that are not finite at keys that every row sees, early in each sequence: +inf; both signs in one column and
    in two; NaN beside an infinity; an infinity at a key that is not finite itself (the score is -inf for half of the rows,
    +inf for the others); most of a row; and sequences without any."""
    inf, page = float("inf"), kc.shape[1]
    for s in range(len(table)):
        at = lambda p: (int(table[s][p // page]), p % page)  # noqa: E731
        (p0, s0), (p1, s1) = at(3), at(40)
        h = s % kc.shape[2]
        kind = s % 7
        if kind == 1:
            vc[p0, s0, h, 1] = inf
        elif kind == 2:
            vc[p0, s0, h, 2], vc[p1, s1, h, 2], vc[p1, s1, h, 9], vc[p0, s0, h, 33] = inf, -inf, -inf, inf
        elif kind == 3:
            vc[p0, s0, h, 4], vc[p1, s1, h, 4], vc[p0, s0, h, 5] = float("nan"), inf, -inf
        elif kind == 4:
            vc[p1, s1, h, 6], vc[p0, s0, h, 7], kc[p1, s1, h, 5] = inf, -inf, inf
        elif kind == 5:
            vc[p0, s0, h, ::2] = -inf
        elif kind == 6:
            vc[p1, s1, h, 60:] = inf


@gpu
@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("rows,heads,kvh", [(1, 2, 2), (3, 4, 1), (10, 8, 2), (16, 16, 2)])  # 1, 12, 40, 128 rows a unit
@pytest.mark.parametrize("n,lens,window", [(7, 2000, 0), (7, 700, 690), (80, 200, 0)])  # units split over SMs, and whole ones
def test_attention_of_values_that_are_not_finite(kind, hd, rows, heads, kvh, n, lens, window):
    from test_target_ops import _check_attention
    _check_attention(kind, hd=hd, heads=heads, kvh=kvh, rows=(rows,) * n, lens=tuple(lens + 5 * i for i in range(n)),
                     window=window, poison=_odd_values, seed=rows)


@gpu
@pytest.mark.parametrize("rows,heads", [(1, 2), (12, 8)])
def test_attention_of_an_infinity_before_the_reference_moves(rows, heads):
    """An infinite value whose weight vanishes against a later key's is infinite all the same; what overflows stays NaN or
    infinite, and other rows, heads and columns keep their bits."""
    torch, dfl = _torch(), _dfl()
    rng = np.random.default_rng(0)
    kc = torch.from_numpy(rng.standard_normal((64, 16, 1, 64)).astype(np.float32)).cuda().to(torch.bfloat16)
    vc = torch.from_numpy(rng.standard_normal((64, 16, 1, 64)).astype(np.float32)).cuda().to(torch.bfloat16)
    q = torch.from_numpy(rng.standard_normal((rows, heads, 64)).astype(np.float32)).cuda().to(torch.bfloat16)
    q[..., 0] = 8.0
    kc[60, 0, 0, 0] = 256.0  # the score there is 256 above the others': 369 in powers of two
    args = (_i32(torch, np.arange(64)[None]), _i32(torch, [1024]))
    want = dfl.paged_attention(q, kc, vc, *args)
    vc[2, 5, 0, 7] = float("-inf")
    got = dfl.paged_attention(q, kc, vc, *args)
    assert (got[..., 7] == float("-inf")).all()
    got[..., 7] = want[..., 7]
    assert torch.equal(got, want) and torch.isfinite(want).all()


@gpu
@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("rows,heads,kvh", [(5, 8, 2), (16, 8, 2), (16, 16, 2)])  # 20, 64 and 128 rows a unit
@pytest.mark.parametrize("lens", [300, 3000])
def test_attention_of_f16_blocks_over_an_8_bit_cache_rounds_once(hd, rows, heads, kvh, lens):
    """f16 queries over an e4m3 cache: weights add no rounding of their own, however many rows share the keys.  Every key but
    one in 64 weighs 65.03125 / 128 of those, which one f16 takes for 65 or 65.0625, 2^-11 off; all values are 1.875, and
    so is the result, to 2^-18 before its one rounding."""
    torch, dfl = _torch(), _dfl()
    page, n = 16, lens // 16 + 1
    scale = float(np.log(128 / 65.03125))
    q = torch.zeros(rows, heads, hd, device="cuda", dtype=torch.float16)
    q[..., 3] = 1.0
    kc = torch.zeros(n, page, kvh, hd, device="cuda")
    kc[..., 3] = -1.0
    kc[::4, 0, :, 3] = 0.0
    vc = torch.full_like(kc, 1.875)
    kc, vc = kc.to(torch.float8_e4m3fn), vc.to(torch.float8_e4m3fn)
    out = dfl.paged_attention(q, kc, vc, torch.arange(n, device="cuda", dtype=torch.int32)[None], _i32(torch, [lens]),
                              scale=scale)
    assert (out == 1.875).all(), out.float().unique()


@gpu
@pytest.mark.parametrize("kind", ["bf16", "f16"])
def test_attention_of_blocks_keeps_every_tiles_key_mask(kind):
    """Blocks over contexts with a third of their pages not held: each tile's keys have a mask of their own, which the
    loaders write while tiles before it are worked on.  Right once, and the same bits in every repetition."""
    torch, dfl = _torch(), _dfl()
    from test_target_ops import _check_attention, _types
    bad = tuple((s, i) for s in range(3) for i in range((s + 1) % 3, 60, 3))
    _check_attention(kind, heads=8, kvh=2, rows=(9, 16, 5), lens=(950, 970, 955), bad=bad, seed=7)
    rng = np.random.default_rng(3)
    n, pages, width = 24, 2000, 80
    table = rng.integers(0, pages, (n, width)).astype(np.int32)
    table[rng.random((n, width)) < 0.33] = -1
    kc, vc = (torch.randn(pages, 16, 2, 128, device="cuda").to(_types()[kind]) for _ in range(2))
    q = torch.randn(n * 16, 8, 128, device="cuda").to(_types()[kind])
    args = (kc, vc, _i32(torch, table), _i32(torch, rng.integers(900, 1280, n)))
    want = dfl.paged_attention(q, *args)
    assert torch.isfinite(want).all()
    for _ in range(50):
        assert torch.equal(dfl.paged_attention(q, *args), want)


# --------------------------------------------------------------------------- the build
def test_binding_is_built_again_for_another_torch(tmp_path, monkeypatch):
    """A torch of another version, or at another place, has the extension compiled again; the same one does not."""
    import importlib.util
    from block_speculative_drafting_gb300.csrc import build as B
    B.build()
    ran = []

    def run(cmd, **kw):
        ran.append(cmd)
        return type("R", (), dict(returncode=0, stdout="", stderr=""))()

    monkeypatch.setattr(B.subprocess, "run", run)
    monkeypatch.setattr(B, "BOUND_FOR", str(tmp_path / "binding.txt"))
    monkeypatch.setattr(B, "_needs", lambda out, deps: False)
    B.build()
    assert len(ran) == 1 and ran[0][-1].startswith("-Wl,-rpath,") and B.BINDING in ran[0]  # not known what it was built for
    B.build()
    assert len(ran) == 1
    old = tmp_path / "torch"
    old.mkdir()
    (old / "__init__.py").write_text("")
    (old / "version.py").write_text("__version__ = '0.0'\n")
    spec = importlib.util.spec_from_file_location("torch", old / "__init__.py")
    monkeypatch.setattr(B.importlib.util, "find_spec", lambda name: spec)
    B.build()
    assert len(ran) == 2
    B.build()
    assert len(ran) == 2
    (old / "version.py").write_text("__version__ = '0.1'\n")
    B.build()
    assert len(ran) == 3


# --------------------------------------------------------------------------- refusals, one change from a call that is served
def _good(torch):
    z = lambda *s, dtype=torch.bfloat16: torch.zeros(*s, dtype=dtype, device="cuda")  # noqa: E731
    i32 = lambda x: _i32(torch, x)  # noqa: E731
    append = dict(k_cache=z(6, 16, 2, 64), v_cache=z(6, 16, 2, 64), k=z(4, 2, 64), v=z(4, 2, 64), table=i32([[0, 1], [2, 3]]),
                  kv_len=i32([20, 30]), row_start=i32([0, 2, 4]), q=z(4, 4, 64), q_out=z(4, 4, 64),
                  inv_freq=z(32, dtype=torch.float64), q_norm=z(64, dtype=torch.float32), k_norm=z(64, dtype=torch.float32))
    attention = dict(q=z(4, 4, 64), k_cache=z(6, 16, 2, 64), v_cache=z(6, 16, 2, 64), table=i32([[0, 1], [2, 3]]),
                     kv_len=i32([20, 30]), row_start=i32([0, 2, 4]), out=z(4, 4, 64), lse=z(4, 4, dtype=torch.float32),
                     workspace=z(1 << 24, dtype=torch.uint8))
    verify = dict(target_logits=z(6, 50), draft_tokens=i32([1, 2, 3, 4]), accept_u=z(4, dtype=torch.float32),
                  sample_u=z(2, dtype=torch.float32), draft_logits=z(4, 50, dtype=torch.float32), draft_start=i32([0, 1, 4]),
                  temperature=z(2, dtype=torch.float32), accepted=i32([0, 0]), next_token=i32([0, 0]),
                  prob=z(4, dtype=torch.float32), workspace=z(1 << 24, dtype=torch.uint8))
    return dict(paged_append=append, paged_attention=attention, verify_drafts=verify)


_SHIFTED = lambda x: x.new_zeros(x.numel() + 1)[1:].view(x.shape)  # noqa: E731  (a base off its alignment)
_WIDE = lambda x: x.new_zeros(*x.shape[:-1], 2 * x.shape[-1])[..., ::2]  # noqa: E731  (columns two apart)
_E4M3 = lambda x: x.new_zeros(x.shape, dtype=__import__("torch").float8_e4m3fn)  # noqa: E731
_SCALES = dict(k_cache=_E4M3, v_cache=_E4M3, k_scale="f2", v_scale="f2")
REFUSALS = [
    # call, changes (None: left out; text: a type, or a float vector's length), message
    ("paged_append", dict(k=lambda x: x.cpu()), "k is not on the call's CUDA device"),
    ("paged_append", dict(table=lambda x: x.cpu()), "table is not on the call's CUDA device"),
    ("paged_append", dict(inv_freq=lambda x: x.cpu()), "inv_freq is not on the call's CUDA device"),
    ("paged_append", dict(k_cache=lambda x: x[None], v_cache=lambda x: x[None]), "k_cache has 5 dimensions"),
    ("paged_append", dict(v_cache=lambda x: x.half()), "of one type"),
    ("paged_append", dict(v_cache=lambda x: x[:, :8]), "differ in shape"),
    ("paged_append", dict(v_cache=lambda x: x[:5]), "differ in shape"),
    ("paged_append", dict(k_cache=_WIDE), "contiguous columns"),
    ("paged_append", dict(v_cache=_WIDE), "contiguous columns"),
    ("paged_append", dict(k_cache=lambda x: x[:1].expand_as(x)), "k_cache is written"),
    ("paged_append", dict(v_cache=lambda x: x[:, :, :1].expand_as(x)), "v_cache is written"),
    ("paged_append", dict(k_cache=_SHIFTED), "16-byte alignment"),
    ("paged_append", dict(k_cache=lambda x: x.new_zeros(6, 16, 2, 65)[..., :64]), "cache strides"),
    ("paged_append", dict(k_cache="double", v_cache="double"), "cache dtype"),
    ("paged_append", dict(k_cache=lambda x: x[..., :32], v_cache=lambda x: x[..., :32], k=lambda x: x[..., :32],
                          v=lambda x: x[..., :32], q=lambda x: x[..., :32], q_out=lambda x: x[..., :32], q_norm=None,
                          k_norm=None, inv_freq=None), "head_dim 32"),
    ("paged_append", dict(k=lambda x: x[:, :1]), "k has 1 heads"),
    ("paged_append", dict(k=lambda x: x[..., :32]), "k has to be"),
    ("paged_append", dict(k=_WIDE), "k has to be"),
    ("paged_append", dict(k=_SHIFTED), "k: base and strides"),
    ("paged_append", dict(v=lambda x: x[:3]), "v has to be"),
    ("paged_append", dict(v="float32"), "one type"),
    ("paged_append", dict(k="double", v="double", q="double"), "k dtype"),
    ("paged_append", dict(table="int64"), "table has to be int32"),
    ("paged_append", dict(table=lambda x: x[0]), "table has to be int32"),
    ("paged_append", dict(table=_WIDE), "table has to be int32"),
    ("paged_append", dict(kv_len="int64"), "kv_len has to be"),
    ("paged_append", dict(kv_len=lambda x: x[:1]), "kv_len has to be"),
    ("paged_append", dict(kv_len=_WIDE), "kv_len has to be"),
    ("paged_append", dict(row_start=lambda x: x[:2]), "row_start has to be"),
    ("paged_append", dict(row_start="int64"), "row_start has to be"),
    ("paged_append", dict(row_start=None, k=lambda x: x[:3], v=lambda x: x[:3], q=lambda x: x[:3], q_out=lambda x: x[:3]),
     "do not divide"),
    ("paged_append", dict(q=None), "q_out without q"),
    ("paged_append", dict(q=lambda x: x[:, :3], q_out=lambda x: x[:, :3]), "q has 3 heads"),
    ("paged_append", dict(q=lambda x: x[:3]), "q has to be"),
    ("paged_append", dict(q_out=lambda x: x[:3]), "q_out has to be"),
    ("paged_append", dict(q_out=lambda x: x[:, :2]), "q_out has 2 heads"),
    ("paged_append", dict(q_out=lambda x: x[:1].expand_as(x)), "q_out is written"),
    ("paged_append", dict(q_out="double"), "q_out dtype"),
    ("paged_append", dict(q_norm=lambda x: x[:32]), "q_norm has to be"),
    ("paged_append", dict(k_norm="bfloat16"), "k_norm has to be"),
    ("paged_append", dict(k_norm=_SHIFTED), "16-byte alignment"),
    ("paged_append", dict(inv_freq="float32"), "inv_freq has to be"),
    ("paged_append", dict(inv_freq=_WIDE), "inv_freq has to be"),
    ("paged_append", dict(inv_freq=lambda x: x[:7]), "rotary 14"),
    ("paged_append", dict(inv_freq=lambda x: x.repeat(2)), "rotary 128"),
    ("paged_append", dict(k_scale="f2", v_scale="f2"), "scales need an E4M3 cache"),
    ("paged_append", {**_SCALES, "v_scale": None}, "come together"),
    ("paged_append", {**_SCALES, "k_scale": "f3"}, "k_scale has to be"),
    ("paged_append", {**_SCALES, "v_scale": lambda x: __import__("torch").zeros(2, device="cuda").double()}, "v_scale has to be"),
    ("paged_attention", dict(q="float16"), "need the cache's type"),
    ("paged_attention", dict(q="float32", out="float32"), "need the cache's type"),
    ("paged_attention", dict(q=_WIDE), "q has to be"),
    ("paged_attention", dict(q=lambda x: x[:, :3], out=lambda x: x[:, :3], lse=lambda x: x[:, :3].contiguous()), "heads 3"),
    ("paged_attention", dict(k_cache=lambda x: x[:, :, :1]), "differ in shape"),
    ("paged_attention", dict(v_cache=lambda x: x.cpu()), "v_cache is not on the call's CUDA device"),
    ("paged_attention", dict(table=lambda x: x.t()), "table has to be int32"),
    ("paged_attention", dict(kv_len=None), "kv_len is None"),
    ("paged_attention", dict(row_start=lambda x: x[:2]), "row_start has to be"),
    ("paged_attention", dict(out=lambda x: x[:3]), "out has to be"),
    ("paged_attention", dict(out=lambda x: x[:, :2]), "out has 2 heads"),
    ("paged_attention", dict(out="float16"), "need the cache's type"),
    ("paged_attention", dict(out=lambda x: x[:, :1].expand_as(x)), "out is written"),
    ("paged_attention", dict(out=_SHIFTED), "out: base and strides"),
    ("paged_attention", dict(lse=lambda x: x[:, :3]), "lse has to be"),
    ("paged_attention", dict(lse=lambda x: x[:3]), "lse has to be"),
    ("paged_attention", dict(lse=lambda x: x.t()), "lse has to be"),
    ("paged_attention", dict(lse="double"), "lse has to be"),
    ("paged_attention", dict(lse=lambda x: x[:1].expand_as(x)), "lse has to be"),
    ("paged_attention", dict(workspace=lambda x: x[:64]), "workspace of 64 bytes"),
    ("paged_attention", dict(workspace=lambda x: x[::2]), "workspace has to be"),
    ("paged_attention", dict(workspace=lambda x: x[8:]), "not 16-byte aligned"),
    ("paged_attention", dict(workspace=lambda x: x.cpu()), "workspace is not on the call's CUDA device"),
    ("paged_attention", dict(window=lambda x: -1), "window -1"),
    ("paged_attention", dict(window=lambda x: 1 << 40), "window"),
    ("paged_attention", dict(scale=lambda x: float("nan")), "scale"),
    ("verify_drafts", dict(target_logits=lambda x: x[:5]), "need 6 target rows, got 5"),
    ("verify_drafts", dict(target_logits=lambda x: x[0]), "target_logits has to be"),
    ("verify_drafts", dict(target_logits=_WIDE), "target_logits has to be"),
    ("verify_drafts", dict(target_logits="double"), "target dtype"),
    ("verify_drafts", dict(target_logits=lambda x: x[:1].expand_as(x)), "row stride"),
    ("verify_drafts", dict(draft_tokens="int64"), "draft_tokens has to be"),
    ("verify_drafts", dict(draft_tokens=_WIDE), "draft_tokens has to be"),
    ("verify_drafts", dict(draft_tokens=lambda x: x.cpu()), "draft_tokens is not on the call's CUDA device"),
    ("verify_drafts", dict(accept_u=None), "accept_u is None"),
    ("verify_drafts", dict(accept_u=lambda x: x[:3]), "accept_u has to be"),
    ("verify_drafts", dict(accept_u="double"), "accept_u has to be"),
    ("verify_drafts", dict(sample_u=lambda x: x[None]), "sample_u has to be"),
    ("verify_drafts", dict(sample_u=_WIDE), "sample_u has to be"),
    ("verify_drafts", dict(draft_logits=lambda x: x[:, :49]), "draft_logits has to be"),
    ("verify_drafts", dict(draft_logits=lambda x: x[:3]), "draft_logits has to be"),
    ("verify_drafts", dict(draft_logits="bfloat16"), "draft_logits has to be"),
    ("verify_drafts", dict(draft_logits=_WIDE), "draft_logits has to be"),
    ("verify_drafts", dict(draft_logits=lambda x: x.new_zeros(3, 2, 50)[:2].transpose(0, 1)), "draft_logits has to be"),
    ("verify_drafts", dict(draft_logits=lambda x: x[:1].expand_as(x)), "row stride"),
    ("verify_drafts", dict(draft_start=lambda x: x[:2]), "draft_start has to be"),
    ("verify_drafts", dict(draft_start="int64"), "draft_start has to be"),
    ("verify_drafts", dict(temperature=lambda x: x[:1]), "temperature has to be"),
    ("verify_drafts", dict(temperature="double"), "temperature has to be"),
    ("verify_drafts", dict(accepted="int64"), "accepted has to be"),
    ("verify_drafts", dict(accepted=lambda x: x[:1].expand(2)), "accepted has to be"),
    ("verify_drafts", dict(next_token=lambda x: x[:1]), "next_token has to be"),
    ("verify_drafts", dict(prob=lambda x: x[:3]), "prob has to be"),
    ("verify_drafts", dict(prob=lambda x: x[:1].expand(4)), "prob has to be"),
    ("verify_drafts", dict(workspace=lambda x: x[:16]), "workspace of 16 bytes"),
    ("verify_drafts", dict(workspace=lambda x: x[8:]), "not 16-byte aligned"),
]


@gpu
@pytest.mark.parametrize("name", ["paged_append", "paged_attention", "verify_drafts"])
def test_calls_one_change_from_the_refused_ones_are_served(name):
    torch, dfl = _torch(), _dfl()
    getattr(dfl, name)(**_good(torch)[name])
    if name != "verify_drafts":
        args = _good(torch)[name]
        sc = dict(k_scale=torch.ones(2, device="cuda"), v_scale=torch.ones(2, device="cuda"))
        getattr(dfl, name)(**{**args, "k_cache": _E4M3(args["k_cache"]), "v_cache": _E4M3(args["v_cache"]), **sc})
    torch.cuda.synchronize()


@gpu
@pytest.mark.parametrize("name,changes,message", REFUSALS, ids=[f"{i}-{r[0]}-{r[2][:24]}" for i, r in enumerate(REFUSALS)])
def test_calls_refused_for_one_thing(name, changes, message):
    """Each by its own check and in its words, and nothing is launched or written."""
    torch, dfl = _torch(), _dfl()
    args = _good(torch)[name]
    outs = [k for k in ("k_cache", "v_cache", "q_out", "out", "lse", "accepted", "next_token", "prob") if k in args]
    before = {k: args[k].clone() for k in outs}
    call = dict(args)
    for key, how in changes.items():
        if how is None:
            call[key] = None
        elif isinstance(how, str) and how[0] == "f" and how[1:].isdigit():
            call[key] = torch.ones(int(how[1:]), device="cuda")
        elif isinstance(how, str):
            call[key] = args[key].to(getattr(torch, how))
        else:
            call[key] = how(args.get(key))
    with pytest.raises(dfl.DFlashError) as e:
        getattr(dfl, name)(**call)
    assert message in str(e.value) and e.value.code in (dfl._abi.DFLASH_EINVAL, dfl._abi.DFLASH_EGEOM, dfl._abi.DFLASH_ECAPACITY)
    torch.cuda.synchronize()
    assert all(torch.equal(args[k], before[k]) for k in outs)


@gpu
@pytest.mark.parametrize("kind,mark", [("bf16", 0x7fc1), ("f16", 0x7e01)])
@pytest.mark.parametrize("rows,heads", [(1, 4), (16, 8)])
def test_attention_does_not_take_what_the_output_held_for_its_own(kind, mark, rows, heads):
    """Whatever NaN the output's buffer held before: split and whole units among one another, values that are not finite
    in some; the same bits as in a fresh buffer, and rows of no sequence keep theirs."""
    torch, dfl = _torch(), _dfl()
    from test_target_ops import _types
    rng = np.random.default_rng(5)
    lens = [150 + 3 * i for i in range(60)] + [9000, 4000]
    need = [-(-x // 16) for x in lens]
    table = np.full((len(lens), max(need)), -1, np.int32)
    ids = rng.permutation(sum(need))
    for s, m in enumerate(need):
        table[s, :m], ids = ids[:m], ids[m:]
    kc, vc = (torch.from_numpy(rng.standard_normal((sum(need), 16, 2, 64)).astype(np.float32)).cuda().to(_types()[kind])
              for _ in range(2))
    _odd_values(torch, kc, vc, table)
    n = rows * len(lens)
    q = torch.from_numpy(rng.standard_normal((n + 3, heads, 64)).astype(np.float32)).cuda().to(_types()[kind])
    args = (kc, vc, _i32(torch, table), _i32(torch, lens))
    start = _i32(torch, np.arange(len(lens) + 1) * rows)
    want = dfl.paged_attention(q, *args, row_start=start, out=torch.zeros_like(q))
    for _ in range(20):
        out = torch.zeros_like(q)
        out.view(torch.int16).fill_(mark)
        dfl.paged_attention(q, *args, row_start=start, out=out)
        assert torch.equal(out.view(torch.int16)[:n], want.view(torch.int16)[:n])
        assert (out.view(torch.int16)[n:] == mark).all()
    assert not torch.isfinite(want).all() and torch.isfinite(want).any()


@gpu
def test_calls_without_rows_take_any_strides():
    """Tensors without elements have whatever strides they came with (those of an empty numpy array are 0)."""
    torch, dfl = _torch(), _dfl()
    good = _good(torch)
    none = lambda *s, dtype=torch.bfloat16: torch.empty(1, dtype=dtype, device="cuda").as_strided((0, *s), (0,) * (len(s) + 1))  # noqa: E731
    a = good["paged_append"]
    start = _i32(torch, [0, 0, 0])
    q = dfl.paged_append(**{**a, "k": none(2, 64), "v": none(2, 64), "q": none(4, 64), "q_out": None, "row_start": start})
    assert q.shape == (0, 4, 64)
    b = good["paged_attention"]
    y = dfl.paged_attention(**{**b, "q": none(4, 64), "out": None, "lse": none(4, dtype=torch.float32), "row_start": start})
    assert y.shape == (0, 4, 64)
    no_pages = none(16, 2, 64)
    y = dfl.paged_attention(b["q"], no_pages, no_pages, b["table"], b["kv_len"], row_start=b["row_start"])
    assert (y == 0).all()
    f32 = torch.float32
    t = torch.randn(2, 50, device="cuda")
    acc, nxt, prob = dfl.verify_drafts(t, none(dtype=torch.int32), none(dtype=f32), torch.full((2,), 0.5, device="cuda"),
                                       draft_logits=none(50, dtype=f32), draft_start=start)
    res, _ = O.verify(f64(t), [], [], [0.5, 0.5])
    assert acc.tolist() == [0, 0] and nxt.tolist() == [r[1] for r in res] and prob.shape == (0,)


@gpu
@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("rows,heads", [(1, 4), (12, 8)])
def test_attention_of_scores_that_are_all_minus_infinity(kind, rows, heads):
    """Rows of which every score is -inf weigh nothing: 0, and -inf; those beside them that see another key do."""
    torch, dfl = _torch(), _dfl()
    from test_target_ops import _types
    rng = np.random.default_rng(2)
    kc, vc = (torch.from_numpy(rng.standard_normal((4, 16, 1, 64)).astype(np.float32)).cuda().to(_types()[kind])
              for _ in range(2))
    q = torch.from_numpy(rng.standard_normal((2 * rows, heads, 64)).astype(np.float32)).cuda().to(_types()[kind])
    q[..., 7] = -1.0
    kc[0, :, 0, 7] = float("inf")  # the first page's keys: scores of -inf for every row
    table, lens = [[0, 1], [0, 2]], [16, 30]
    lse = torch.zeros(2 * rows, heads, device="cuda")
    out = dfl.paged_attention(q, kc, vc, _i32(torch, table), _i32(torch, lens), lse=lse)
    ref, rl, mag, _ = O.paged_attention(f64(q), f64(kc), f64(vc), table, lens)
    assert (out[:rows] == 0).all() and (lse[:rows] == -float("inf")).all()
    assert (np.abs(f64(out) - ref) <= 2.0 ** -8 * np.abs(ref) + 1e-3 * mag).all()
    got = f64(lse)
    some = np.isfinite(rl)
    assert np.array_equal(np.isneginf(got), np.isneginf(rl)) and np.abs(got[some] - rl[some]).max() < 1e-3


@gpu
def test_attention_of_a_prompt_with_an_infinity_that_every_row_sees():
    """4096 rows of 8 heads have such a column, in split and in whole units: still a matter of milliseconds (10.6 here;
    3077 where every share that had such rows went through all of them)."""
    torch, dfl = _torch(), _dfl()
    g = torch.Generator("cuda").manual_seed(0)
    n, page = 2048, 64
    kc, vc = (torch.randn(4 * n // page, page, 2, 64, device="cuda", generator=g).to(torch.bfloat16) for _ in range(2))
    q = torch.randn(2 * n, 8, 64, device="cuda", generator=g).to(torch.bfloat16)
    vc[:, 5, :, 9] = float("inf")
    vc[:, 6, :, 10], vc[:, 7, :, 10] = float("inf"), float("-inf")
    table = torch.arange(4 * n // page, device="cuda", dtype=torch.int32).view(2, -1)
    args = (q, kc, vc, table, _i32(torch, [2 * n, n + 100]))
    out = dfl.paged_attention(*args)
    assert (out[..., 9] == float("inf")).all() and torch.isnan(out[..., 10]).all()
    rest = [c for c in range(64) if c not in (9, 10)]
    assert torch.isfinite(out[..., rest]).all()
    a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    torch.cuda.synchronize()
    a.record()
    dfl.paged_attention(*args)
    b.record()
    torch.cuda.synchronize()
    assert a.elapsed_time(b) < 500
