"""Calls around a target's small cache that once answered wrongly or were never made by a test."""
import ctypes as C
import os
import re

import numpy as np
import pytest

from oracle import target as O
from test_target_ops import _cache_struct, _dfl, _i32, _layout, _rows_struct, _starts, _torch, _types, f64
from test_target_small_cache import (_any_cache, _cache4, _cached4, _check_evict, _good, _raw, _values4, _weights_struct)

gpu = pytest.mark.gpu


@pytest.fixture(scope="module")
def lib():
    from block_speculative_drafting_gb300.csrc.build import build
    build()
    return _dfl().lib()


# --------------------------------------------------------------------------- evict: keys and values are apart
@pytest.mark.parametrize("cache,bad", [(_cache_struct, dict(v=4096)), (_cache4, dict(v=4096)), (_cache4, dict(v_block=4096)),
                                       (_cache4, dict(v=4096, v_block=4096))], ids=["bf16", "codes", "blocks", "both"])
def test_evict_refuses_keys_and_values_in_one_memory(lib, cache, bad):
    """Rows of both would move at once, over one another."""
    from block_speculative_drafting_gb300 import _abi
    w, r = _weights_struct(), _rows_struct(n_rows=0)
    call = lambda c, r=r: lib.dflash_paged_evict(C.byref(c), C.byref(r), 8, 2, 3, C.byref(w), C.byref(w), 4096, None,  # noqa: E731
                                                 None, 4096, 16, None)
    assert call(cache(**bad)) == _abi.DFLASH_EINVAL and b"one memory" in lib.dflash_last_error(None)
    assert call(cache()) == _abi.DFLASH_ECAPACITY  # apart: the next check is the workspace's
    assert call(cache(k=None, v=None, k_block=None, v_block=None, n_pages=0)) == _abi.DFLASH_ECAPACITY
    assert call(cache(**bad), _rows_struct(n_rows=0, n_seqs=0)) == 0


def test_evict_refuses_lengths_and_counts_in_one_memory(lib):
    """The counts grow by what is taken out, the lengths are set: of one memory they were the sum of both."""
    from block_speculative_drafting_gb300 import _abi
    w, r, c = _weights_struct(), _rows_struct(n_rows=0), _cache4()
    call = lambda new, evicted: lib.dflash_paged_evict(C.byref(c), C.byref(r), 8, 2, 3, C.byref(w), C.byref(w), new, None,  # noqa: E731
                                                       evicted, 4096, 16, None)
    assert call(8192, 8192) == _abi.DFLASH_EINVAL and b"one memory" in lib.dflash_last_error(None)
    assert call(8192, 12288) == call(4096, 8192) == _abi.DFLASH_ECAPACITY  # (4096 is kv_len: new_len may be)


@gpu
def test_evict_refuses_one_tensor_as_keys_and_values():
    torch, dfl = _torch(), _dfl()
    args = _good(torch)["paged_evict"]
    for bad in (dict(v_cache=args["k_cache"]), dict(v_block=args["k_block"])):
        with pytest.raises(dfl.DFlashError, match="one memory"):
            dfl.paged_evict(**{**args, **bad})
    # pages that hold both, one behind the other, are apart
    both = torch.zeros(6, 2, 16, 2, 32, dtype=torch.uint8, device="cuda")
    dfl.paged_evict(**{**args, "k_cache": both[:, 0], "v_cache": both[:, 1]})
    torch.cuda.synchronize()


# --------------------------------------------------------------------------- append: one memory holds the values
@gpu
@pytest.mark.parametrize("kind", ["bf16", "e4m3", "e2m1"])
@pytest.mark.parametrize("rows", [1, 900])
def test_append_into_one_memory_leaves_the_values_there(kind, rows):
    torch, dfl = _torch(), _dfl()
    gen = torch.Generator("cuda").manual_seed(rows)
    k, v = torch.randn(2, rows, 3, 128, device="cuda", generator=gen).to(torch.bfloat16)
    pages = -(-rows // 16)
    table, lens = torch.arange(pages, dtype=torch.int32, device="cuda")[None], torch.tensor([rows], dtype=torch.int32).cuda()
    scale = torch.full((3,), 0.25, device="cuda") if kind != "bf16" else None
    type_ = {"bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn, "e2m1": torch.uint8}[kind]

    def cache():
        c = torch.zeros(pages, 16, 3, 64 if kind == "e2m1" else 128, device="cuda").to(type_)
        return c, torch.zeros(pages, 16, 3, 8, device="cuda").to(torch.float8_e4m3fn) if kind == "e2m1" else None

    (one, blocks), (a, a_blocks), (b, b_blocks) = cache(), cache(), cache()
    kw = dict(k_scale=scale, v_scale=scale)
    for _ in range(5):
        dfl.paged_append(one, one, k, v, table, lens, k_block=blocks, v_block=blocks, **kw)
        dfl.paged_append(a, b, k, v, table, lens, k_block=a_blocks, v_block=b_blocks, **kw)
        torch.cuda.synchronize()
        assert torch.equal(one.view(torch.uint8), b.view(torch.uint8)) and not torch.equal(a.view(torch.uint8), b.view(torch.uint8))
        assert blocks is None or torch.equal(blocks.view(torch.uint8), b_blocks.view(torch.uint8))


# --------------------------------------------------------------------------- read: either output alone names the type
@gpu
@pytest.mark.parametrize("given", ["k_out", "v_out"])
def test_read_takes_its_type_from_either_output(given):
    torch, dfl = _torch(), _dfl()
    args = {k: v for k, v in _good(torch)["paged_read"].items() if k not in ("k_out", "v_out", "dtype")}
    to = torch.full((4, 2, 64), 7.0, device="cuda")
    got = dfl.paged_read(**args, **{given: to})
    want = dfl.paged_read(**args, dtype=torch.float32)
    assert got["kv".index(given[0])] is to
    assert all(x.dtype == torch.float32 and torch.equal(x, y) for x, y in zip(got, want))
    assert dfl.paged_read(**args)[0].dtype == torch.bfloat16

# --------------------------------------------------------------------------- key weights of many rows
def _few_rows():
    """Rows times group a sequence, on average, up to which the warp-MMA kernel serves a call."""
    src = os.path.join(os.path.dirname(_dfl().__file__), "csrc", "k_paged_weights.cu")
    with open(src) as f:
        (most,) = re.findall(r"if \(per <= (\d+)\)", f.read())
    return int(most)


def _check_many(kind, src, group, rows, lens, kvh=1, hd=128, page=16, window=0, uniform=False, bad=(), order="slot", extra=0,
                scale=None, seed=0, spread=1.0, poison=None, nothing=(), few=False):
    """A call that the tcgen05 kernel serves (or with `few` the warp-MMA one), against the formula in 64 bits.  Tolerances as in test_target_small_cache.py."""
    torch, dfl = _torch(), _dfl()
    rng = np.random.default_rng(seed)
    table, n_pages = _layout(torch, rng, [max(l, 0) for l in lens], rows, page, bad=bad)
    R, heads, cap, starts = sum(rows) + extra, group * kvh, table.shape[1] * page, None if uniform else _starts(rows)
    assert (-(-R // len(lens)) * group > _few_rows()) != few
    q = torch.from_numpy(spread * rng.standard_normal((R, heads, hd)).astype(np.float32)).cuda().to(_types()[src])
    kc, kb, ks, k64 = _any_cache(torch, rng, (n_pages, page, kvh, hd), kind, order)
    if poison is not None:
        k64 = poison(torch, kc, kb, table, k64.copy())
    factor, q64 = hd ** -0.5 if scale is None else scale, f64(q)
    lse, seen = np.full((R, heads), -np.inf, np.float32), {}
    for s, a, n in O.rows_of(len(lens), R, starts):
        L = min(max(lens[s], 0), cap) if n else 0
        j = np.arange(L)
        ids = table[s][j // page] if L else np.zeros(0, int)
        held = (ids >= 0) & (ids < n_pages)
        keys = k64[np.where(held, ids, 0), j % page]
        p = lens[s] - n + np.arange(n)[:, None]
        see = (j <= p) & held & ((j > p - window) if window else True)
        for h in range(kvh):
            x = q64[a:a + n, h * group:(h + 1) * group].reshape(n * group, hd)
            with np.errstate(all="ignore"):
                sc = np.where(np.repeat(see, group, 0), factor * (x @ keys[:, h].T), -np.inf)
                size = factor * (np.abs(x) @ np.abs(keys[:, h]).T)
                real = np.where(np.isnan(sc), -np.inf, sc)  # (the lse is an argument: it need not be NaN)
                m = real.max(1, initial=-1e300, keepdims=True)
                ls = (m + np.log(np.exp(real - m).sum(1, keepdims=True)))[:, 0]
            lse[a:a + n, h * group:(h + 1) * group] = ls.reshape(n, group)
            seen[s, h] = a, n, L, held, sc, size
    for r, h in nothing:
        lse[r, h] = -np.inf
    w0 = rng.random((len(lens), kvh, cap + 5)).astype(np.float32)
    want, amp = w0.astype(np.float64), np.zeros(w0.shape)
    for (s, h), (a, n, L, held, sc, size) in seen.items():
        ls = lse[a:a + n, h * group:(h + 1) * group].reshape(-1, 1).astype(np.float64)
        with np.errstate(all="ignore"):
            w = np.where(ls == -np.inf, 0.0, np.exp(sc - ls))
            size = np.where(w == 0, 0.0, w * size)
        old = np.where(np.arange(L) < lens[s] - n, want[s, h, :L], 0.0)
        want[s, h, :L] = np.where(held, old + w.sum(0), want[s, h, :L])
        amp[s, h, :L] = size.sum(0)
    W = torch.from_numpy(w0).cuda()
    got = dfl.paged_key_weights(W, q, kc, _i32(torch, table), _i32(torch, lens), torch.from_numpy(lse).cuda(),
                                row_start=None if uniform else _i32(torch, starts), scale=scale, window=window, k_scale=ks,
                                k_block=kb)
    torch.cuda.synchronize()
    assert got is W
    g, terms = f64(W), max(rows) * group
    with np.errstate(all="ignore"):
        tol = hd * 2.0 ** -23 * amp + (2.0 ** -19 + terms * 2.0 ** -24) * np.abs(want) + 1e-37
        assert np.array_equal(np.isnan(want), np.isnan(g))
        off = np.where(np.isnan(want), 0.0, np.abs(g - want) / tol)
    assert off.max() <= 1, (off.max(), np.argwhere(off > 1)[:4])
    still = want == w0  # what the call does not reach stays
    assert np.array_equal(g[still], want[still])


KINDS = [("bf16", "bf16"), ("f16", "f16"), ("e4m3", "bf16"), ("e4m3", "f16"), ("e2m1", "bf16"), ("e2m1", "f16")]
# a sequence's rows under a group of 8: one tile of 128 queries, three, six (the keys stay from two or three on)
MANY = [9, 38, 88]


@gpu
@pytest.mark.parametrize("kind,src", KINDS)
@pytest.mark.parametrize("rows", MANY)
def test_weights_of_many_rows_windows(kind, src, rows):
    """Windows shorter than a tile of keys, of some tiles, and longer than the sequence."""
    for window, hd in ((5, 128), (140, 64), (333, 128), (5000, 64)):
        _check_many(kind, src, 8, (rows, rows + 1), (rows + 420, rows + 90), hd=hd, window=window, page=48, seed=window)


@gpu
@pytest.mark.parametrize("kind,src", KINDS)
@pytest.mark.parametrize("rows", MANY)
def test_weights_of_many_rows_holes(kind, src, rows):
    """Pages that are not held, rows of no sequence, a sequence without rows, rows before position 0, rows of lse -inf,
    uniform rows (row_start None), both orders of slots and heads."""
    nothing = [(r, h) for r in range(0, 3 * rows, 5) for h in (0, 3)] + [(rows // 2, h) for h in range(8)]
    _check_many(kind, src, 8, (rows, 0, 3 * rows, 3), (rows + 300, 9, 3 * rows - rows // 2, 150), extra=4, nothing=nothing,
                bad=((0, 1), (0, 2), (2, 0), (3, 1)), page=64, order="head", seed=rows)
    _check_many(kind, src, 8, (rows,) * 3, (rows + 200, rows // 2, rows + 129), uniform=True, hd=64, nothing=nothing, kvh=2,
                page=33, seed=rows + 1)


@gpu
@pytest.mark.parametrize("kind,src", KINDS)
@pytest.mark.parametrize("rows", MANY)
def test_weights_of_many_rows_values(kind, src, rows):
    """Keys of NaN that all rows, some rows and one row see, and behind the last token; large scores; large queries."""
    lens, page = (rows + 200, rows + 131), 16

    def nan(kc, kb, at):
        if kb is None:
            kc[at][0, 7] = float("nan")
        else:
            kb.view(_torch().uint8)[at][0, 2] = 0x7f

    def poison(torch, kc, kb, table, k64):
        for s, p in ((0, 150), (0, lens[0] - 1 - rows // 2), (1, lens[1] - 1), (1, 3)):
            at = int(table[s][p // page]), p % page
            nan(kc, kb, at)
            k64[at][0, 7] = np.nan
        for s, l in enumerate(lens):
            for slot in range(l % page, page if l % page else 0):
                nan(kc, kb, (int(table[s][l // page]), slot))
        return k64

    _check_many(kind, src, 8, (rows, rows), lens, poison=poison, seed=rows, page=page)
    _check_many(kind, src, 8, (rows, rows), lens, spread=20.0, scale=0.5, seed=rows)
    wide = 1e3 if src == "f16" else 1e6
    _check_many(kind, src, 8, (rows, rows), lens, spread=wide, scale=1 / wide, hd=64, seed=rows + 1)


@gpu
@pytest.mark.parametrize("kind,src", KINDS)
def test_weights_of_many_rows_one_long_among_short(kind, src):
    """One sequence's rows alone put the average over the rule; the others have one or none; heads of several groups."""
    _check_many(kind, src, 3, (1, 1, 0, 200, 1, 1, 1, 1), (700, 40, 30, 700, 1, 129, 128, 257), kvh=3, page=7, hd=64)
    _check_many(kind, src, 1, (300, 2), (300, 2), kvh=2, page=16)


@gpu
@pytest.mark.parametrize("kind,src", KINDS)
@pytest.mark.parametrize("rows", [9, 88])
def test_weights_of_many_rows_repeat_bit_for_bit(kind, src, rows):
    torch, dfl = _torch(), _dfl()
    rng = np.random.default_rng(rows)
    lens = (1500 + rows, rows, 300 + rows)
    table, n_pages = _layout(torch, rng, lens, (rows,) * 3, 16)
    kc, kb, ks, k64 = _any_cache(torch, rng, (n_pages, 16, 2, 128), kind)
    q = torch.from_numpy(rng.standard_normal((3 * rows, 16, 128)).astype(np.float32)).cuda().to(_types()[src])
    table, lens = _i32(torch, table), _i32(torch, lens)
    lse = torch.empty(3 * rows, 16, device="cuda")
    same = dict(k_scale=ks, k_block=kb)
    dfl.paged_attention(q, kc, kc, table, lens, v_block=kb, v_scale=ks, lse=lse, **same)
    assert rows * 8 > _few_rows()
    make = lambda: torch.zeros(3, 2, table.shape[1] * 16, device="cuda")  # noqa: E731
    call = lambda w, **kw: dfl.paged_key_weights(w, q, kc, table, lens, lse, **same, **kw)  # noqa: E731
    want = call(make())
    # each row and query head hands out a weight of 1 in all, but for the scores' rounding (a sum of 128 products kept to 24
    # bits each), the lse's too, and the exponential's
    norm = lambda x: np.linalg.norm(x, axis=-1).max()  # noqa: E731
    off = 2 * 128 * 2.0 ** -24 * 128 ** -0.5 * norm(f64(q)) * norm(k64) + 2.0 ** -19
    assert (want.double().sum(-1) - 8 * rows).abs().max() <= 8 * rows * off
    streams = [torch.cuda.Stream() for _ in range(3)]
    bufs = [make() for _ in range(9)]
    torch.cuda.synchronize()
    for i, w in enumerate(bufs):
        call(w, stream=streams[i % 3].cuda_stream)
    torch.cuda.synchronize()
    assert all(torch.equal(w, want) for w in bufs)


# --------------------------------------------------------------------------- key weights, many rows of one sequence among few
@gpu
@pytest.mark.parametrize("kind,src", KINDS)
@pytest.mark.parametrize("hd", [64, 128])
def test_weights_of_one_long_sequence_among_short_ones(kind, src, hd):
    """Sequences of several sets of 64 rows in a call that the warp-MMA kernel serves: shares of the line end in their tiles."""
    rng = np.random.default_rng(hd)
    for at, long, group, kvh, window, n in ((0, 75, 8, 2, 0, 20), (30, 150, 4, 1, 0, 31), (7, 260, 3, 2, 200, 40), (35, 40, 5, 3, 0, 36)):
        rows = [int(x) for x in rng.integers(0, 2, n)]
        lens = [int(x) for x in rng.integers(1, 200, n)]
        rows[at], lens[at] = long, long + int(rng.integers(300, 700))
        rows[n // 2], lens[n // 2] = long // 2, long // 3  # (rows before position 0, and few keys)
        _check_many(kind, src, group, tuple(rows), tuple(lens), kvh=kvh, hd=hd, window=window, page=48, few=True, seed=at)


@gpu
def test_weights_of_one_long_sequence_among_short_ones_cost_what_both_do():
    """31 sequences of one row and one of 400: once 26 times the two calls on their own (a few CTAs had all of its rows).  The
    bound is 5 times: fixed times, and a kernel for few rows."""
    torch, dfl = _torch(), _dfl()
    L, page = 4096, 64
    kc = torch.randn(32 * L // page, page, 8, 128, device="cuda").to(torch.bfloat16)
    table = torch.arange(32 * L // page, dtype=torch.int32, device="cuda").view(32, -1)

    def time(rows):
        n, R = len(rows), sum(rows)
        q, lse = torch.randn(R, 32, 128, device="cuda").to(torch.bfloat16), torch.full((R, 32), 9.0, device="cuda")
        w, start, lens = torch.zeros(n, 8, L, device="cuda"), _i32(torch, _starts(rows)), _i32(torch, (L,) * n)
        t = []
        for _ in range(7):
            a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            a.record()
            for _ in range(4):
                dfl.paged_key_weights(w, q, kc, table[:n], lens, lse, row_start=start)
            b.record()
            torch.cuda.synchronize()
            t.append(a.elapsed_time(b))
        return sorted(t)[3]

    assert time((1,) * 31 + (400,)) < 5 * (time((1,) * 32) + time((400,)))


# --------------------------------------------------------------------------- 4-bit append of keys and values as they come
def _check_bare(src="bf16", hd=128, kvh=2, page=16, rows=(1, 3), lens=(5, 40), bad=(), order="slot", extra=0, uniform=False,
                powers=False, scaled=True, put=None, seed=0):
    """Without queries, norms and a rotation: the kernel that is written for such calls."""
    torch, dfl = _torch(), _dfl()
    rng = np.random.default_rng(seed)
    table, n_pages = _layout(torch, rng, lens, rows, page, bad=bad)
    R = sum(rows) + extra
    kv = torch.from_numpy(rng.standard_normal((R, 2 * kvh + 1, hd)).astype(np.float32)).cuda().to(_types()[src])
    k, v = kv[:, :kvh], kv[:, kvh + 1:]  # slices of a wider projection
    if put is not None:
        put(k, v)
    caches = [_cached4(torch, rng, (n_pages, page, kvh, hd), order)[:2] for _ in range(2)]
    old = [[_raw(x) for x in c] for c in caches]
    make = lambda: torch.from_numpy((np.exp2(-rng.integers(3, 7, kvh)) if powers else (0.5 + rng.random(kvh)) / 64)  # noqa: E731
                                    .astype(np.float32)).cuda()
    sc = [make(), make()] if scaled else [None, None]
    starts = None if uniform else _starts(rows)
    got = dfl.paged_append(caches[0][0], caches[1][0], k, v, _i32(torch, table), _i32(torch, lens),
                           row_start=None if uniform else _i32(torch, starts), k_scale=sc[0], v_scale=sc[1],
                           k_block=caches[0][1], v_block=caches[1][1])
    torch.cuda.synchronize()
    assert got is None
    slots = O.paged_append(f64(k), f64(v), None, table, lens, page, n_pages, starts)[0]
    at = tuple(np.array(x, dtype=int) for x in zip(*slots)) if slots else (np.zeros(0, int),) * 2
    for side, (codes, blocks) in enumerate(caches):
        # every other slot as it was
        for x, was in zip((codes, blocks), old[side]):
            now, before = (y.reshape(n_pages, page, kvh, -1).copy() for y in (_raw(x), was))
            now[at] = before[at] = 0
            assert np.array_equal(now, before)
        if not slots:
            continue
        t = np.stack([kv_[side] for kv_ in slots.values()])
        t = t / (f64(sc[side])[:, None] if scaled else 1.0)
        g = t.reshape(*t.shape[:-1], -1, 16)
        s, y = f64(blocks)[at], _values4(codes, blocks)[at].reshape(g.shape)
        # x / scale and t / s (or max|t| / 6) round in 32 bits, half a step each; x / a power of two is exact
        e = (2 if scaled and not powers else 1) * 2.0 ** -24
        with np.errstate(all="ignore"):
            top = np.abs(g).max(-1) / 6
            lo, hi = O.round_e4m3(top * (1 - e)), O.round_e4m3(top * (1 + e))
            assert np.array_equal(np.isnan(s), np.isnan(top)) and (np.isnan(s) | ((s >= lo) & (s <= hi))).all()
            u = np.where(s[..., None] > 0, g / s[..., None], 0.0).clip(-64, 64)
            a, b = O.round_e2m1(u * (1 - e)), O.round_e2m1(u * (1 + e))
            y = np.where(s[..., None] > 0, y / s[..., None], 0.0)
            ok = np.isnan(s)[..., None] | ((y >= np.minimum(a, b)) & (y <= np.maximum(a, b)))
        assert ok.all(), (side, np.argwhere(~ok)[:4])


def _odd_values(k, v):
    """Blocks of zeros, of values under the smallest scale, with NaN and infinities, ties, and far beyond the largest scale."""
    torch = _torch()
    k[0, 0, :16] = 0.0
    k[0, 0, 16:32] = 1e-6
    k[0, 0, 32] = float("nan")
    k[0, -1, 3] = float("inf")
    k[0, -1, 20] = -float("inf")
    v[-1, 0, 5] = 6e4
    v[-1, 0, 6] = -6e4
    v[-1, -1, :16] = torch.arange(16, device="cuda") / 4
    v[-1, -1, 16:32] = -torch.arange(16, device="cuda") / 128
    v[-1, -1, 63] = float("nan")


@gpu
@pytest.mark.parametrize("src", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("hd", [64, 128])
def test_bare_append4(src, hd):
    _check_bare(src, hd, powers=True, put=_odd_values, seed=hd)
    _check_bare(src, hd, kvh=3, rows=(2, 0, 5), lens=(2, 9, 130), put=_odd_values, seed=1)
    _check_bare(src, hd, kvh=9, scaled=False, rows=(4, 3), lens=(2, 41), extra=3, page=7, order="head", seed=2)
    _check_bare(src, hd, kvh=1, rows=(4,) * 3, lens=(9, 4, 64), uniform=True, page=1, seed=3)
    _check_bare(src, hd, kvh=40, rows=(4, 3, 40), lens=(2, 40, 41), bad=((1, 2), (2, 0), (2, 1), (2, 2)), page=16, extra=2, seed=5)


@gpu
@pytest.mark.parametrize("src", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("hd,kvh", [(64, 40), (128, 19)])
def test_bare_append4_rounds_of_heads(src, hd, kvh):
    """Rows enough for a warp each, with more heads than it has on their way at once."""
    _check_bare(src, hd, kvh=kvh, rows=(900, 1), lens=(1000, 2000), page=64, powers=True, put=_odd_values, seed=6)
    _check_bare(src, hd, kvh=kvh, rows=(300, 700), lens=(300, 700), page=48, order="head", seed=7)


# --------------------------------------------------------------------------- eviction from many heads
# (type, head_dim): rows that a CTA moves at a time where a (sequence, head)'s keys are one CTA's
ROUND = {("bf16", 128): 128, ("f16", 64): 256, ("e4m3", 128): 256, ("e2m1", 128): 512, ("e4m3", 64): 512, ("e2m1", 64): 1024}


@gpu
@pytest.mark.parametrize("kind,hd", ROUND)
@pytest.mark.parametrize("rounds,aside", [(2, False), (3, True), (5, False)])
def test_evict_many_heads_in_rounds(kind, hd, rounds, aside):
    """Heads enough for the whole-row form, an even and odd number of rounds, the last one whole or not; weights and
    block scales, whose rounds are 2048 tokens, take several too with the longest."""
    keep = rounds * ROUND[kind, hd] - (0 if rounds == 2 else 5)
    n, kvh = (8, 8) if keep < 3000 else (13, 4)
    assert 3 * n * kvh >= _torch().cuda.get_device_properties(0).multi_processor_count
    rng = np.random.default_rng(keep)
    lens = [keep, keep + 1, keep - 1, 2 * keep + 7] + [int(keep + rng.integers(2, keep)) for _ in range(n - 4)]
    _check_evict(kind, hd, kvh=kvh, page=48, lens=lens, keep=keep, first=3, recent=keep // 4, aside=aside, order="head" if aside else "slot",
                 given=not aside, bad=((3, 1),), seed=rounds)
