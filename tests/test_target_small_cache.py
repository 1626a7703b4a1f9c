"""What keeps the target's cache small (the 4-bit cache in paged_append, paged_read and paged_attention;
paged_key_weights; paged_evict) against plain float64 (oracle/target.py), and the refusals of these calls.

Tolerances, from the arithmetic (a rounding to type t is off by half a step, finfo(t).eps / 2 relative):
  append     x / (head's scale) and the norm and rotation before it are 32-bit: t is off by d = 2^-20 of the pair's
             magnitude (2^-23 of |t| without either).  The block scale then is one of the e4m3 values that max|t| +- d gives,
             and a code one that t +- d gives with that scale; without norm and rotation and with scales that are powers of two
             both are the definition's own
  read       code * block scale is exact, times the head's scale rounds in 32 bits, then to the output's type
  attention  as for the other caches (tests/test_target_ops.py): elements are exact in the products; a bf16 output's weights
             are one f16 (its half step, relative), a f16 output's are a pair
  weights    a score is a sum of head_dim products kept to 23 bits each, which moves exp(s - lse) by as much relative; the
             exponential is within 2^-20; N terms add up in 32 bits
  evict      nothing is computed: equal
"""
import ctypes as C

import numpy as np
import pytest

from oracle import target as O
from test_target_ops import (HALF, TINY, _cache_struct, _cached, _dfl, _head_struct, _i32, _layout, _rows_struct, _starts,
                             _torch, _types, f64)

gpu = pytest.mark.gpu
E2M1 = O.E2M1


# --------------------------------------------------------------------------- refusals (no device)
@pytest.fixture(scope="module")
def lib():
    from block_speculative_drafting_gb300.csrc.build import build
    build()
    return _dfl().lib()


def _cache4(**kw):
    from block_speculative_drafting_gb300 import _abi
    c = _cache_struct(dtype=_abi.E2M1, k_block=4096, v_block=8192)
    for st in (c.k_strides, c.v_strides):
        st[0], st[1], st[2] = 16 * 2 * 32, 2 * 32, 32
    for st in (c.k_block_strides, c.v_block_strides):
        st[0], st[1], st[2] = 16 * 2 * 4, 2 * 4, 4
    for k, v in kw.items():
        if k.endswith("_strides"):
            for i in range(3):
                getattr(c, k)[i] = v[i]
        else:
            setattr(c, k, v)
    return c


def _weights_struct(**kw):
    from block_speculative_drafting_gb300 import _abi
    w = _abi.KeyWeights(4096, 64, 128, 64)
    for k, v in kw.items():
        setattr(w, k, v)
    return w


BAD_BLOCKS = [dict(k_block=None), dict(v_block=None), dict(k_block=4098), dict(k_strides=(1024, 72, 32)),
              dict(v_block_strides=(128, 8, 6)), dict(k_block_strides=(-128, 8, 4)), dict(k_scale=4096),
              dict(v_strides=(1 << 31, 64, 32)), dict(k_block_strides=(1 << 31, 8, 4))]


@pytest.mark.parametrize("bad", BAD_BLOCKS, ids=lambda b: next(iter(b)))
def test_paged_calls_refuse_bad_block_scales(lib, bad):
    from block_speculative_drafting_gb300 import _abi
    c, r, k, q = _cache4(**bad), _rows_struct(), _head_struct(2), _head_struct(4)
    w = _weights_struct()
    e = _rows_struct(n_rows=0)
    assert lib.dflash_paged_append(C.byref(c), C.byref(r), C.byref(k), C.byref(k), C.byref(q), C.byref(q), None, None,
                                   1e-6, None, None) == _abi.DFLASH_EINVAL
    assert lib.dflash_paged_attention(C.byref(c), C.byref(r), C.byref(q), C.byref(q), None, 0.1, 0, 4096, 1 << 40,
                                      None) == _abi.DFLASH_EINVAL
    assert lib.dflash_paged_read(C.byref(c), C.byref(r), C.byref(k), C.byref(k), None) == _abi.DFLASH_EINVAL
    assert lib.dflash_paged_key_weights(C.byref(c), C.byref(r), C.byref(q), 4096, 0.1, 0, C.byref(w),
                                        None) == _abi.DFLASH_EINVAL
    assert lib.dflash_paged_evict(C.byref(c), C.byref(e), 8, 0, 0, C.byref(w), C.byref(w), 4096, None, None, 4096, 1 << 40,
                                  None) == _abi.DFLASH_EINVAL
    assert lib.dflash_last_error(None) != b""


def test_paged_read_refuses_bad_arguments(lib):
    from block_speculative_drafting_gb300 import _abi

    def call(c=_cache4(), r=_rows_struct(), k=_head_struct(2), v=_head_struct(2, data=8192)):
        ref = lambda x: None if x is None else C.byref(x)  # noqa: E731
        return lib.dflash_paged_read(ref(c), ref(r), ref(k), ref(v), None)

    for bad in (dict(c=None), dict(r=None), dict(k=None, v=None), dict(v=_head_struct(2)), dict(k=_head_struct(3)), dict(v=_head_struct(2, dtype=0)),
                dict(v=_head_struct(2, dtype=3), k=None), dict(k=_head_struct(2, data=4104)),
                dict(k=_head_struct(2, row_stride=130)), dict(r=_rows_struct(n_rows=5)), dict(r=_rows_struct(table=None))):
        assert call(**bad) == _abi.DFLASH_EINVAL, bad
    assert call(r=_rows_struct(n_rows=0)) == 0 and call(r=_rows_struct(n_rows=0), k=None) == 0


def test_paged_key_weights_refuses_bad_arguments(lib):
    from block_speculative_drafting_gb300 import _abi

    def call(c=_cache4(), r=_rows_struct(), q=_head_struct(4), lse=4096, scale=0.1, window=0, w=_weights_struct()):
        ref = lambda x: None if x is None else C.byref(x)  # noqa: E731
        return lib.dflash_paged_key_weights(ref(c), ref(r), ref(q), lse, scale, window, ref(w), None)

    for bad in (dict(c=None), dict(r=None), dict(q=None), dict(q=_head_struct(3)), dict(q=_head_struct(4, dtype=0)),
                dict(c=_cache_struct(dtype=2)), dict(lse=None), dict(lse=4098), dict(scale=0.0), dict(scale=float("nan")),
                dict(window=-1), dict(window=(1 << 30) + 1), dict(w=None), dict(w=_weights_struct(data=None)),
                dict(w=_weights_struct(data=4098)), dict(w=_weights_struct(positions=63)),
                dict(w=_weights_struct(seq_stride=-1)), dict(w=_weights_struct(head_stride=-1)),
                dict(r=_rows_struct(max_pages=(1 << 27) - 8192), w=_weights_struct(positions=1 << 31), q=_head_struct(65536),
                     c=_cache4(kv_heads=2))):
        assert call(**bad) == _abi.DFLASH_EINVAL, bad
    assert call(r=_rows_struct(n_rows=0)) == 0


def test_paged_evict_refuses_bad_arguments(lib):
    from block_speculative_drafting_gb300 import _abi
    rows = lambda **kw: _rows_struct(**{"n_rows": 0, **kw})  # noqa: E731

    def call(c=_cache4(), r=rows(), keep=8, first=2, recent=3, w=_weights_struct(), o="w", new=4096, kept=None, evicted=None,
             ws=4096, nb=1 << 40):
        ref = lambda x: None if x is None else C.byref(x)  # noqa: E731
        return lib.dflash_paged_evict(ref(c), ref(r), keep, first, recent, ref(w), ref(w if o == "w" else o), new, kept,
                                      evicted, ws, nb, None)

    for bad in (dict(c=None), dict(r=None), dict(r=_rows_struct()), dict(r=rows(row_start=4096)), dict(keep=0),
                dict(keep=4), dict(first=-1), dict(recent=-1), dict(first=2 ** 31 - 1, recent=2 ** 31 - 1),
                dict(w=None), dict(o=None), dict(w=_weights_struct(positions=63)), dict(o=_weights_struct(head_stride=65)),
                dict(o=_weights_struct(data=8192, positions=63)), dict(new=None), dict(new=4098), dict(kept=4098),
                dict(evicted=4098), dict(ws=None), dict(ws=4104), dict(r=rows(kv_len=None)), dict(r=rows(table=None)),
                dict(r=rows(n_seqs=1 << 23, table_stride=0), c=_cache4(kv_heads=64))):
        assert call(**bad) == _abi.DFLASH_EINVAL, bad
    assert call(nb=16) == _abi.DFLASH_ECAPACITY
    assert call(r=rows(n_seqs=0)) == 0  # nothing to do, nothing launched
    size = lib.dflash_paged_evict_workspace
    assert size(3, 2, 8, 0) >= 3 * 8 and size(3, 2, 8, 1) >= size(3, 2, 8, 0) + 3 * 2 * 8 * 4
    for bad in ((-1, 2, 8, 1), (3, 0, 8, 1), (3, 2, 0, 1), (1 << 23, 64, 8, 1)):
        assert size(*bad) == _abi.DFLASH_EINVAL


def test_append_refuses_a_misaligned_count_of_evicted_tokens(lib):
    from block_speculative_drafting_gb300 import _abi
    c, r, k = _cache4(), _rows_struct(), _head_struct(2)
    assert lib.dflash_paged_append_at(C.byref(c), C.byref(r), C.byref(k), C.byref(k), None, None, None, None, 1e-6, None,
                                      4098, None) == _abi.DFLASH_EINVAL


# --------------------------------------------------------------------------- the oracle's own pins
def test_oracle_rounds_as_the_types_do():
    torch = _torch()
    x = np.concatenate([np.linspace(0, 500, 4001), np.exp2(np.arange(-14, 9.0, 0.37)), [2.0 ** -10, 3 * 2.0 ** -10]])
    want = torch.from_numpy(np.minimum(x, 448)).float().to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(O.round_e4m3(x.astype(np.float32)), want)
    for v, c in ((0.2, 0), (0.25, 0), (0.26, 0.5), (0.75, 1), (1.25, 1), (1.75, 2), (2.5, 2), (2.51, 3), (3.5, 4), (5, 4),
                 (5.01, 6), (99, 6), (-0.75, -1), (-5, -4)):
        assert O.round_e2m1(v) == c
    y, s = O.quantise_e2m1([0.0] * 15 + [12.0])
    assert s == [2.0] and y[-1] == 6.0


def test_oracle_keeps_by_hand():
    w = [9, 1, 5, 5, 0, 5, 7, 2]
    assert O.kept_slots(w, 8, 8, 0, 0) == list(range(8))
    assert O.kept_slots(w, 8, 4, 0, 0) == [0, 2, 3, 6]
    assert O.kept_slots(w, 8, 4, 2, 1) == [0, 1, 6, 7]
    assert O.kept_slots(w, 7, 4, 1, 3) == [0, 4, 5, 6]
    assert O.kept_slots([0.0, float("nan"), -1.0, -0.0], 4, 2, 0, 0) == [0, 3]


# --------------------------------------------------------------------------- 4-bit caches
def _cached4(torch, rng, shape, order="slot", scale=1.0):
    """(codes, blocks, float64 values without the heads' scales)"""
    y, s = O.quantise_e2m1(scale * rng.standard_normal(shape))
    code = np.argmin(np.abs(np.abs(y)[..., None] - E2M1), -1) + 8 * (y < 0)
    codes = torch.from_numpy((code[..., 0::2] | (code[..., 1::2] << 4)).astype(np.uint8)).cuda()
    blocks = torch.from_numpy(s.astype(np.float32)).cuda().to(torch.float8_e4m3fn)
    if order == "head":  # [page][head][slot] in memory
        codes = codes.permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3)
        blocks = blocks.view(torch.uint8).permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3).view(torch.float8_e4m3fn)
    return codes, blocks, (y.reshape(*s.shape, 16) * s[..., None]).reshape(shape)


def _values4(codes, blocks):
    """float64 values of codes and blocks, without the heads' scales"""
    c = codes.cpu().numpy().astype(int)
    c = np.stack((c & 15, c >> 4), -1).reshape(*c.shape[:-1], -1)
    y = np.where(c >= 8, -1.0, 1.0) * E2M1[c & 7]
    return (y.reshape(*y.shape[:-1], -1, 16) * f64(blocks)[..., None]).reshape(y.shape)


def _raw(t):
    return t.contiguous().view(-1).cpu().numpy().copy() if t.element_size() == 1 and "float" not in str(t.dtype) else \
        t.contiguous().view(_torch().uint8).view(-1).cpu().numpy().copy()


def _check_append4(src="bf16", hd=128, heads=4, kvh=2, page=16, rows=(1, 3), lens=(5, 40), rotary=None, interleaved=False,
                   norm=False, uniform=False, bad=(), order="slot", extra=0, powers=False, evicted=None, x=None, seed=0):
    torch, dfl = _torch(), _dfl()
    rng = np.random.default_rng(seed)
    table, n_pages = _layout(torch, rng, lens, rows, page, bad=bad)
    R = sum(rows) + extra
    qkv = torch.from_numpy(rng.standard_normal((R, heads + 2 * kvh, hd)).astype(np.float32)).cuda().to(_types()[src])
    q, k, v = qkv.split((heads, kvh, kvh), 1)
    if x is not None:
        x(k, v)
    kc, kb, _ = _cached4(torch, rng, (n_pages, page, kvh, hd), order)
    vc, vb, _ = _cached4(torch, rng, (n_pages, page, kvh, hd), order)
    old = [_values4(kc, kb), _values4(vc, vb)]
    sc = [torch.from_numpy((np.exp2(-rng.integers(3, 7, kvh)) if powers else (0.5 + rng.random(kvh)) / 64)
                           .astype(np.float32)).cuda() for _ in range(2)]
    gains = [torch.from_numpy((1 + 0.1 * rng.standard_normal(hd)).astype(np.float32)).cuda() if norm else None
             for _ in range(2)]
    f = (1e4 ** (-np.arange(0, rotary, 2) / rotary)) if rotary else None
    q_out = torch.full((R, heads, hd), 7.0, device="cuda", dtype=q.dtype)
    dfl.paged_append(kc, vc, k, v, _i32(torch, table), _i32(torch, lens),
                     row_start=None if uniform else _i32(torch, _starts(rows)), q=q, q_out=q_out,
                     inv_freq=None if f is None else torch.from_numpy(f).cuda(), interleaved=interleaved,
                     q_norm=gains[0], k_norm=gains[1], k_scale=sc[0], v_scale=sc[1], k_block=kb, v_block=vb,
                     evicted=None if evicted is None else _i32(torch, evicted))
    torch.cuda.synchronize()
    gn = [None if g is None else f64(g) for g in gains]
    turned = list(lens) if evicted is None else [l + e for l, e in zip(lens, evicted)]
    starts = None if uniform else _starts(rows)
    slots, _, touched = O.paged_append(f64(k), f64(v), f64(q), table, lens, page, n_pages, starts)
    for r in range(R):
        if r not in touched:
            assert (f64(q_out)[r] == 7.0).all()  # rows of no sequence stay
    # the same rows at the positions they are rotated as, one page a row
    R_of = {(pg, sl): None for pg, sl in slots}
    for s, a, n in O.rows_of(len(lens), R, starts):
        for i in range(n):
            at = O.slot_of(table[s], page, n_pages, lens[s] - n + i)
            if at is not None:
                kk = f64(k)[a + i]
                if gn[1] is not None:
                    kk = O.rms_head(kk, gn[1], 1e-6)
                if f is not None:
                    kk = O.rotate(kk, turned[s] - n + i, f, interleaved, 1.0)
                R_of[at] = (kk, f64(v)[a + i])
    for idx, (codes, blocks) in enumerate(((kc, kb), (vc, vb))):
        got = _values4(codes, blocks)
        got_s = f64(blocks)
        want = old[idx].copy()
        for (pg, sl), kv in R_of.items():
            t = kv[idx] / f64(sc[idx])[:, None]
            g = t.reshape(kvh, -1, 16)
            if powers and f is None and not norm:
                d = np.zeros_like(g)
            elif idx == 1 or (f is None and not norm):
                d = 2.0 ** -23 * np.abs(g)
            else:
                d = np.broadcast_to(2.0 ** -20 * np.abs(t).max(-1)[:, None, None], g.shape)
            with np.errstate(all="ignore"):
                lo, hi = O.round_e4m3((np.abs(g) - d).clip(0).max(-1) / 6), O.round_e4m3((np.abs(g) + d).max(-1) / 6)
                s = got_s[pg, sl]
                assert (np.isnan(s) == np.isnan(lo)).all()
                assert (np.isnan(s) | ((s >= lo) & (s <= hi))).all(), (idx, pg, sl)
                y = got[pg, sl].reshape(g.shape) / np.where(s > 0, s, 1.0)[..., None]
                u = np.where(s[..., None] > 0, 1.0 / s[..., None], 0.0)
                e = 2.0 ** -23
                a, b = O.round_e2m1((g - d) * u * (1 - e)), O.round_e2m1((g + d) * u * (1 + e))
                a, b = np.minimum(a, O.round_e2m1((g - d) * u * (1 + e))), np.maximum(b, O.round_e2m1((g + d) * u * (1 - e)))
                ok = np.isnan(s)[..., None] | ((y >= a) & (y <= b))
            assert ok.all(), (idx, pg, sl, np.argwhere(~ok)[:4])
            want[pg, sl] = got[pg, sl]
        assert np.array_equal(got, want, equal_nan=True)  # every other slot as it was
    return kc, kb, vc, vb


@gpu
@pytest.mark.parametrize("src", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("hd", [64, 128])
def test_append4_types(src, hd):
    _check_append4(src, hd=hd, powers=True, seed=hd)
    _check_append4(src, hd=hd, rotary=hd, norm=True, seed=hd + 1)


@gpu
@pytest.mark.parametrize("rotary,interleaved", [(16, False), (64, True), (112, False), (128, True)])
def test_append4_rotations(rotary, interleaved):
    _check_append4(rotary=rotary, interleaved=interleaved, seed=3)


@gpu
@pytest.mark.parametrize("page", [1, 3, 16, 48, 64])
@pytest.mark.parametrize("order", ["slot", "head"])
def test_append4_pages(page, order):
    _check_append4("f16", hd=64, page=page, order=order, rows=(4, 0, 1, 7), lens=(4, 0, 33, 64), rotary=32, seed=page)


@gpu
def test_append4_uniform_heads_and_what_is_not_held():
    _check_append4(heads=8, kvh=1, rows=(4, 4), lens=(9, 4), uniform=True, rotary=128)
    _check_append4(heads=15, kvh=3, rows=(1,), lens=(1,), uniform=True, rotary=64)
    _check_append4(heads=40, kvh=40, hd=64, rows=(2, 1), lens=(2, 17), norm=True)
    _check_append4(rows=(4, 3, 40), lens=(2, 40, 41), bad=((1, 2), (2, 0), (2, 1), (2, 2)), rotary=64, extra=3, seed=5)
    _check_append4(rows=(1, 700), lens=(5, 800), heads=2, kvh=1, hd=64, page=64, seed=6)


@gpu
@pytest.mark.parametrize("kind", ["bf16", "e4m3", "e2m1"])
def test_append_rotates_by_the_evicted_tokens_too(kind):
    torch, dfl = _torch(), _dfl()
    if kind == "e2m1":
        _check_append4(rotary=128, rows=(2, 3, 1), lens=(5, 40, 33), evicted=(0, 1000, 7), heads=6, kvh=3, seed=1)
        return
    # the row whose slot is p and whose sequence has lost e tokens is the row of position p + e
    rng = np.random.default_rng(0)
    x = torch.from_numpy(rng.standard_normal((3, 2, 64)).astype(np.float32)).cuda()
    f = dfl.rope_inv_freq(64, 1e4)[0]
    T = _types()[kind]
    def call(lens, evicted):  # noqa: E306
        kc = torch.zeros(64, 16, 2, 64, device="cuda").to(T)
        table = torch.arange(64, dtype=torch.int32, device="cuda").view(1, 64).expand(3, 64).contiguous()
        q = dfl.paged_append(kc, kc.clone(), x, x, table, _i32(torch, lens), q=x, inv_freq=f,
                             evicted=None if evicted is None else _i32(torch, evicted))
        return q, kc.view(torch.uint8).view(64 * 16, -1)
    q1, c1 = call((10, 20, 300), (90, 0, 600))
    q2, c2 = call((100, 20, 900), None)
    assert torch.equal(q1, q2)
    for a, b in ((9, 99), (19, 19), (299, 899)):
        assert torch.equal(c1[a], c2[b])


@gpu
def test_append4_special_values():
    torch = _torch()

    def put(k, v):
        k[0, 0, :16] = 0.0                                  # a block of zeros: scale 0
        k[0, 0, 16:32] = 1e-9                               # under the smallest scale: 0
        k[0, 0, 32] = float("nan")                          # its block is NaN, the next one is not
        k[0, 1, 3] = float("inf")                           # the largest scale and code
        k[0, 1, 20] = -float("inf")
        v[0, 0, 5] = 1e30                                   # clamped to 6 * 448 of the head's scale
        v[0, 1, :16] = torch.arange(16, device="cuda") / 4  # ties

    kc, kb, vc, vb = _check_append4("f32", rows=(1,), lens=(1,), powers=True, x=put)
    y, s = _values4(kc, kb), f64(kb)
    at = np.argwhere(np.isnan(s).any((2, 3)))
    assert len(at) == 1
    pg, sl = at[0]
    assert s[pg, sl, 0, 0] == 0 and s[pg, sl, 0, 1] == 0 and (y[pg, sl, 0, :32] == 0).all()
    assert np.isnan(y[pg, sl, 0, 32:48]).all() and np.isfinite(y[pg, sl, 0, 48:]).all()
    assert y[pg, sl, 1, 3] == 6 * 448 and y[pg, sl, 1, 20] == -6 * 448 and _values4(vc, vb)[pg, sl, 0, 5] == 6 * 448


# --------------------------------------------------------------------------- read
def _any_cache(torch, rng, shape, kind, order="slot"):
    """(k_cache, k_block or None, k_scale or None, float64 values)"""
    kvh = shape[2]
    if kind == "e2m1":
        c, b, y = _cached4(torch, rng, shape, order, 16.0)
    else:
        (c, y), b = _cached(torch, rng, shape, kind, order), None
    s = None
    if kind in ("e4m3", "e2m1"):
        s = torch.from_numpy((0.5 + rng.random(kvh)).astype(np.float32) / 16).cuda()
        y = y * f64(s)[:, None]
    return c, b, s, y


@gpu
@pytest.mark.parametrize("kind", ["bf16", "f16", "e4m3", "e2m1"])
@pytest.mark.parametrize("out", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("hd,kvh,order", [(64, 3, "slot"), (128, 2, "head"), (128, 9, "slot")])
def test_read(kind, out, hd, kvh, order):
    torch, dfl = _torch(), _dfl()
    rng = np.random.default_rng(hd)
    page, lens, rows = 7, (3, 0, 40, 15), (3, 0, 17, 20)  # (the last: five rows before position 0)
    table, n_pages = _layout(torch, rng, lens, rows, page, bad=((2, 4),))
    kc, kb, ks, k64 = _any_cache(torch, rng, (n_pages, page, kvh, hd), kind, order)
    vc, vb, vs, v64 = _any_cache(torch, rng, (n_pages, page, kvh, hd), kind, order)
    R = sum(rows) + 2
    kw = dict(row_start=_i32(torch, _starts(rows)), k_scale=ks, v_scale=vs, k_block=kb, v_block=vb)
    wide = torch.full((R, 2 * kvh, hd), 7.0, device="cuda", dtype=_types()[out])  # k and v side by side, strided
    k, v = dfl.paged_read(kc, vc, _i32(torch, table), _i32(torch, lens), R, k_out=wide[:, :kvh], v_out=wide[:, kvh:], **kw)
    torch.cuda.synchronize()
    want = np.full((R, 2 * kvh, hd), 7.0)
    for s, a, n in O.rows_of(4, R, _starts(rows)):
        for i in range(n):
            at = O.slot_of(table[s], page, n_pages, lens[s] - n + i)
            want[a + i] = 0.0 if at is None else np.concatenate((k64[at], v64[at]))
    got = f64(wide)
    assert (np.abs(got - want) <= (HALF[out] + 2.0 ** -23) * np.abs(want) + TINY[out]).all()
    assert (got[R - 2:] == 7.0).all()
    k2, v2 = dfl.paged_read(kc, vc, _i32(torch, table), _i32(torch, lens), R, dtype=_types()[out], **kw)
    assert torch.equal(k2[:R - 2], k[:R - 2]) and torch.equal(v2[:R - 2], v[:R - 2])


@gpu
def test_read_gives_back_what_append_was_given():
    """4-bit values whose blocks hold a code of 6 are the same codes when written again: whole caches, read with row_start
    the sum of the lengths."""
    torch, dfl = _torch(), _dfl()
    rng = np.random.default_rng(4)
    lens, page = (40, 3), 16
    table, n_pages = _layout(torch, rng, lens, lens, page)
    kc, kb, _ = _cached4(torch, rng, (n_pages, page, 2, 64), scale=16.0)
    kc[..., ::8] |= 7  # a block's first column: 6 or -6
    args = (_i32(torch, table), _i32(torch, lens))
    kw = dict(row_start=_i32(torch, _starts(lens)))
    k, v = dfl.paged_read(kc, kc, *args, 43, k_block=kb, v_block=kb, dtype=torch.float32, **kw)
    assert torch.equal(k, v)
    c2, b2 = (torch.zeros_like(kc) for _ in range(2)), (torch.zeros_like(kb) for _ in range(2))
    (c2, c3), (b2, b3) = c2, b2
    dfl.paged_append(c2, c3, k, v, *args, k_block=b2, v_block=b3, **kw)
    old, new = _values4(kc, kb), _values4(c2, b2)
    for s, l in enumerate(lens):
        for p in range(l):
            at = O.slot_of(table[s], page, n_pages, p)
            assert np.array_equal(old[at], new[at])
            assert np.array_equal(f64(kb)[at], f64(b2)[at])
    assert torch.equal(c2, c3)


# --------------------------------------------------------------------------- attention
def _check_attention4(src="bf16", hd=128, heads=4, kvh=2, page=16, rows=(1,), lens=(40,), window=0, uniform=False, bad=(),
                      order="slot", extra=0, scale=None, seed=0, poison=None, spread=1.0, amp=16.0):
    torch, dfl = _torch(), _dfl()
    rng = np.random.default_rng(seed)
    table, n_pages = _layout(torch, rng, [max(l, 0) for l in lens], rows, page, bad=bad)
    R = sum(rows) + extra
    q = torch.from_numpy(spread * rng.standard_normal((R, heads, hd)).astype(np.float32)).cuda().to(_types()[src])
    kc, kb, _ = _cached4(torch, rng, (n_pages, page, kvh, hd), order, amp)
    vc, vb, _ = _cached4(torch, rng, (n_pages, page, kvh, hd), order, amp)
    if poison is not None:
        poison(torch, kb, vb, table)
    ks, vs = (torch.from_numpy((0.5 + rng.random(kvh)).astype(np.float32) / 16).cuda() for _ in range(2))
    k64, v64 = _values4(kc, kb) * f64(ks)[:, None], _values4(vc, vb) * f64(vs)[:, None]
    out = torch.full((R, heads, hd), 7.0, device="cuda", dtype=q.dtype)
    lse = torch.full((R, heads), 7.0, device="cuda")
    start = None if uniform else _i32(torch, _starts(rows))
    dfl.paged_attention(q, kc, vc, _i32(torch, table), _i32(torch, lens), row_start=start, scale=scale, window=window,
                        k_scale=ks, v_scale=vs, k_block=kb, v_block=vb, out=out, lse=lse)
    torch.cuda.synchronize()
    ref, rl, mag, touched = O.paged_attention(f64(q), k64, v64, table, lens, None if uniform else _starts(rows), scale,
                                              window)
    got, gl = f64(out), f64(lse)
    for r in range(R):
        if r not in touched:
            assert (got[r] == 7.0).all() and (gl[r] == 7.0).all()
    t = np.array(touched, dtype=int)
    if not len(t):
        return
    got, gl, ref, rl, mag = got[t], gl[t], ref[t], rl[t], mag[t]
    norm = lambda x: np.linalg.norm(np.where(np.isfinite(x), x, 0.0), axis=-1).max()  # noqa: E731
    s_err = hd * 2.0 ** -24 * (hd ** -0.5 if scale is None else scale) * norm(f64(q)) * norm(k64) + 2.0 ** -20
    p_err = s_err + (HALF["f16"] if src == "bf16" else 0.0)
    with np.errstate(all="ignore"):
        small = max(max(lens), 1) * 2.0 ** -32 * np.abs(np.where(np.isfinite(v64), v64, 0.0)).max()
        tol = HALF[src] * np.abs(ref) + TINY[src] + 2 * p_err * mag + small
        fine = np.isfinite(ref)
        assert np.array_equal(fine, np.isfinite(got)), "finite where the definition is"
        d = np.abs(got - ref)[fine]
        assert (d <= tol[fine]).all(), float((d / np.maximum(tol[fine], 1e-30)).max())
    assert np.array_equal(np.isneginf(rl), np.isneginf(gl)) and np.array_equal(np.isnan(rl), np.isnan(gl))
    ok = np.isfinite(rl)
    assert (np.abs(gl[ok] - rl[ok]) <= s_err + 2.0 ** -21 * np.abs(rl[ok])).all()


@gpu
@pytest.mark.parametrize("src", ["bf16", "f16"])
@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("group,rows", [(1, 1), (4, 1), (8, 1), (3, 3), (3, 5), (4, 4), (4, 5), (5, 8), (8, 16), (4, 40)])
def test_attention4_types_and_tiles(src, hd, group, rows):
    _check_attention4(src, hd=hd, heads=2 * group, kvh=2, rows=(rows, 1), lens=(rows + 300, 130), seed=group + rows)


@gpu
@pytest.mark.parametrize("page", [1, 3, 16, 48, 128, 1000])
@pytest.mark.parametrize("order", ["slot", "head"])
@pytest.mark.parametrize("rows", [2, 9])
def test_attention4_pages(page, order, rows):
    _check_attention4(page=page, order=order, rows=(rows, 1, rows), lens=(700, 17, 250), seed=page)


@gpu
@pytest.mark.parametrize("length", [0, 1, 2, 15, 16, 17, 31, 32, 33, 127, 128, 129, 255, 256, 257, 1000])
def test_attention4_lengths(length):
    _check_attention4("f16", rows=(1, 2), lens=(length, length + 2), seed=length)
    _check_attention4(rows=(12,), lens=(length + 3,), seed=length)  # (rows before position 0 at the shortest)


@gpu
@pytest.mark.parametrize("window", [1, 7, 16, 100, 5000])
@pytest.mark.parametrize("rows", [1, 3, 6, 33])
def test_attention4_windows(window, rows):
    _check_attention4(rows=(rows, 1), lens=(400, 90), window=window, seed=window)


@gpu
def test_attention4_ragged_padded_and_bad_pages():
    for heads in (4, 40):
        _check_attention4(heads=heads, rows=(3, 0, 1, 5), lens=(70, 9, 1, 300), extra=4,
                          bad=((0, 1), (3, 0), (3, 7), (3, 8)), seed=1)
    _check_attention4(rows=(2, 2), lens=(30, 50), uniform=True)
    _check_attention4("f16", rows=(1,), lens=(9000,), heads=2, kvh=1, page=64, hd=64)
    _check_attention4(rows=(2, 1, 1), lens=(3000, 10, 4100), heads=8, kvh=2, page=32)
    _check_attention4(rows=(16,), lens=(5000,), heads=4, kvh=1, page=128)
    _check_attention4(heads=3, kvh=1, rows=(1,) * 9, lens=(5, 900, 33, 64, 1, 0, 1200, 65, 31), seed=2)


@gpu
@pytest.mark.parametrize("src,hd,heads,kvh,rows,window", [("bf16", 128, 32, 8, 1, 0), ("f16", 64, 16, 8, 1, 0),
                                                          ("bf16", 128, 12, 12, 2, 0), ("bf16", 64, 12, 6, 4, 0),
                                                          ("bf16", 128, 32, 8, 3, 0), ("f16", 128, 12, 4, 5, 0),
                                                          ("bf16", 128, 16, 8, 2, 90)])
def test_attention4_heads_together(src, hd, heads, kvh, rows, window):
    """Units enough for the heads of a key to go together, over more sequences than a warp looks at in one go."""
    rng = np.random.default_rng(heads + rows)
    n = 45 if kvh >= 6 else 60
    r = tuple(int(x) for x in rng.integers(0, rows + 1, n - 3)) + (rows,) * 3
    lens = tuple(int(x) for x in rng.integers(1, 700, n - 3)) + (0, 2900, 33)
    _check_attention4(src, hd=hd, heads=heads, kvh=kvh, rows=r, lens=lens, window=window, page=48, bad=((1, 0), (4, 1)),
                      seed=rows)


@gpu
def test_attention4_large_scores():
    _check_attention4(rows=(3,), lens=(500,), spread=20.0, scale=0.5)
    _check_attention4("f16", rows=(9,), lens=(500,), spread=20.0, scale=0.5)
    _check_attention4(rows=(3,), lens=(500,), spread=1e6, scale=1e-6)
    # the largest scales that a block can have, and queries at the ends of bf16
    _check_attention4(rows=(2,), lens=(100,), amp=2000.0, spread=1e30, scale=1e-30)
    _check_attention4(rows=(7,), lens=(100,), amp=2000.0, spread=1e-30, scale=1e25)


@gpu
@pytest.mark.parametrize("src", ["bf16", "f16"])
@pytest.mark.parametrize("hd,heads,kvh,rows", [(128, 4, 2, (2, 4)), (64, 16, 2, (1, 9)), (128, 2, 2, (3, 3)),
                                               (128, 32, 2, (3, 9)), (64, 6, 2, (1, 2))])
def test_attention4_keeps_what_rows_may_not_see_out(src, hd, heads, kvh, rows):
    """Block scales of NaN: at every slot of no row's view, at positions that only later rows see, at a window's edge."""
    lens, page = (5, 130), 16

    def free(torch, kb, vb, table):
        used = np.zeros((kb.shape[0], page), bool)
        for s, l in enumerate(lens):
            for p in range(free.lo[s], l):
                used[table[s][p // page], p % page] = True
        for b in (kb, vb):
            b.view(torch.uint8)[torch.from_numpy(~used).cuda()] = 0x7f
        free.more(torch, kb.view(torch.uint8), vb.view(torch.uint8), table)

    def later(torch, kb, vb, table):
        at = int(table[1][129 // 16]), 129 % 16
        vb[at][0, ::3] = 0xff
        vb[at][1, 1] = 0x7f
        kb[at][1, 2] = 0x7f

    kw = dict(hd=hd, heads=heads, kvh=kvh, rows=rows, lens=lens)
    free.lo, free.more = (0, 0), lambda *a: None
    _check_attention4(src, poison=free, **kw)
    free.more = later
    _check_attention4(src, poison=free, **kw)
    free.lo = (0, 100)
    free.more = lambda torch, kb, vb, table: vb[int(table[1][101 // 16]), 101 % 16].fill_(0x7f)
    _check_attention4(src, window=31 - rows[1], poison=free, **kw)


@gpu
def test_attention4_codes_in_torchs_own_type_and_in_place():
    torch, dfl = _torch(), _dfl()
    rng = np.random.default_rng(0)
    kc, kb, _ = _cached4(torch, rng, (6, 16, 2, 64))
    q = torch.from_numpy(rng.standard_normal((3, 4, 64)).astype(np.float32)).cuda().to(torch.bfloat16)
    args = (_i32(torch, [[0, 1, 2, 3, 4, 5]]), _i32(torch, [90]))
    kw = dict(k_block=kb, v_block=kb)
    a = dfl.paged_attention(q, kc, kc, *args, **kw)
    c = kc.view(torch.float4_e2m1fn_x2)
    ws = torch.empty(dfl.paged_attention_workspace(q, c, 1), dtype=torch.uint8, device="cuda")
    b = dfl.paged_attention(q, c, c, *args, workspace=ws, **kw)
    assert torch.equal(a, b)
    assert dfl.paged_attention(q, kc, kc, *args, out=q, **kw) is q and torch.equal(a, q)


@gpu
def test_attention4_repeats_bit_for_bit_on_streams_and_threads():
    torch, dfl = _torch(), _dfl()
    rng = np.random.default_rng(0)
    lens = (900, 33, 4000, 7)
    table, n_pages = _layout(torch, rng, lens, (1, 1, 1, 1), 16)
    kc, kb, _ = _cached4(torch, rng, (n_pages, 16, 2, 128))
    table, lens = _i32(torch, table), _i32(torch, lens)
    for rows in (1, 9):
        q = torch.from_numpy(rng.standard_normal((4 * rows, 8, 128)).astype(np.float32)).cuda().to(torch.bfloat16)
        call = lambda **kw: dfl.paged_attention(q, kc, kc, table, lens, k_block=kb, v_block=kb, **kw)  # noqa: E731
        want = call()
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream() for _ in range(3)]
        outs = []
        for i in range(12):
            with torch.cuda.stream(streams[i % 3]):
                outs.append(call())
        outs.append(call(stream=streams[0].cuda_stream))
        torch.cuda.synchronize()
        assert all(torch.equal(o, want) for o in outs)


# --------------------------------------------------------------------------- key weights
def _check_weights(kind="bf16", src=None, hd=128, heads=4, kvh=2, page=16, rows=(1,), lens=(40,), window=0, uniform=False,
                   bad=(), order="slot", extra=0, scale=None, seed=0, spread=1.0, poison=None, lse=None, wide=5):
    torch, dfl = _torch(), _dfl()
    rng = np.random.default_rng(seed)
    src = src or (kind if kind in ("bf16", "f16") else "bf16")
    table, n_pages = _layout(torch, rng, [max(l, 0) for l in lens], rows, page, bad=bad)
    R = sum(rows) + extra
    q = torch.from_numpy(spread * rng.standard_normal((R, heads, hd)).astype(np.float32)).cuda().to(_types()[src])
    kc, kb, ks, k64 = _any_cache(torch, rng, (n_pages, page, kvh, hd), kind, order)
    if poison is not None:
        k64 = poison(torch, kc, kb, table, k64)
    starts = None if uniform else _starts(rows)
    with np.errstate(all="ignore"):
        _, l64, _, _ = O.paged_attention(f64(q), k64, np.zeros_like(k64), table, lens, starts, scale, window)
    ls = torch.from_numpy(l64.astype(np.float32)).cuda()
    if lse is not None:
        lse(ls)
    w0 = torch.from_numpy(rng.random((len(lens), kvh, table.shape[1] * page + wide)).astype(np.float32)).cuda()
    w = w0.clone()
    got = dfl.paged_key_weights(w, q, kc, _i32(torch, table), _i32(torch, lens), ls,
                                row_start=None if uniform else _i32(torch, starts), scale=scale, window=window, k_scale=ks,
                                k_block=kb)
    torch.cuda.synchronize()
    assert got is w
    want, amp = O.paged_key_weights(f64(w0), f64(q), f64(ls), k64, table, lens, starts, scale, window)
    terms = -(-R // len(lens)) * (heads // kvh) * len(lens)
    g = f64(w)
    with np.errstate(all="ignore"):
        # the score, the exponential's argument (|s - lse| in 32 bits) and the sums
        tol = hd * 2.0 ** -23 * amp + (2.0 ** -19 + terms * 2.0 ** -24) * np.abs(want)
        assert np.array_equal(np.isnan(want), np.isnan(g))
        ok = ~np.isnan(want)
        assert (np.abs(g - want)[ok] <= tol[ok] + 1e-37).all(), float((np.abs(g - want)[ok] / (tol[ok] + 1e-37)).max())
    for s, a, n in O.rows_of(len(lens), R, starts):  # what the call does not reach stays
        L = min(max(lens[s], 0), table.shape[1] * page) if n else 0
        assert np.array_equal(g[s, :, L:], f64(w0)[s, :, L:])
    return w


@gpu
@pytest.mark.parametrize("kind,src", [("bf16", "bf16"), ("f16", "f16"), ("e4m3", "bf16"), ("e4m3", "f16"),
                                      ("e2m1", "bf16"), ("e2m1", "f16")])
@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("group,rows", [(1, 1), (4, 1), (3, 5), (8, 16)])
def test_weights_types_and_tiles(kind, src, hd, group, rows):
    _check_weights(kind, src, hd=hd, heads=2 * group, kvh=2, rows=(rows, 1), lens=(rows + 150, 130), seed=group + rows)


@gpu
@pytest.mark.parametrize("page", [1, 3, 16, 48, 128, 1000])
@pytest.mark.parametrize("order", ["slot", "head"])
def test_weights_pages(page, order):
    _check_weights("e2m1", page=page, order=order, rows=(2, 1, 3), lens=(300, 17, 130), seed=page)


@gpu
@pytest.mark.parametrize("length", [0, 1, 2, 15, 16, 17, 127, 128, 129, 400])
def test_weights_lengths(length):
    _check_weights(rows=(1, 2), lens=(length, length + 2), seed=length)
    _check_weights("e4m3", rows=(7,), lens=(length + 3,), seed=length)


@gpu
@pytest.mark.parametrize("kind,hd", [("bf16", 128), ("e4m3", 64), ("e2m1", 128)])
@pytest.mark.parametrize("rows", [9, 18, 34])
def test_weights_many_short_sequences(kind, hd, rows):
    """Shares of many heads, some of one tile of keys: the warps with a pair's second tile then skip it, and must not
    take what they wait for next for done."""
    rng = np.random.default_rng(rows)
    r = rng.integers(rows - 1, rows + 1, 50)
    lens = [int(a + rng.integers(0, 60) if rng.random() < 0.4 else a + rng.integers(0, 330)) for a in r]
    _check_weights(kind, hd=hd, heads=64, kvh=8, rows=tuple(int(x) for x in r), lens=tuple(lens), page=64, seed=rows)


@gpu
@pytest.mark.parametrize("window", [1, 7, 16, 100, 5000])
@pytest.mark.parametrize("rows", [1, 6, 33])
def test_weights_windows(window, rows):
    _check_weights("f16", rows=(rows, 1), lens=(200, 90), heads=2, kvh=1, window=window, seed=window)


@gpu
def test_weights_ragged_padded_and_bad_pages():
    _check_weights(rows=(3, 0, 1, 5), lens=(70, 9, 1, 200), extra=4, bad=((0, 1), (3, 0), (3, 7), (3, 8)), seed=1)
    _check_weights("e2m1", rows=(2, 2), lens=(30, 50), uniform=True)
    _check_weights("f16", heads=40, kvh=1, hd=64, rows=(4, 30), lens=(30, 150))
    _check_weights("bf16", heads=2, kvh=1, hd=64, rows=(130, 300), lens=(140, 300), page=64)
    _check_weights("e2m1", heads=12, kvh=1, rows=(40,), lens=(300,), page=64)


@gpu
def test_weights_large_scores_and_rows_that_see_nothing():
    _check_weights(rows=(3,), lens=(200,), spread=20.0, scale=0.5)
    _check_weights("e2m1", rows=(3,), lens=(200,), spread=1e6, scale=1e-6)

    def nothing(lse):
        lse[1] = float("-inf")

    def keys(torch, kc, kb, table, k64):  # keys that only the last row sees: NaN for all of its sum alone
        p = 129
        at = int(table[0][p // 16]), p % 16
        kc[at][1, 5] = float("nan")
        k64 = k64.copy()
        k64[at][1, 5] = np.nan
        return k64

    _check_weights(rows=(4,), lens=(130,), lse=nothing)
    _check_weights(rows=(4,), lens=(130,), poison=keys)


@gpu
def test_weights_repeat_bit_for_bit_and_in_strided_buffers():
    torch, dfl = _torch(), _dfl()
    rng = np.random.default_rng(0)
    table, n_pages = _layout(torch, rng, (3000, 70), (4, 4), 16)
    kc, kb, ks, _ = _any_cache(torch, rng, (n_pages, 16, 2, 128), "e2m1")
    q = torch.from_numpy(rng.standard_normal((8, 8, 128)).astype(np.float32)).cuda().to(torch.bfloat16)
    table, lens = _i32(torch, table), _i32(torch, (3000, 70))
    lse = torch.empty(8, 8, device="cuda")
    dfl.paged_attention(q, kc, kc, table, lens, k_block=kb, v_block=kb, k_scale=ks, v_scale=ks, lse=lse)
    P = table.shape[1] * 16
    call = lambda w, **kw: dfl.paged_key_weights(w, q, kc, table, lens, lse, k_scale=ks, k_block=kb, **kw)  # noqa: E731
    want = call(torch.zeros(2, 2, P, device="cuda"))
    # every row of a head's queries hands out a weight of 1
    per = want.sum(-1)
    assert (per - 16).abs().max() < 16 * 2.0 ** -18
    big = torch.zeros(2, 3, P + 7, device="cuda")
    for _ in range(2):
        w = torch.zeros(2, 3, P + 7, device="cuda")
        assert torch.equal(call(w[:, 1:, 3:P + 3])[..., :P], want) and (w[:, 0] == 0).all()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = call(big[:, :2, :P], stream=s.cuda_stream)
    s.synchronize()
    assert torch.equal(got, want)


# --------------------------------------------------------------------------- evict
def _check_evict(kind="bf16", hd=128, kvh=2, page=16, lens=(40,), keep=16, first=0, recent=0, bad=(), order="slot", seed=0,
                 weights=None, aside=False, given=True):
    torch, dfl = _torch(), _dfl()
    rng = np.random.default_rng(seed)
    n = len(lens)
    table, n_pages = _layout(torch, rng, [max(l, 0) for l in lens], [1] * n, page, bad=bad)
    cap = table.shape[1] * page
    caches = []
    for _ in range(2):
        c, b, _, _ = _any_cache(torch, rng, (n_pages, page, kvh, hd), kind, order)
        caches += [c] if b is None else [c, b]
    w = rng.standard_normal((n, kvh, cap + 3)).astype(np.float32)
    w = np.round(w * 8) / 8  # (many equal ones)
    if weights is not None:
        weights(w)
    w = w.astype(np.float32)
    W = torch.from_numpy(w.copy()).cuda()
    out = torch.full_like(W, 7.0) if aside else None
    kept = torch.full((n, kvh, keep), 9, dtype=torch.int32, device="cuda") if given else None
    evicted = torch.arange(n, dtype=torch.int32, device="cuda") if given else None
    old = [f64(c.view(torch.uint8) if c.element_size() == 1 else c) for c in caches]
    four = len(caches) == 4
    L = _i32(torch, lens)
    new = dfl.paged_evict(caches[0], caches[2 if four else 1], W, _i32(torch, table), L, keep, first=first, recent=recent,
                          k_block=caches[1] if four else None, v_block=caches[3] if four else None, weights_out=out,
                          kept=kept, evicted=evicted)
    torch.cuda.synchronize()
    want = [x.copy() for x in old]
    want_w = np.full_like(w, 7.0) if aside else w.copy()
    for s in range(n):
        length = min(max(lens[s], 0), cap)
        assert new[s].item() == min(length, keep) and L[s].item() == lens[s]
        if given:
            assert evicted[s].item() == s + length - min(length, keep)
        for h in range(kvh):
            slots = O.kept_slots(w[s, h], length, keep, first, recent)
            if given:
                assert kept[s, h].tolist() == slots + [-1] * (keep - len(slots))
            want_w[s, h, :len(slots)] = w[s, h, slots]
            for i, j in enumerate(slots):
                a, b = O.slot_of(table[s], page, n_pages, i), O.slot_of(table[s], page, n_pages, j)
                if a is not None and b is not None:
                    for x, y in zip(want, old):
                        x[a][h] = y[b][h]
    for c, x in zip(caches, want):
        assert np.array_equal(f64(c.view(torch.uint8) if c.element_size() == 1 else c), x)
    assert np.array_equal(f64(W if out is None else out), want_w.astype(np.float64), equal_nan=True)
    if aside:
        assert np.array_equal(f64(W), w.astype(np.float64), equal_nan=True)


@gpu
@pytest.mark.parametrize("kind", ["bf16", "f16", "e4m3", "e2m1"])
@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("aside", [False, True])
def test_evict_types(kind, hd, aside):
    _check_evict(kind, hd=hd, lens=(40, 16, 17, 300, 0), keep=16, first=2, recent=5, aside=aside)


@gpu
@pytest.mark.parametrize("page", [1, 3, 16, 48, 1000])
@pytest.mark.parametrize("order", ["slot", "head"])
def test_evict_pages(page, order):
    _check_evict("e2m1", page=page, order=order, lens=(300, 17, 130), keep=33, first=1, recent=8, seed=page)


@gpu
@pytest.mark.parametrize("keep,first,recent", [(1, 0, 0), (1, 1, 0), (1, 0, 1), (7, 3, 4), (64, 0, 64), (64, 64, 0),
                                               (63, 0, 0), (199, 4, 100), (200, 5, 5), (300, 0, 0)])
def test_evict_budgets(keep, first, recent):
    _check_evict(lens=(200, 65, 64, 1), keep=keep, first=first, recent=recent, given=keep % 2 == 0)


@gpu
def test_evict_long_heads_and_bad_pages():
    _check_evict(lens=(9001,), keep=4500, kvh=1, hd=64, recent=64, page=64)
    _check_evict("e4m3", lens=(5000, 4097), keep=2050, kvh=1, hd=64, first=4, page=64)
    _check_evict("e2m1", lens=(30,) * 40, keep=20, kvh=9, hd=64, given=False)
    _check_evict(lens=(100, 90), keep=40, bad=((0, 0), (0, 5), (1, 3)), seed=3)
    _check_evict(lens=(-5, 10 ** 6, 2 ** 31 - 1)[:1], keep=4)


@gpu
def test_evict_lengths_past_the_table():
    torch, dfl = _torch(), _dfl()
    c = torch.arange(4 * 16 * 64, device="cuda").view(4, 16, 1, 64).to(torch.bfloat16)
    w = torch.zeros(2, 1, 32, device="cuda")
    w[:, :, 20] = 1.0
    kept = torch.zeros(2, 1, 3, dtype=torch.int32, device="cuda")
    lens = _i32(torch, (2 ** 31 - 1, -2 ** 31))
    assert dfl.paged_evict(c, c.clone(), w, _i32(torch, [[0, 1], [2, 3]]), lens, 3, kept=kept, new_len=lens) is lens
    assert lens.tolist() == [3, 0] and kept.tolist() == [[[0, 1, 20]], [[-1, -1, -1]]]


@gpu
def test_evict_special_weights():
    def put(w):
        w[0, 0, :40] = np.nan
        w[0, 0, 7] = -np.inf
        w[0, 1, :40] = 0.0
        w[0, 1, ::2] = -0.0
        w[1, 0, :40] = np.inf
        w[1, 1, :40] = np.float32(1e-45)
        w[1, 1, 9] = 3.4e38
        w[1, 1, 11] = -3.4e38

    for keep in (1, 5, 39):
        _check_evict(lens=(40, 40), keep=keep, weights=put)


@gpu
@pytest.mark.parametrize("spread", ["equal", "wide", "near"])
def test_evict_finds_the_border_at_any_digit(spread):
    """Weights all alike, over all exponents, and apart in their last bits: ties to the lowest position."""
    rng = np.random.default_rng(7)

    def put(w):
        if spread == "equal":
            w[:] = 0.25
        elif spread == "wide":
            w[:] = np.exp2(rng.uniform(-120, 120, w.shape)) * rng.choice([-1, 1], w.shape)
        else:
            w[:] = (np.float32(1.0).view(np.int32) + rng.integers(0, 600, w.shape)).astype(np.int32).view(np.float32)

    _check_evict(lens=(3000, 1500), keep=700, kvh=2, hd=64, weights=put, recent=3)


# --------------------------------------------------------------------------- refusals and odd calls through Python
def _good(torch):
    z = lambda *s, dtype=torch.bfloat16: torch.zeros(*s, dtype=dtype, device="cuda")  # noqa: E731
    e = torch.float8_e4m3fn
    i32 = lambda x: _i32(torch, x)  # noqa: E731
    cache = dict(k_cache=z(6, 16, 2, 32, dtype=torch.uint8), v_cache=z(6, 16, 2, 32, dtype=torch.uint8),
                 k_block=torch.zeros(6, 16, 2, 4, device="cuda").to(e), v_block=torch.zeros(6, 16, 2, 4, device="cuda").to(e))
    rows = dict(table=i32([[0, 1], [2, 3]]), kv_len=i32([20, 30]))
    append = dict(cache, **rows, k=z(4, 2, 64), v=z(4, 2, 64), row_start=i32([0, 2, 4]), evicted=i32([0, 3]))
    read = dict(cache, **rows, rows=4, row_start=i32([0, 2, 4]), k_out=z(4, 2, 64), v_out=z(4, 2, 64), dtype=torch.bfloat16)
    attention = dict(cache, **rows, q=z(4, 4, 64), row_start=i32([0, 2, 4]), out=z(4, 4, 64))
    weights = dict(rows, weights=z(2, 2, 32, dtype=torch.float32), q=z(4, 4, 64), k_cache=cache["k_cache"],
                   k_block=cache["k_block"], lse=z(4, 4, dtype=torch.float32), row_start=i32([0, 2, 4]))
    evict = dict(cache, **rows, weights=z(2, 2, 32, dtype=torch.float32), keep=8, first=2, recent=2,
                 weights_out=z(2, 2, 32, dtype=torch.float32), new_len=i32([0, 0]), kept=z(2, 2, 8, dtype=torch.int32),
                 evicted=i32([0, 0]), workspace=z(1 << 16, dtype=torch.uint8))
    return dict(paged_append=append, paged_read=read, paged_attention=attention, paged_key_weights=weights, paged_evict=evict)


_WIDE = lambda x: x.new_zeros(*x.shape[:-1], 2 * x.shape[-1])[..., ::2]  # noqa: E731  (columns two apart)
REFUSALS = [
    ("paged_append", dict(k_block=None), "needs k_block"),
    ("paged_append", dict(v_block=None), "needs v_block"),
    ("paged_append", dict(k_block=lambda x: x.float()), "k_block has to be"),
    ("paged_append", dict(k_block=lambda x: x[:, :8]), "k_block has to be"),
    ("paged_append", dict(v_block=lambda x: x[:, :, :, :2]), "v_block has to be"),
    ("paged_append", dict(v_block=lambda x: x.cpu()), "v_block is not on the call's CUDA device"),
    ("paged_append", dict(v_block=lambda x: x[:1].expand_as(x)), "v_block is written"),
    ("paged_append", dict(k_block=lambda x: x.view(x.dtype).reshape(-1)[:1].expand(6, 16, 2, 4)), "k_block has to be"),
    ("paged_append", dict(k_cache=lambda x: x.new_zeros(6, 16, 2, 32, dtype=__import__("torch").bfloat16)), "of one type"),
    ("paged_append", dict(k_cache=lambda x: x.new_zeros(6, 16, 2, 40)[..., :32]), "cache strides"),
    ("paged_append", dict(k_cache=lambda x: x[..., :16], v_cache=lambda x: x[..., :16], k_block=lambda x: x[..., :2],
                          v_block=lambda x: x[..., :2], k=lambda x: x[..., :32], v=lambda x: x[..., :32]), "head_dim 32"),
    ("paged_append", dict(evicted=lambda x: x[:1]), "evicted has to be"),
    ("paged_append", dict(evicted=lambda x: x.long()), "evicted has to be"),
    ("paged_read", dict(k_block=None), "needs k_block"),
    ("paged_read", dict(rows=lambda x: -1), "rows -1"),
    ("paged_read", dict(rows=lambda x: 1 << 24), "rows 16777216"),
    ("paged_read", dict(k_out=lambda x: x[:3]), "k_out has to be"),
    ("paged_read", dict(v_out=lambda x: x[:, :1]), "v_out has 1 heads"),
    ("paged_read", dict(v_out=lambda x: x.half()), "v_out is not of the dtype"),
    ("paged_read", dict(k_out=lambda x: x[:1].expand_as(x)), "k_out is written"),
    ("paged_read", dict(dtype=lambda x: __import__("torch").float64, k_out=None, v_out=None), "dtype is not"),
    ("paged_read", dict(table=lambda x: x.long()), "table has to be int32"),
    ("paged_attention", dict(k_block=None), "needs k_block"),
    ("paged_attention", dict(v_block=lambda x: x.transpose(0, 1)), "v_block has to be"),
    ("paged_attention", dict(q=lambda x: x.float(), out=None), "need the cache's type"),
    ("paged_key_weights", dict(weights=lambda x: x.double()), "weights has to be"),
    ("paged_key_weights", dict(weights=lambda x: x[..., :31]), "weights of 31 positions, the table names 32"),
    ("paged_key_weights", dict(weights=lambda x: x[:, :1]), "weights has to be"),
    ("paged_key_weights", dict(weights=lambda x: x[:1]), "weights has to be"),
    ("paged_key_weights", dict(weights=_WIDE), "weights has to be"),
    ("paged_key_weights", dict(weights=lambda x: x[:, :1].expand(2, 2, 32)), "weights is written"),
    ("paged_key_weights", dict(weights=lambda x: x.cpu()), "weights is not on the call's CUDA device"),
    ("paged_key_weights", dict(lse=lambda x: x[:3]), "lse has to be"),
    ("paged_key_weights", dict(lse=lambda x: x.t()), "lse has to be"),
    ("paged_key_weights", dict(k_block=None), "needs k_block"),
    ("paged_key_weights", dict(k_cache=lambda x: x.new_zeros(6, 16, 2, 64).bfloat16()), "block scales need"),
    ("paged_key_weights", dict(q=lambda x: x.float()), "q needs the cache's type"),
    ("paged_key_weights", dict(q=lambda x: x[:, :3], lse=lambda x: x[:, :3].contiguous()), "q has 3 heads"),
    ("paged_key_weights", dict(k_scale=lambda x: __import__("torch").ones(3, device="cuda")), "k_scale has to be"),
    ("paged_key_weights", dict(window=lambda x: -1), "window -1"),
    ("paged_key_weights", dict(scale=lambda x: 0.0), "scale 0"),
    ("paged_evict", dict(keep=lambda x: 0, kept=None), "keep 0"),
    ("paged_evict", dict(keep=lambda x: 3, kept=None), "keep 3, first 2, recent 2"),
    ("paged_evict", dict(first=lambda x: -1), "first -1"),
    ("paged_evict", dict(recent=lambda x: 1 << 40), "recent"),
    ("paged_evict", dict(v_block=None), "needs v_block"),
    ("paged_evict", dict(weights=lambda x: x[..., :31]), "weights of 31 positions"),
    ("paged_evict", dict(weights_out=lambda x: x[..., :31]), "out of 31 positions"),
    ("paged_evict", dict(weights_out=lambda x: x[:1].expand_as(x)), "weights_out is written"),
    ("paged_evict", dict(weights_out=None, weights=lambda x: x[:1].expand_as(x)), "weights is written"),
    ("paged_evict", dict(new_len=lambda x: x[:1]), "new_len has to be"),
    ("paged_evict", dict(new_len=lambda x: x.long()), "new_len has to be"),
    ("paged_evict", dict(kept=lambda x: x[..., :7]), "kept has to be"),
    ("paged_evict", dict(kept=lambda x: x.transpose(0, 1)), "kept has to be"),
    ("paged_evict", dict(evicted=lambda x: x[:1]), "evicted has to be"),
    ("paged_evict", dict(kv_len=None), "kv_len is None"),
    ("paged_evict", dict(k_cache=lambda x: x[:1].expand_as(x)), "k_cache is written"),
    ("paged_evict", dict(workspace=lambda x: x[:8]), "workspace of 8 bytes"),
    ("paged_evict", dict(workspace=lambda x: x[8:]), "not 16-byte aligned"),
]
CALLS = ["paged_append", "paged_read", "paged_attention", "paged_key_weights", "paged_evict"]


@gpu
@pytest.mark.parametrize("name", CALLS)
def test_calls_one_change_from_the_refused_ones_are_served(name):
    torch, dfl = _torch(), _dfl()
    getattr(dfl, name)(**_good(torch)[name])
    torch.cuda.synchronize()


@gpu
@pytest.mark.parametrize("name,changes,message", REFUSALS, ids=[f"{i}-{r[0]}-{r[2][:24]}" for i, r in enumerate(REFUSALS)])
def test_calls_refused_for_one_thing(name, changes, message):
    """Each by its own check and in its words, and nothing is launched or written."""
    torch, dfl = _torch(), _dfl()
    args = _good(torch)[name]
    tensors = [k for k, v in args.items() if isinstance(v, torch.Tensor) and k != "workspace"]
    before = {k: _raw(args[k]) for k in tensors}
    call = dict(args)
    for key, how in changes.items():
        call[key] = None if how is None else how(args.get(key))
    with pytest.raises(dfl.DFlashError) as e:
        getattr(dfl, name)(**call)
    assert message in str(e.value) and e.value.code in (dfl._abi.DFLASH_EINVAL, dfl._abi.DFLASH_EGEOM, dfl._abi.DFLASH_ECAPACITY)
    torch.cuda.synchronize()
    assert all(np.array_equal(_raw(args[k]), before[k]) for k in tensors)


@gpu
@pytest.mark.parametrize("name", CALLS)
def test_calls_without_rows_or_sequences(name):
    torch, dfl = _torch(), _dfl()
    args = _good(torch)[name]
    empty = {"table": lambda x: x[:0], "kv_len": lambda x: x[:0], "row_start": lambda x: x[:1] * 0, "k": lambda x: x[:0],
             "v": lambda x: x[:0], "q": lambda x: x[:0], "lse": lambda x: x[:0], "out": lambda x: x[:0],
             "k_out": lambda x: x[:0], "v_out": lambda x: x[:0], "weights": lambda x: x[:0], "weights_out": lambda x: x[:0],
             "new_len": lambda x: x[:0], "kept": lambda x: x[:0], "evicted": lambda x: x[:0], "rows": lambda x: 0}
    before = {k: _raw(v) for k, v in args.items() if k.endswith(("_cache", "_block"))}
    getattr(dfl, name)(**{k: empty[k](v) if k in empty else v for k, v in args.items()})
    if name != "paged_evict":  # no rows, but sequences
        some = {k: f for k, f in empty.items() if k not in ("table", "kv_len", "weights", "evicted")}
        some["row_start"] = lambda x: x * 0
        getattr(dfl, name)(**{k: some[k](v) if k in some else v for k, v in args.items()})
    torch.cuda.synchronize()
    assert all(np.array_equal(_raw(args[k]), v) for k, v in before.items())


# --------------------------------------------------------------------------- together
def _steps(torch, dfl, st, steps=3, **kw):
    """Decoding steps over a cache that is cut back as it grows: one drafted block a step."""
    ys = []
    for i in range(steps):
        st["lens"].add_(st["rows"])
        q = dfl.paged_append(st["kc"], st["vc"], st["k"][i], st["v"][i], st["table"], st["lens"], row_start=st["start"],
                             q=st["q"][i], inv_freq=st["f"], evicted=st["evicted"], **st["four"], **kw)
        y = dfl.paged_attention(q, st["kc"], st["vc"], st["table"], st["lens"], row_start=st["start"], lse=st["lse"],
                                **st["four"], **kw)
        one = {x: st["four"][x] for x in ("k_scale", "k_block")}
        dfl.paged_key_weights(st["w"], q, st["kc"], st["table"], st["lens"], st["lse"], row_start=st["start"], **one, **kw)
        blocks = {x: st["four"][x] for x in ("k_block", "v_block")}
        dfl.paged_evict(st["kc"], st["vc"], st["w"], st["table"], st["lens"], st["keep"], first=2, recent=6,
                        new_len=st["lens"], evicted=st["evicted"], **blocks, **kw)
        ys.append(y)
    return torch.stack(ys)


def _steps_state(torch, dfl, seed=0, steps=3):
    rng = np.random.default_rng(seed)
    R = lambda *s: torch.from_numpy(rng.standard_normal(s).astype(np.float32)).cuda().to(torch.bfloat16)  # noqa: E731
    rows = (4, 1, 3)
    kc, kb, _ = _cached4(torch, rng, (24, 8, 2, 64))
    vc, vb, _ = _cached4(torch, rng, (24, 8, 2, 64))
    s = torch.full((2,), 0.125, device="cuda")
    return dict(kc=kc, vc=vc, four=dict(k_block=kb, v_block=vb, k_scale=s, v_scale=s.clone()), keep=24,
                q=R(steps, 8, 4, 64), k=R(steps, 8, 2, 64), v=R(steps, 8, 2, 64), w=torch.from_numpy(rng.random((3, 2, 64)).astype(np.float32)).cuda(),
                table=_i32(torch, rng.permutation(24).reshape(3, 8)), lens=_i32(torch, (22, 0, 30)),
                start=_i32(torch, _starts(rows)), rows=_i32(torch, rows), f=dfl.rope_inv_freq(64, 1e4)[0],
                lse=torch.empty(8, 4, device="cuda"), evicted=_i32(torch, (0, 0, 5)))


@gpu
def test_steps_over_a_cache_that_is_cut_back_match_the_oracle():
    """Every call of the run is checked from the state that the call before left."""
    torch, dfl = _torch(), _dfl()
    st = _steps_state(torch, dfl)
    start, table = st["start"].tolist(), st["table"].tolist()
    for i in range(3):
        st["lens"].add_(st["rows"])
        lens, gone = st["lens"].tolist(), st["evicted"].tolist()
        q = dfl.paged_append(st["kc"], st["vc"], st["k"][i], st["v"][i], st["table"], st["lens"], row_start=st["start"],
                             q=st["q"][i], inv_freq=st["f"], evicted=st["evicted"], **st["four"])
        for s, a, n in O.rows_of(3, 8, start):
            for r in range(n):
                want = O.rotate(f64(st["q"][i])[a + r], lens[s] - n + r + gone[s], f64(st["f"].double()), False, 1.0)
                assert (np.abs(f64(q)[a + r] - want) <= HALF["bf16"] * np.abs(want) + 2.0 ** -20 * 6).all()
        k64, v64 = _values4(st["kc"], st["four"]["k_block"]) / 8, _values4(st["vc"], st["four"]["v_block"]) / 8
        y = dfl.paged_attention(q, st["kc"], st["vc"], st["table"], st["lens"], row_start=st["start"], lse=st["lse"],
                                **st["four"])
        ref, _, mag, _ = O.paged_attention(f64(q), k64, v64, table, lens, start)
        assert (np.abs(f64(y) - ref) <= HALF["bf16"] * np.abs(ref) + (2 * HALF["f16"] + 1e-4) * mag).all()
        w0 = f64(st["w"])
        dfl.paged_key_weights(st["w"], q, st["kc"], st["table"], st["lens"], st["lse"], row_start=st["start"],
                              k_scale=st["four"]["k_scale"], k_block=st["four"]["k_block"])
        want, _ = O.paged_key_weights(w0, f64(q), f64(st["lse"]), k64, table, lens, start)
        assert np.abs(f64(st["w"]) - want).max() <= 1e-4
        w1 = f64(st["w"])
        kept = torch.empty(3, 2, 24, dtype=torch.int32, device="cuda")
        dfl.paged_evict(st["kc"], st["vc"], st["w"], st["table"], st["lens"], 24, first=2, recent=6, new_len=st["lens"],
                        evicted=st["evicted"], kept=kept, k_block=st["four"]["k_block"], v_block=st["four"]["v_block"])
        k2 = _values4(st["kc"], st["four"]["k_block"]) / 8
        for s in range(3):
            assert st["lens"][s].item() == min(lens[s], 24)
            assert st["evicted"][s].item() == gone[s] + lens[s] - min(lens[s], 24)
            for h in range(2):
                slots = O.kept_slots(w1[s, h], lens[s], 24, 2, 6)
                assert kept[s, h].tolist()[:len(slots)] == slots
                for a, b in enumerate(slots):
                    assert np.array_equal(k2[O.slot_of(table[s], 8, 24, a)][h], k64[O.slot_of(table[s], 8, 24, b)][h])


@gpu
def test_steps_captured_and_replayed_with_new_contents():
    torch, dfl = _torch(), _dfl()
    st, other = _steps_state(torch, dfl), _steps_state(torch, dfl, 5)
    flat = lambda d: {**{k: v for k, v in d.items() if isinstance(v, torch.Tensor)}, **d["four"]}  # noqa: E731
    copy = lambda d: {**{k: v.clone() if isinstance(v, torch.Tensor) else v for k, v in d.items()},  # noqa: E731
                      "four": {k: v.clone() for k, v in d["four"].items()}}
    keep = copy(st)
    _steps(torch, dfl, copy(st))
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = _steps(torch, dfl, st)
    for src in (keep, other, keep):
        for k, v in flat(st).items():
            v.view(torch.uint8).copy_(flat(src)[k].view(torch.uint8))
        now = copy(st)
        g.replay()
        torch.cuda.synchronize()
        y2 = _steps(torch, dfl, now)
        torch.cuda.synchronize()
        assert torch.equal(y, y2)
        assert all(np.array_equal(_raw(v), _raw(flat(now)[k])) for k, v in flat(st).items() if k != "lse")


@gpu
def test_steps_from_two_threads_on_streams_of_their_own():
    import threading
    torch, dfl = _torch(), _dfl()
    want = [_steps(torch, dfl, _steps_state(torch, dfl, s)) for s in (1, 2)]
    torch.cuda.synchronize()
    got, errors = [None, None], []

    def work(i):
        try:
            st = _steps_state(torch, dfl, i + 1)
            stream = torch.cuda.Stream()
            stream.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(stream):
                for _ in range(4):
                    s = {**{k: v.clone() if isinstance(v, torch.Tensor) else v for k, v in st.items()},
                         "four": {k: v.clone() for k, v in st["four"].items()}}
                    got[i] = _steps(torch, dfl, s)
            stream.synchronize()
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    ts = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    [t.start() for t in ts]
    [t.join() for t in ts]
    assert not errors, errors
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@gpu
def test_offsets_past_32_bits():
    """Codes and block scales whose byte offsets pass 2^32: the last pages of a cache of 5 GB of codes."""
    torch, dfl = _torch(), _dfl()
    n_pages, page, hd = 1300000, 64, 128
    kc = torch.empty(n_pages, page, 1, hd // 2, dtype=torch.uint8, device="cuda")
    kb = torch.empty(n_pages, page, 1, hd // 16, dtype=torch.uint8, device="cuda")
    kb[:64] = 0x7f
    kb = kb.view(torch.float8_e4m3fn)
    rng = np.random.default_rng(0)
    c, b, y = _cached4(torch, rng, (8, page, 1, hd))
    kc[-8:] = c
    kb.view(torch.uint8)[-8:] = b.view(torch.uint8)
    ids = np.arange(n_pages - 8, n_pages)[rng.permutation(8)]
    table, lens = _i32(torch, ids[None]), _i32(torch, [500])
    q = torch.from_numpy(rng.standard_normal((2, 4, hd)).astype(np.float32)).cuda().to(torch.bfloat16)
    kw = dict(k_block=kb, v_block=kb)
    rel = [list(ids - (n_pages - 8))]
    for rows in (2, 40):
        qq = q.repeat(rows // 2, 1, 1)
        lse = torch.empty(rows, 4, device="cuda")
        out = dfl.paged_attention(qq, kc, kc, table, lens, lse=lse, **kw)
        ref, _, mag, _ = O.paged_attention(f64(qq), y, y, rel, [500])
        assert (np.abs(f64(out) - ref) <= HALF["bf16"] * np.abs(ref) + (2 * HALF["f16"] + 1e-4) * mag).all()
    w = torch.zeros(1, 1, 512, device="cuda")
    lse = torch.empty(2, 4, device="cuda")
    dfl.paged_attention(q, kc, kc, table, lens, lse=lse, **kw)
    dfl.paged_key_weights(w, q, kc, table, lens, lse, k_block=kb)
    want, _ = O.paged_key_weights(np.zeros((1, 1, 512)), f64(q), f64(lse), y, rel, [500])
    assert np.abs(f64(w) - want).max() <= 1e-4 * want.max()
    k, _ = dfl.paged_read(kc, kc, table, lens, 500, **kw, dtype=torch.float32)
    assert np.array_equal(f64(k)[:, 0], np.stack([y[rel[0][p // page], p % page, 0] for p in range(500)]))
    kept = torch.empty(1, 1, 100, dtype=torch.int32, device="cuda")
    vc, vb = kc.clone(), kb.clone()
    dfl.paged_evict(kc, vc, w, table, lens, 100, kept=kept, k_block=kb, v_block=vb)
    moved = [y[rel[0][p // page], p % page] for p in kept[0, 0].tolist()]
    for codes, blocks in ((kc, kb), (vc, vb)):
        got = _values4(codes[-8:], blocks[-8:])
        assert np.array_equal(np.stack([got[rel[0][i // page], i % page] for i in range(100)]), np.stack(moved))
