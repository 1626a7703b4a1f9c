"""The target's verification pass (paged_append, paged_attention, verify_drafts) against plain float64 (oracle/target.py),
and the refusals of its calls.

Tolerances, from the arithmetic.  An output rounded once to a type t is off by half a step, finfo(t).eps / 2 relative
(and half the smallest step near zero); what comes before that rounding is 32-bit:
  append     a rotated element is two products of f32 values (each off by about 2^-23) and a sine or cosine within
             2^-21: 2^-20 of the pair's magnitude covers them
  attention  a score is a sum of head_dim f32 products: off by head_dim 2^-24 sum|q k| at most, which moves a
             probability by as much relative; values enter as sum p |v| of that.  P itself is rounded to 16 bits where
             many rows share the keys (its half step, relative)
  verify     sums in 64 bits of exponentials within 2^-20: whole numbers are equal wherever the deciding numbers are
             further than 1e-5 (relative) from their border
"""
import ctypes as C
import itertools

import numpy as np
import pytest

from oracle import target as O

gpu = pytest.mark.gpu


def _dfl():
    import block_speculative_drafting_gb300 as dfl
    return dfl


def _torch():
    return pytest.importorskip("torch")


def _types():
    t = _torch()
    return {"bf16": t.bfloat16, "f16": t.float16, "f32": t.float32, "e4m3": t.float8_e4m3fn}


HALF = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "f32": 2.0 ** -24, "e4m3": 2.0 ** -4}  # a rounding, relative
TINY = {"bf16": 0.0, "f16": 2.0 ** -25, "f32": 0.0, "e4m3": 2.0 ** -10}  # half the smallest step


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


# --------------------------------------------------------------------------- refusals (no device)
def _cache_struct(**kw):
    from block_speculative_drafting_gb300 import _abi
    c = _abi.PagedCache(4096, 8192, _abi.BF16, 2, 64, 16, 4)
    for st in (c.k_strides, c.v_strides):
        st[0], st[1], st[2] = 16 * 2 * 64, 2 * 64, 64
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def _rows_struct(**kw):
    from block_speculative_drafting_gb300 import _abi
    r = _abi.PagedRows(2, 4, 4, None, 4096, 4096, 4)
    for k, v in kw.items():
        setattr(r, k, v)
    return r


def _head_struct(heads, dtype=1, **kw):
    from block_speculative_drafting_gb300 import _abi
    h = _abi.HeadRows(4096, dtype, heads, heads * 64, 64)
    for k, v in kw.items():
        setattr(h, k, v)
    return h


@pytest.fixture(scope="module")
def lib():
    from block_speculative_drafting_gb300.csrc.build import build
    build()
    return _dfl().lib()


BAD_CACHES = [("dtype", 0, -1), ("dtype", 9, -1), ("head_dim", 96, -2), ("kv_heads", 0, -1), ("page_size", 0, -1),
              ("page_size", 65537, -1), ("n_pages", -1, -1), ("k", None, -1), ("v", 8200, -1), ("k_scale", 4096, -1)]
BAD_ROWS = [("n_seqs", -1, -1), ("n_rows", -1, -1), ("n_rows", 5, -1), ("n_rows", 1 << 24, -1), ("max_pages", -1, -1),
            ("max_pages", 1 << 30, -1), ("kv_len", None, -1), ("table", None, -1), ("table", 4098, -1),
            ("table_stride", 3, -1), ("n_seqs", 0, -1)]


@pytest.mark.parametrize("field,value,code", BAD_CACHES + BAD_ROWS)
def test_paged_calls_refuse_bad_descriptions(lib, field, value, code):
    of_cache = (field, value, code) in BAD_CACHES
    c = _cache_struct(**({field: value} if of_cache else {}))
    r = _rows_struct(**({} if of_cache else {field: value}))
    k, q = _head_struct(2), _head_struct(4)
    assert lib.dflash_paged_append(C.byref(c), C.byref(r), C.byref(k), C.byref(k), C.byref(q), C.byref(q), None, None,
                                   1e-6, None, None) == code
    assert lib.dflash_last_error(None) != b""
    assert lib.dflash_paged_attention(C.byref(c), C.byref(r), C.byref(q), C.byref(q), None, 0.1, 0, 4096, 1 << 40,
                                      None) == code


def test_paged_append_refuses_bad_arguments(lib):
    from block_speculative_drafting_gb300 import _abi
    c, r, k, q = _cache_struct(), _rows_struct(), _head_struct(2), _head_struct(4)

    def call(k=k, v=k, q=q, qo=q, qn=None, kn=None, eps=1e-6, rot=None, c=c, r=r):
        ref = lambda x: None if x is None else C.byref(x)  # noqa: E731
        return lib.dflash_paged_append(ref(c), ref(r), ref(k), ref(v), ref(q), ref(qo), qn, kn, eps, ref(rot), None)

    bad_rot = [_abi.Rotation(4096, n, 0, 1.0) for n in (0, 8, 24, 80, -16)]
    bad_rot += [_abi.Rotation(None, 64, 0, 1.0), _abi.Rotation(4100, 64, 0, 1.0),
                _abi.Rotation(4096, 64, 0, float("nan"))]
    calls = [dict(c=None), dict(r=None), dict(k=None), dict(v=None), dict(qo=None), dict(q=None),
             dict(k=_head_struct(3)), dict(v=_head_struct(2, data=4104)), dict(k=_head_struct(2, row_stride=130)),
             dict(q=_head_struct(3), qo=_head_struct(3)), dict(qo=_head_struct(6)), dict(qo=_head_struct(4, dtype=2)),
             dict(q=_head_struct(4, dtype=3)), dict(v=_head_struct(2, dtype=2)), dict(qn=4100), dict(kn=4096, eps=-1.0),
             dict(kn=4096, eps=float("nan"))]
    for bad in calls + [dict(rot=x) for x in bad_rot]:
        assert call(**bad) == _abi.DFLASH_EINVAL, bad
    assert call(r=_rows_struct(n_rows=0)) == 0  # nothing to do, nothing launched


def test_paged_attention_refuses_bad_arguments(lib):
    from block_speculative_drafting_gb300 import _abi
    c, r, q = _cache_struct(), _rows_struct(), _head_struct(4)

    def call(c=c, r=r, q=q, out=q, lse=None, scale=0.1, window=0, ws=4096, n=1 << 40):
        ref = lambda x: None if x is None else C.byref(x)  # noqa: E731
        return lib.dflash_paged_attention(ref(c), ref(r), ref(q), ref(out), lse, scale, window, ws, n, None)

    for bad in [dict(c=None), dict(r=None), dict(q=None), dict(out=None), dict(q=_head_struct(4, dtype=0)),
                dict(out=_head_struct(4, dtype=2)), dict(q=_head_struct(4, dtype=2), out=_head_struct(4, dtype=2)),
                dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")), dict(window=-1), dict(window=(1 << 30) + 1),
                dict(lse=4097), dict(out=_head_struct(2)), dict(q=_head_struct(5), out=_head_struct(5))]:
        assert call(**bad) == _abi.DFLASH_EINVAL, bad
    assert call(r=_rows_struct(n_rows=0)) == 0
    # more tiles of keys than a 32-bit count: 2^16 sequences of 2^31 - 2^17 positions
    wide = dict(n_seqs=1 << 16, n_rows=1 << 16, max_pages=(1 << 27) - (1 << 13), table_stride=1 << 27)
    assert call(r=_rows_struct(**wide)) == _abi.DFLASH_EINVAL


def test_binding_refuses_tensors_of_the_host_and_other_objects(lib):
    torch, dfl = pytest.importorskip("torch"), _dfl()
    x, i = torch.zeros(2, 16, 2, 64), torch.zeros(2, 2, dtype=torch.int32)
    refused = [lambda: dfl.paged_append(x, x, x[0], x[0], i, i[0]), lambda: dfl.paged_attention(x[0], x, x, i, i[0]),
               lambda: dfl.verify_drafts(x[0, 0], i[0, :1], x[0, 0, 0, :1], x[0, 0, 0, :1]),
               lambda: dfl.paged_attention_workspace(x[0], x, 2)]
    for call in refused:
        with pytest.raises(dfl.DFlashError, match="CUDA device"):
            call()
    for call in (lambda: dfl.paged_append(None, x, x, x, i, i), lambda: dfl.paged_attention([1.0], x, x, i, i),
                 lambda: dfl.verify_drafts(3, i, x, x)):
        with pytest.raises(TypeError, match="has to be a tensor"):
            call()


def test_verify_refuses_bad_arguments(lib):
    from block_speculative_drafting_gb300 import _abi
    good = dict(target=4096, dtype=0, stride=100, dl=None, ds=100, tok=4096, start=None, temp=None, au=4096, su=4096,
                n=2, d=4, vocab=100, acc=4096, nxt=4096, prob=None, ws=4096, nb=1 << 40)

    def call(**kw):
        return lib.dflash_verify(*{**good, **kw}.values(), None)

    for bad in [dict(target=None), dict(dtype=3), dict(dtype=-1), dict(stride=99), dict(dl=4096, ds=99), dict(tok=None),
                dict(au=None), dict(su=None), dict(n=-1), dict(n=0), dict(d=-1), dict(d=5), dict(d=1 << 24),
                dict(vocab=0), dict(vocab=1 << 30), dict(acc=None), dict(nxt=None), dict(target=4098), dict(tok=4097),
                dict(start=4098)]:
        assert call(**bad) == _abi.DFLASH_EINVAL, bad
    assert call(n=0, d=0) == 0


def test_python_refuses_bad_tensors(lib):
    torch, dfl = _torch(), _dfl()
    k = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    cache = torch.zeros(3, 16, 2, 64, dtype=torch.bfloat16)
    table, kv_len = torch.zeros(2, 4, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    calls = [lambda: dfl.paged_append(cache, cache, k, k, table, kv_len),  # not on a GPU
             lambda: dfl.paged_append(cache, cache, k[:, :1], k[:, :1], table, kv_len),
             lambda: dfl.paged_append(cache, cache, k, k, table.long(), kv_len),
             lambda: dfl.paged_append(cache, cache, k, k, table, kv_len.long()),
             lambda: dfl.paged_append(cache, cache, k.double(), k, table, kv_len),
             lambda: dfl.paged_append(cache, cache[:, :8], k, k, table, kv_len),
             lambda: dfl.paged_append(cache[:, :, :, ::2], cache[:, :, :, ::2], k[..., ::2], k[..., ::2], table, kv_len),
             lambda: dfl.paged_append(cache[:1].expand(3, 16, 2, 64), cache, k, k, table, kv_len),
             lambda: dfl.paged_attention(k, cache, cache, table, kv_len),
             lambda: dfl.paged_attention(k[..., :32], cache, cache, table, kv_len),
             lambda: dfl.paged_attention(k, cache, cache, table, kv_len, lse=torch.zeros(4, 3)),
             lambda: dfl.verify_drafts(torch.zeros(5, 9), torch.zeros(4, dtype=torch.int32), torch.zeros(4),
                                       torch.zeros(2)),
             lambda: dfl.verify_drafts(torch.zeros(6, 9), torch.zeros(4, dtype=torch.int32), torch.zeros(4),
                                       torch.zeros(2), draft_logits=torch.zeros(4, 8)),
             lambda: dfl.verify_drafts(torch.zeros(6, 9), torch.zeros(4, dtype=torch.int64), torch.zeros(4),
                                       torch.zeros(2))]
    for i, f in enumerate(calls):
        with pytest.raises(dfl.DFlashError) as e:
            f()
        assert e.value.code == dfl._abi.DFLASH_EINVAL, i


def test_rope_frequencies():
    torch, dfl = _torch(), _dfl()
    f, s = dfl.rope_inv_freq(64, 1e4, device="cpu")
    assert f.dtype == torch.float64 and f.shape == (32,) and s == 1.0
    assert np.allclose(f.numpy(), 1e4 ** (-np.arange(32) / 32.0), rtol=1e-14, atol=0)
    g, s = dfl.rope_inv_freq(64, 1e4, scaling="linear", factor=8.0, device="cpu")
    assert np.allclose(g.numpy() * 8, f.numpy(), rtol=1e-14, atol=0) and s == 1.0
    y, s = dfl.rope_inv_freq(64, 1e4, scaling="yarn", factor=8.0, trained=4096, device="cpu")
    turns = 4096 * f.numpy() / (2 * np.pi)
    ratio = y.numpy() / f.numpy()
    assert np.allclose(ratio[turns > 40], 1.0) and np.allclose(ratio[turns < 0.8], 1 / 8.0)
    assert (np.diff(ratio) <= 1e-12).all() and abs(s - (0.1 * np.log(8.0) + 1.0)) < 1e-12
    for bad in (dict(rotary=7), dict(rotary=64, scaling="yarn"), dict(rotary=64, scaling="other"),
                dict(rotary=64, factor=0.0)):
        with pytest.raises(ValueError):
            dfl.rope_inv_freq(**bad, device="cpu")


# --------------------------------------------------------------------------- the oracle's own pins
def test_oracle_attention_of_equal_keys_is_the_mean():
    rng = np.random.default_rng(0)
    v = rng.standard_normal((2, 4, 1, 8))
    out, lse, _, _ = O.paged_attention(np.ones((1, 2, 8)), np.zeros((2, 4, 1, 8)), v, [[1, 0]], [6])
    want = np.concatenate((v[1], v[0, :2])).mean(0)[0]
    assert np.allclose(out[0], want) and np.allclose(lse, np.log(6))


def test_oracle_verify_by_hand():
    t = np.log(np.array([[.5, .25, .25], [.1, .8, .1], [.2, .3, .5]]))
    # first draft kept (u = .4 < .5), second refused (u = .9 >= .1): token from [.1, .8, 0] / .9
    res, prob = O.verify(t, [0, 2], [.4, .9], [.05])
    assert res[0][:2] == (1, 0) and np.allclose(prob, [.5, .1])
    assert O.verify(t, [0, 2], [.4, .9], [.5])[0][0][:2] == (1, 1)
    assert O.verify(t, [0, 1], [.4, .5], [.6])[0][0][:2] == (2, 2)
    q = np.log(np.array([[.25, .5, .25]]))
    # u q < p: .9 * .5 >= .25 refuses draft 1; left max(p - q, 0) = [.25, 0, 0]
    assert O.verify(t[:2], [1], [.9], [.99], draft_logits=q)[0][0][:2] == (0, 0)


# --------------------------------------------------------------------------- inputs on the GPU
def _layout(torch, rng, lens, rows, page, spare=2, bad=()):
    """A shuffled table that holds each sequence's tokens; (sequence, page index) pairs of `bad` get bad ids."""
    n = len(lens)
    need = [max(0, -(-l // page)) for l in lens]
    width = max(1, max(need) + 1)
    n_pages = sum(need) + spare
    ids = rng.permutation(n_pages)
    table = np.full((n, width), -1, np.int32)
    at = 0
    for s, m in enumerate(need):
        table[s, :m] = ids[at:at + m]
        at += m
    for j, (s, i) in enumerate(bad):
        table[s, i] = (-1, n_pages, 2 ** 31 - 1, -2 ** 31)[j % 4]
    return table, n_pages


def _cached(torch, rng, shape, kind, order="slot"):
    """A cache tensor [pages][page][heads][hd] and its float64 values (codes, unscaled)."""
    x = torch.from_numpy(rng.standard_normal(shape).astype(np.float32) * (16 if kind == "e4m3" else 1)).cuda()
    x = x.to(_types()[kind])
    if order == "head":  # [page][head][slot] in memory
        y = torch.empty((shape[0], shape[2], shape[1], shape[3]), dtype=x.dtype, device="cuda")
        y.permute(0, 2, 1, 3).view(torch.uint8).copy_(x.view(torch.uint8)) if kind == "e4m3" else \
            y.permute(0, 2, 1, 3).copy_(x)
        x = y.permute(0, 2, 1, 3)
    return x, f64(x)


def _i32(torch, x):
    return torch.tensor(np.asarray(x, np.int32), device="cuda")


def _starts(rows):
    return np.concatenate(([0], np.cumsum(rows)))


# --------------------------------------------------------------------------- append
def _check_append(kind, src, hd=128, heads=4, kvh=2, page=16, rows=(1, 3), lens=(5, 40), rotary=None, interleaved=False,
                  norm=False, uniform=False, bad=(), order="slot", out=None, extra=0, scale=1.0, far=None, seed=0):
    torch, dfl = _torch(), _dfl()
    rng = np.random.default_rng(seed)
    T = _types()
    table, n_pages = _layout(torch, rng, lens, rows, page, bad=bad)
    R = sum(rows) + extra
    qkv = torch.from_numpy(rng.standard_normal((R, heads + 2 * kvh, hd)).astype(np.float32)).cuda().to(T[src])
    q, k, v = qkv.split((heads, kvh, kvh), 1)
    kc, k0 = _cached(torch, rng, (n_pages, page, kvh, hd), kind, order)
    vc, v0 = _cached(torch, rng, (n_pages, page, kvh, hd), kind, order)
    sc = [torch.from_numpy((0.5 + rng.random(kvh)).astype(np.float32) / 16).cuda() for _ in range(2)] \
        if kind == "e4m3" else [None, None]
    gains = [torch.from_numpy((1 + 0.1 * rng.standard_normal(hd)).astype(np.float32)).cuda() if norm else None
             for _ in range(2)]
    f = (1e4 ** (-np.arange(0, rotary, 2) / rotary)) if rotary else None
    q_out = torch.full((R, heads, hd), 7.0, device="cuda", dtype=T[out or src])
    got = dfl.paged_append(kc, vc, k, v, _i32(torch, table), _i32(torch, lens),
                           row_start=None if uniform else _i32(torch, _starts(rows)), q=q, q_out=q_out,
                           inv_freq=None if f is None else torch.from_numpy(f).cuda(), interleaved=interleaved,
                           rope_scale=scale, q_norm=gains[0], k_norm=gains[1], k_scale=sc[0], v_scale=sc[1])
    torch.cuda.synchronize()
    assert got is q_out
    gn = [None if g is None else f64(g) for g in gains]
    slots, qr, touched = O.paged_append(f64(k), f64(v), f64(q), table, lens, page, n_pages,
                                        None if uniform else _starts(rows), f, interleaved, scale, gn[0], gn[1])

    def near(got, ref, amp, kind, what):
        tol = HALF[kind] * np.abs(ref) + TINY[kind] + 2.0 ** -20 * amp
        assert (np.abs(got - ref) <= tol).all(), (what, float(np.max(np.abs(got - ref) / tol)))

    gq = f64(got)
    for r in range(R):
        if r in touched:
            near(gq[r], qr[r], scale * np.abs(qr[r]).max() + 1, out or src, ("q", r))
        else:
            assert (gq[r] == 7.0).all()  # rows of no sequence stay
    for got_c, old, idx, s in ((f64(kc), k0, 0, sc[0]), (f64(vc), v0, 1, sc[1])):
        want = old.copy()
        for (pg, sl), kv in slots.items():
            x = kv[idx]
            if s is not None:
                x = np.clip(x / f64(s)[:, None], -448, 448)
            near(got_c[pg, sl], x, np.abs(x).max() + (0 if s is not None else 1), kind, ("cache", idx, pg, sl))
            want[pg, sl] = got_c[pg, sl]
        assert np.array_equal(got_c, want)  # every other slot as it was
    return got


@gpu
@pytest.mark.parametrize("kind,src", [("bf16", "bf16"), ("f16", "f16"), ("e4m3", "bf16"), ("e4m3", "f32"),
                                      ("bf16", "f32"), ("f16", "bf16")])
@pytest.mark.parametrize("hd", [64, 128])
def test_append_types(kind, src, hd):
    _check_append(kind, src, hd=hd, rotary=hd, norm=True, seed=hd)


@gpu
@pytest.mark.parametrize("rotary,interleaved", [(None, False), (16, False), (16, True), (64, False), (64, True),
                                                (112, False), (128, True)])
def test_append_rotations(rotary, interleaved):
    _check_append("bf16", "bf16", rotary=rotary, interleaved=interleaved, scale=1.25, out="f32", seed=3)


@gpu
@pytest.mark.parametrize("page", [1, 3, 16, 48, 64])
@pytest.mark.parametrize("order", ["slot", "head"])
def test_append_pages(page, order):
    _check_append("f16", "f16", hd=64, page=page, order=order, rows=(4, 0, 1, 7), lens=(4, 0, 33, 64), rotary=32, seed=page)


@gpu
def test_append_uniform_and_heads():
    _check_append("bf16", "bf16", heads=8, kvh=1, rows=(4, 4), lens=(9, 4), uniform=True, rotary=128)
    _check_append("e4m3", "f16", heads=15, kvh=3, rows=(1,), lens=(1,), uniform=True, rotary=64)
    _check_append("bf16", "bf16", heads=40, kvh=40, hd=64, rows=(2, 1), lens=(2, 17), norm=True)


@gpu
def test_append_skips_what_is_not_held():
    # rows before position 0, past the table, on bad pages, and rows of no sequence
    _check_append("bf16", "bf16", rows=(4, 3, 40), lens=(2, 40, 41), bad=((1, 2), (2, 0), (2, 1), (2, 2)), rotary=64,
                  extra=3, seed=5)
    torch, dfl = _torch(), _dfl()
    kc = torch.zeros(2, 4, 2, 64, dtype=torch.bfloat16, device="cuda")
    k = torch.ones(3, 2, 64, dtype=torch.bfloat16, device="cuda")
    for kv, start in ((100, None), (-5, None), (2 ** 31 - 1, None), (4, [3, 3]), (4, [-7, 99]), (4, [5, 1]), (2, [0, 2])):
        a, b = torch.zeros_like(kc), torch.zeros_like(kc)
        dfl.paged_append(a, b, k, k, _i32(torch, [[1]]), _i32(torch, [kv]),
                         row_start=None if start is None else _i32(torch, start))
        slots, _, _ = O.paged_append(f64(k), f64(k), None, [[1]], [kv], 4, 2, start)
        want = np.zeros((2, 4, 2, 64))
        for (p, s), x in slots.items():
            want[p, s] = x[0]
        assert np.array_equal(f64(a), want) and np.array_equal(f64(b), want), (kv, start)


@gpu
def test_append_far_positions_and_special_values():
    torch, dfl = _torch(), _dfl()
    rng = np.random.default_rng(11)
    # positions whose angle turns up to 10^8 times: the reduced angle keeps its accuracy
    lens = [2 ** 20 + 3, 2 ** 27 + 1]
    page, hd = 65536, 64
    width = 2 ** 27 // page + 2
    table = np.full((2, width), -1, np.int32)
    table[0, lens[0] // page], table[1, lens[1] // page] = 1, 0
    kc = torch.zeros(2, page, 1, hd, dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    x = torch.from_numpy(rng.standard_normal((2, 1, hd)).astype(np.float32)).cuda()
    f = 1e4 ** (-np.arange(0, hd, 2) / hd)
    q = dfl.paged_append(kc, vc, x, x, _i32(torch, table), _i32(torch, lens), q=x, inv_freq=torch.from_numpy(f).cuda())
    _, ref, _ = O.paged_append(f64(x), f64(x), f64(x), table, lens, page, 2, None, f)
    # p f in 64 bits is itself off by 2^-53 of up to 2^27: far below
    assert np.abs(f64(q) - ref).max() <= 2.0 ** -19 * np.abs(f64(x)).max()
    for s in range(2):
        assert np.abs(f64(kc)[table[s, lens[s] // page], (lens[s] - 1) % page] - ref[s]).max() <= 2.0 ** -7 * 4
    # NaN and infinity: NaN stays, an infinity is the largest finite code of an 8-bit cache
    y = torch.zeros(1, 1, hd, device="cuda")
    y[0, 0, :4] = torch.tensor([float("nan"), float("inf"), -float("inf"), 1e9], device="cuda")
    kc = torch.zeros(1, 4, 1, hd, device="cuda").to(torch.float8_e4m3fn)
    vc = kc.clone()
    dfl.paged_append(kc, vc, y, y, _i32(torch, [[0]]), _i32(torch, [1]))
    got = f64(kc)[0, 0, 0, :4]
    assert np.isnan(got[0]) and list(got[1:]) == [448.0, -448.0, 448.0]
    assert (f64(kc)[0, 1:] == 0).all()


@gpu
def test_append_in_place_queries():
    torch, dfl = _torch(), _dfl()
    rng = np.random.default_rng(2)
    x = torch.from_numpy(rng.standard_normal((6, 8, 128)).astype(np.float32)).cuda().to(torch.bfloat16)
    kc = torch.zeros(2, 16, 2, 128, dtype=torch.bfloat16, device="cuda")
    f, s = dfl.rope_inv_freq(128, 1e6)
    args = (kc, kc.clone(), x[:, :2], x[:, 2:4], _i32(torch, [[0, 1]]), _i32(torch, [20]))
    a = dfl.paged_append(*args, q=x[:, 4:], inv_freq=f)
    q = x[:, 4:]
    b = dfl.paged_append(*args, q=q, q_out=q, inv_freq=f)
    assert b is q and torch.equal(a, b)


# --------------------------------------------------------------------------- attention
def _check_attention(kind, src=None, hd=128, heads=4, kvh=2, page=16, rows=(1,), lens=(40,), window=0, uniform=False, bad=(),
                     order="slot", extra=0, scale=None, seed=0, poison=None, spread=1.0):
    torch, dfl = _torch(), _dfl()
    rng = np.random.default_rng(seed)
    T = _types()
    src = src or kind
    table, n_pages = _layout(torch, rng, [max(l, 0) for l in lens], rows, page, bad=bad)
    R = sum(rows) + extra
    q = torch.from_numpy(spread * rng.standard_normal((R, heads, hd)).astype(np.float32)).cuda().to(T[src])
    kc, k64 = _cached(torch, rng, (n_pages, page, kvh, hd), kind, order)
    vc, v64 = _cached(torch, rng, (n_pages, page, kvh, hd), kind, order)
    if poison is not None:
        poison(torch, kc, vc, table)
        k64, v64 = f64(kc), f64(vc)
    ks = vs = None
    if kind == "e4m3":
        ks, vs = (torch.from_numpy((0.5 + rng.random(kvh)).astype(np.float32) / 16).cuda() for _ in range(2))
        k64, v64 = k64 * f64(ks)[:, None], v64 * f64(vs)[:, None]
    out = torch.full((R, heads, hd), 7.0, device="cuda", dtype=T[src])
    lse = torch.full((R, heads), 7.0, device="cuda")
    start = None if uniform else _i32(torch, _starts(rows))
    args = dict(row_start=start, scale=scale, window=window, k_scale=ks, v_scale=vs, out=out, lse=lse)
    dfl.paged_attention(q, kc, vc, _i32(torch, table), _i32(torch, lens), **args)
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
    # a score's error: head_dim f32 additions, of partial sums up to |q| |k|
    norm = lambda x: np.linalg.norm(np.where(np.isfinite(x), x, 0.0), axis=-1).max()  # noqa: E731
    s_err = hd * 2.0 ** -24 * (hd ** -0.5 if scale is None else scale) * norm(f64(q)) * norm(k64) + 2.0 ** -20
    # an 8-bit cache's P is one f16 where more than 16 rows share the keys, a hi + lo pair otherwise
    one_p = kind == "e4m3" and -(-R // len(lens)) * (heads // kvh) > 16
    p_err = s_err + (HALF["f16"] if one_p else 0.0)
    with np.errstate(all="ignore"):
        tol = HALF[src] * np.abs(ref) + TINY[src] + 2 * p_err * mag
        fine = np.isfinite(ref)
        assert np.array_equal(fine, np.isfinite(got)), "finite where the definition is"
        assert np.array_equal(np.isnan(ref), np.isnan(got))
        assert np.array_equal(ref[~fine & ~np.isnan(ref)], got[~fine & ~np.isnan(ref)])
        d = np.abs(got - ref)[fine]
        assert (d <= tol[fine]).all(), float((d / np.maximum(tol[fine], 1e-30)).max())
    assert np.array_equal(np.isneginf(rl), np.isneginf(gl)) and np.array_equal(np.isnan(rl), np.isnan(gl))
    ok = np.isfinite(rl)
    assert (np.abs(gl[ok] - rl[ok]) <= s_err + 2.0 ** -21 * np.abs(rl[ok])).all()


@gpu
@pytest.mark.parametrize("kind,src", [("bf16", "bf16"), ("f16", "f16"), ("e4m3", "bf16"), ("e4m3", "f16")])
@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("group,rows", [(1, 1), (4, 1), (3, 5), (4, 5), (5, 8), (8, 16), (4, 40)])
def test_attention_types_and_tiles(kind, src, hd, group, rows):
    # one to ten tiles of 16 query rows a unit; two sequences of different lengths
    _check_attention(kind, src, hd=hd, heads=2 * group, kvh=2, rows=(rows, rows), lens=(rows + 3, 300), uniform=True,
                     seed=group)


@gpu
@pytest.mark.parametrize("page", [1, 3, 16, 48, 128, 1000])
@pytest.mark.parametrize("order", ["slot", "head"])
def test_attention_pages(page, order):
    _check_attention("bf16", page=page, order=order, rows=(2, 1, 3), lens=(127, 128, 129), seed=page)


@gpu
@pytest.mark.parametrize("length", [0, 1, 2, 15, 16, 17, 127, 128, 129, 1000])
def test_attention_lengths(length):
    _check_attention("f16", rows=(1, 1), lens=(length, 5), heads=8, kvh=2, uniform=True)
    _check_attention("e4m3", "bf16", rows=(3, 2), lens=(length, 5), hd=64, heads=6, kvh=1)


@gpu
@pytest.mark.parametrize("window", [1, 7, 16, 100, 5000])
@pytest.mark.parametrize("rows", [1, 6, 33])
def test_attention_windows(window, rows):
    _check_attention("bf16", rows=(rows, 2, rows), lens=(400, 2, rows), window=window, heads=4, kvh=1)


@gpu
def test_attention_ragged_padded_and_bad_pages():
    _check_attention("bf16", rows=(0, 3, 0, 1, 2, 0), lens=(9, 200, 0, 77, 2, 4), extra=4, seed=1)
    # no page held, some not held, positions before 0, lengths past the table
    _check_attention("bf16", rows=(1, 2, 1), lens=(10, 100, 33), bad=((0, 0), (1, 1), (1, 3), (2, 2)), seed=2)
    _check_attention("f16", rows=(4, 2, 1, 1), lens=(2, 0, -7, 1), seed=3)
    _check_attention("e4m3", "f16", rows=(5,), lens=(4000,), bad=tuple((0, i) for i in range(0, 250, 3)), window=900, seed=4)


@gpu
def test_attention_bad_row_starts_and_lengths():
    torch, dfl = _torch(), _dfl()
    rng = np.random.default_rng(0)
    kc, k64 = _cached(torch, rng, (4, 16, 1, 64), "bf16")
    vc, v64 = _cached(torch, rng, (4, 16, 1, 64), "bf16")
    q = torch.from_numpy(rng.standard_normal((6, 2, 64)).astype(np.float32)).cuda().to(torch.bfloat16)
    table = np.array([[0, 1], [2, 3]], np.int32)
    for start, lens in (([0, 3, 6], (100, 2 ** 31 - 1)), ([-4, 2, 99], (20, 30)), ([6, 6, 6], (3, 4)),
                        ([0, 0, 0], (3, 4)), ([2, 4, 3], (20, 30)), ([0, 2, 6], (-2 ** 31, 32)), ([5, 2, 4], (9, 9))):
        out = torch.full_like(q, 7.0)
        dfl.paged_attention(q, kc, vc, _i32(torch, table), _i32(torch, lens), row_start=_i32(torch, start), out=out)
        ref, _, mag, touched = O.paged_attention(f64(q), k64, v64, table, [min(l, 2 ** 31 - 1) for l in lens], start) \
            if max(lens) < 1000 else (None, None, None, None)
        got = f64(out)
        assert np.isfinite(got).all()
        if ref is not None:
            for r in range(6):
                if r in touched:
                    assert (np.abs(got[r] - ref[r]) <= HALF["bf16"] * np.abs(ref[r]) + 1e-4 * mag[r]).all(), (start, r)
                else:
                    assert (got[r] == 7.0).all(), (start, r)


@gpu
@pytest.mark.parametrize("kind", ["bf16", "f16", "e4m3"])
def test_attention_keeps_what_rows_may_not_see_out(kind):
    """Slots of no row's view hold NaN and infinities; slots that only later rows see hold them too (there the later
    rows' results are not finite, the earlier rows' are)."""
    def free(torch, kc, vc, table):  # every slot past the lengths, and every page of no sequence
        nan = torch.tensor(float("nan"), device="cuda").to(kc.dtype)
        page = kc.shape[1]
        used = np.zeros((kc.shape[0], page), bool)
        for s, l in enumerate(free.lens):
            for p in range(free.lo[s], l):
                if 0 <= table[s][p // page] < kc.shape[0]:
                    used[table[s][p // page], p % page] = True
        for c in (kc, vc):
            raw = c.view(torch.uint8) if kind == "e4m3" else c
            bits = 0x7f if kind == "e4m3" else float("nan")
            raw[torch.from_numpy(~used).cuda()] = bits
        del nan
        free.more(torch, kc, vc, table)

    free.lens, free.lo, free.more = (5, 130), (0, 0), lambda *a: None
    _check_attention(kind, "f16" if kind == "e4m3" else kind, rows=(2, 4), lens=(5, 130), poison=free)
    # the last row's value is not finite: the rows before it do not see it
    def later(torch, kc, vc, table):
        p = 129
        raw = vc.view(torch.uint8) if kind == "e4m3" else vc
        raw[int(table[1][p // 16]), p % 16, 0, ::3] = 0xff if kind == "e4m3" else float("inf")
        raw[int(table[1][p // 16]), p % 16, 1, 1] = 0x7f if kind == "e4m3" else float("nan")
        rk = kc.view(torch.uint8) if kind == "e4m3" else kc
        rk[int(table[1][p // 16]), p % 16, 1, 5] = 0x7f if kind == "e4m3" else float("nan")

    free.more = later
    for hd, heads, kvh, rows in ((128, 4, 2, (2, 4)), (64, 16, 2, (1, 9)), (128, 2, 2, (3, 3)), (128, 32, 2, (3, 9))):
        _check_attention(kind, "f16" if kind == "e4m3" else kind, hd=hd, heads=heads, kvh=kvh, rows=rows, lens=(5, 130),
                         poison=free)
    # a window's edge: keys that the first rows see and the last do not
    free.lo, free.more = (0, 100), lambda torch, kc, vc, table: (vc.view(torch.uint8) if kind == "e4m3" else vc)[
        int(table[1][101 // 16]), 101 % 16].fill_(0x7f if kind == "e4m3" else float("inf"))
    _check_attention(kind, "f16" if kind == "e4m3" else kind, rows=(2, 4), lens=(5, 130), window=27, poison=free)


@gpu
def test_attention_large_scores_and_infinities():
    # scores of a few hundred: the reference moves, differences of exponents keep their accuracy
    _check_attention("bf16", rows=(3,), lens=(500,), spread=20.0, scale=0.5)
    _check_attention("e4m3", "bf16", rows=(3,), lens=(500,), spread=1e6, scale=1e-6)
    torch, dfl = _torch(), _dfl()
    # an infinite query: NaN in its own row and head only
    rng = np.random.default_rng(0)
    kc, _ = _cached(torch, rng, (4, 16, 1, 64), "bf16")
    q = torch.ones(4, 2, 64, dtype=torch.bfloat16, device="cuda")
    q[2, 1, 3] = float("inf")
    out = dfl.paged_attention(q, kc, kc, _i32(torch, [[0, 1, 2, 3]]), _i32(torch, [60]))
    bad = ~torch.isfinite(out).all(-1)
    assert bad.sum() == 1 and bad[2, 1]


@gpu
def test_attention_splits_long_contexts():
    # one unit over many SMs (joined in order), and many units of several SMs each
    _check_attention("bf16", rows=(1,), lens=(9000,), heads=2, kvh=1, page=64, hd=64)
    _check_attention("f16", rows=(2, 1, 1), lens=(3000, 10, 4100), heads=8, kvh=2, page=32)
    _check_attention("e4m3", "bf16", rows=(16,), lens=(5000,), heads=4, kvh=1, page=128)


@gpu
def test_attention_offsets_past_32_bits():
    """Pages whose byte offsets pass 2^32: a cache of 4.5 GB a tensor (one shared by k and v), its last pages read."""
    torch, dfl = _torch(), _dfl()
    n_pages, page, hd = 280000, 64, 128
    kc = torch.empty(n_pages, page, 1, hd, dtype=torch.bfloat16, device="cuda")
    kc.view(-1, 128)[:4096].fill_(float("nan"))
    rng = np.random.default_rng(0)
    tail = torch.from_numpy(rng.standard_normal((8, page, 1, hd)).astype(np.float32)).cuda().to(torch.bfloat16)
    kc[-8:] = tail
    ids = np.arange(n_pages - 8, n_pages)[rng.permutation(8)]
    q = torch.from_numpy(rng.standard_normal((2, 4, hd)).astype(np.float32)).cuda().to(torch.bfloat16)
    k = torch.from_numpy(rng.standard_normal((2, 1, hd)).astype(np.float32)).cuda().to(torch.bfloat16)
    dfl.paged_append(kc, kc, k, k, _i32(torch, ids[None]), _i32(torch, [500]))
    out = dfl.paged_attention(q, kc, kc, _i32(torch, ids[None]), _i32(torch, [500]))
    c = f64(kc[-8:])
    assert np.array_equal(c[ids[498 // 64] - (n_pages - 8), 498 % 64], f64(k)[0])
    ref, _, mag, _ = O.paged_attention(f64(q), c, c, [list(ids - (n_pages - 8))], [500])
    assert (np.abs(f64(out) - ref) <= HALF["bf16"] * np.abs(ref) + 1e-4 * mag).all()


@gpu
@pytest.mark.parametrize("kind,src", [("bf16", "bf16"), ("f16", "f16"), ("e4m3", "f16"), ("e4m3", "bf16")])
@pytest.mark.parametrize("rows", [1, 6, 20])
def test_attention_small_weights_in_sum(kind, src, rows):
    """One key far above thousands of equal ones that carry all of the output: weights of 2^-17.6, which a 16-bit float
    with five exponent bits holds to 7 bits alone, still come to their sum."""
    torch, dfl = _torch(), _dfl()
    T = _types()
    n, hd, heads = 4096, 64, 4
    q = torch.zeros(rows, heads, hd, device="cuda", dtype=T[src])
    q[:, :, 3] = 1.0
    kc = torch.zeros(n // 16, 16, 1, hd, device="cuda")
    kc[0, 0, 0, 3] = 16.0
    vc = 1.0 + torch.arange(hd, device="cuda").float().remainder(8).expand(n // 16, 16, 1, hd) / 8
    vc = vc.clone()
    vc[0, 0] = 0.0
    kc, vc = kc.to(T[kind]), vc.to(T[kind])
    table, scale = torch.arange(n // 16, device="cuda", dtype=torch.int32)[None], 12.2107 / 16
    out = dfl.paged_attention(q, kc, vc, table, _i32(torch, [n]), scale=scale)
    ref, _, mag, _ = O.paged_attention(f64(q), f64(kc), f64(vc), table.tolist(), [n], None, scale, 0)
    # scores: one product (exact), scaled: 2^-23 of 17.6 twice at most; one f16 P: half a step of it
    one_p = kind == "e4m3" and rows * heads > 16
    p_err = 2.0 ** -22 * 18 + 2.0 ** -20 + (HALF["f16"] if one_p else 0.0)
    assert (np.abs(f64(out) - ref) <= HALF[src] * np.abs(ref) + 2 * p_err * mag).all()


@gpu
@pytest.mark.parametrize("kind,src", [("bf16", "bf16"), ("f16", "f16"), ("e4m3", "bf16")])
@pytest.mark.parametrize("rows", [4, 16, 32])
def test_attention_many_units_of_several_tiles(kind, src, rows):
    # three units and more a CTA, none of them a single tile: what a CTA hands from unit to unit
    lens = tuple(260 + 13 * i for i in range(30))
    _check_attention(kind, src, hd=64, heads=64, kvh=16, rows=(rows,) * 30, lens=lens, uniform=True, seed=rows)


@gpu
def test_passes_from_two_threads_at_once():
    import threading
    torch, dfl = _torch(), _dfl()
    states = [_pass_state(torch, dfl, seed) for seed in (3, 4)]
    want = [_pass(dfl, st) for st in states]
    torch.cuda.synchronize()
    wrong = []

    def work(st, expect):
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(50):
                y, v = _pass(dfl, st)
                if not (torch.equal(y, expect[0]) and all(torch.equal(a, b) for a, b in zip(v, expect[1]))):
                    wrong.append(1)

    threads = [threading.Thread(target=work, args=x) for x in zip(states, want)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong


@gpu
def test_calls_keep_no_reference_to_their_arguments():
    import sys
    torch, dfl = _torch(), _dfl()
    st = _pass_state(torch, dfl)
    out, lse = torch.empty_like(st["q"]), torch.empty(12, 8, device="cuda")
    keep = dict(st, out=out, lse=lse)
    before = {k: sys.getrefcount(v) for k, v in keep.items()}
    for scale in (1.0, -1.0):  # served, refused
        for _ in range(5):
            try:
                dfl.paged_append(st["kc"], st["vc"], st["k"], st["v"], st["table"], st["lens"], row_start=st["start"],
                                 q=st["q"], q_out=out, inv_freq=st["f"], eps=scale, rope_scale=1.0)
                y = dfl.paged_attention(out, st["kc"], st["vc"], st["table"], st["lens"], row_start=st["start"],
                                        scale=scale, out=out, lse=lse)
                assert y is out
                del y
            except dfl.DFlashError:
                assert scale < 0
    made = dfl.paged_attention(st["q"], st["kc"], st["vc"], st["table"], st["lens"], row_start=st["start"])
    assert sys.getrefcount(made) == 2
    assert {k: sys.getrefcount(v) for k, v in keep.items()} == before


@gpu
def test_attention_out_in_place_of_q():
    torch, dfl = _torch(), _dfl()
    for heads in (4, 32):  # the warps' kernel, and the tensor memory's
        q = torch.randn(9, heads, 64, device="cuda", dtype=torch.bfloat16)
        kc, vc = (torch.randn(30, 16, 2, 64, device="cuda", dtype=torch.bfloat16) for _ in range(2))
        args = (kc, vc, torch.arange(30, device="cuda", dtype=torch.int32).reshape(3, 10), _i32(torch, [160, 3, 77]))
        want = dfl.paged_attention(q, *args)
        assert dfl.paged_attention(q, *args, out=q) is q and torch.equal(q, want)
        with pytest.raises(dfl.DFlashError, match="strides"):
            dfl.paged_attention(q, *args, out=q.flatten().as_strided((9, heads, 64), (64, 9 * 64, 1)))


@gpu
def test_attention_many_heads_of_one_and_an_empty_cache():
    # more query heads of a key/value head than rows of any tile
    _check_attention("bf16", heads=160, kvh=1, rows=(1, 1), lens=(70, 300), uniform=True)
    _check_attention("e4m3", "f16", hd=64, heads=200, kvh=1, rows=(2,), lens=(129,), uniform=True)
    torch, dfl = _torch(), _dfl()
    for heads in (4, 40):  # no page at all
        kc = torch.empty(0, 16, 2, 64, dtype=torch.bfloat16, device="cuda")
        q = torch.ones(2, heads, 64, dtype=torch.bfloat16, device="cuda")
        lse = torch.zeros(2, heads, device="cuda")
        for table in ([[0, -1], [5, 2 ** 31 - 1]], [[], []]):
            t = torch.tensor(table, dtype=torch.int32, device="cuda")
            out = dfl.paged_attention(q, kc, kc, t, _i32(torch, [20, 0]), lse=lse)
            assert (out == 0).all() and (lse == -float("inf")).all()
            dfl.paged_append(kc, kc, q[:, :2], q[:, :2], t, _i32(torch, [20, 0]))


@gpu
def test_passes_on_two_streams_at_once():
    torch, dfl = _torch(), _dfl()
    states = [_pass_state(torch, dfl, seed) for seed in (1, 2)]
    want = [_pass(dfl, st) for st in states]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in states]
    for _ in range(30):
        got = []
        for st, s in zip(states, streams):
            with torch.cuda.stream(s):
                got.append(_pass(dfl, st))
        torch.cuda.synchronize()
        for (y, v), (y2, v2) in zip(want, got):
            assert torch.equal(y, y2) and all(torch.equal(a, b) for a, b in zip(v, v2))
    # a stream by its handle, the default one's included
    for handle in (streams[0].cuda_stream, 0, torch.cuda.default_stream().cuda_stream):
        y = dfl.paged_attention(states[0]["q"], states[0]["kc"], states[0]["vc"], states[0]["table"], states[0]["lens"],
                                row_start=states[0]["start"], stream=handle)
        torch.cuda.synchronize()
        assert torch.equal(y, dfl.paged_attention(states[0]["q"], states[0]["kc"], states[0]["vc"], states[0]["table"],
                                                  states[0]["lens"], row_start=states[0]["start"]))


@gpu
def test_attention_repeats_bit_for_bit_and_on_another_stream():
    torch, dfl = _torch(), _dfl()
    rng = np.random.default_rng(0)
    kc, _ = _cached(torch, rng, (300, 16, 2, 128), "bf16")
    q = torch.from_numpy(rng.standard_normal((3, 8, 128)).astype(np.float32)).cuda().to(torch.bfloat16)
    table, lens = _i32(torch, rng.permutation(300).reshape(3, 100)), _i32(torch, [1600, 3, 777])
    a = dfl.paged_attention(q, kc, kc, table, lens)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    b = dfl.paged_attention(q, kc, kc, table, lens, stream=side.cuda_stream)
    with torch.cuda.stream(side):
        c = dfl.paged_attention(q, kc, kc, table, lens)
    side.synchronize()
    assert torch.equal(a, b) and torch.equal(a, c)
    need = dfl.paged_attention_workspace(q, kc, 3)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    assert torch.equal(a, dfl.paged_attention(q, kc, kc, table, lens, workspace=ws))
    with pytest.raises(dfl.DFlashError) as e:
        dfl.paged_attention(q, kc, kc, table, lens, workspace=ws[:need - 16])
    assert e.value.code == dfl._abi.DFLASH_ECAPACITY


# --------------------------------------------------------------------------- verification
def _check_verify(V=300, counts=(3, 0, 5), kind="f32", drawn=True, temperature=0.8, seed=0, uniform=False, extra=0,
                  sharp=2.0, edit=None, stride=0, temps=None):
    torch, dfl = _torch(), _dfl()
    rng = np.random.default_rng(seed)
    d, n = sum(counts), len(counts)
    D = d + extra
    seq = np.repeat(np.arange(n), counts)
    t = torch.full((D + n, V + stride), float("nan"), dtype=_types()[kind], device="cuda")[:, :V]
    t.copy_(torch.from_numpy(sharp * rng.standard_normal((D + n, V)).astype(np.float32)))
    base = f64(t)
    dl = np.zeros((D, V), np.float32)
    tok = np.zeros(D, np.uint32)
    for j in range(d):
        dl[j] = base[j + seq[j]] + 0.5 * rng.standard_normal(V)
        tok[j] = np.argmax(dl[j] / (temperature or 1.0) + rng.gumbel(size=V))
    dl_t, tok_t = torch.from_numpy(dl).cuda(), torch.from_numpy(tok.astype(np.int64)).cuda().to(torch.int32)
    au = torch.from_numpy(rng.random(D).astype(np.float32)).cuda()
    su = torch.from_numpy(rng.random(n).astype(np.float32)).cuda()
    temps = np.full(n, temperature, np.float32) if temps is None else np.asarray(temps, np.float32)
    if edit is not None:
        edit(torch, t, dl_t, tok_t, au, su)
    start = None if uniform else _starts(counts)
    acc, nxt, prob = (torch.full((m,), 77, dtype=y, device="cuda")
                      for m, y in ((n, torch.int32), (n, torch.int32), (D, torch.float32)))
    out = dfl.verify_drafts(t, tok_t, au, su, draft_logits=dl_t if drawn else None,
                            draft_start=None if uniform else _i32(torch, start),
                            temperature=torch.from_numpy(temps).cuda(), accepted=acc, next_token=nxt, prob=prob)
    torch.cuda.synchronize()
    assert out[0] is acc and out[1] is nxt and out[2] is prob
    toks = tok_t.cpu().numpy().astype(np.int64)
    toks = np.where(toks < 0, 2 ** 32 + toks, toks)
    res, pref = O.verify(f64(t), toks, f64(au), f64(su), f64(dl_t) if drawn else None, start, temps)
    got = list(zip(acc.tolist(), nxt.tolist()))
    for s, (a, x, margin) in enumerate(res):
        if margin > 1e-5:
            assert got[s] == (a, x), (s, got[s], (a, x), margin)
    gp = f64(prob)
    assert (gp[d:] == 77).all()
    assert (np.abs(gp[:d] - pref[:d]) <= 2e-6 * np.abs(pref[:d]) + 1e-37).all()
    return res, got


@gpu
@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("V", [1, 2, 7, 33, 300, 5003, 40001])
@pytest.mark.parametrize("drawn", [False, True])
def test_verify_vocabularies(kind, V, drawn):
    for seed in range(4):
        _check_verify(V, (3, 0, 5, 1), kind, drawn, seed=seed, stride=seed)


@gpu
@pytest.mark.parametrize("temperature", [0.0, 0.1, 1.0, 3.0, 1e-38, 1e35, float("inf"), float("nan"), -1.0])
@pytest.mark.parametrize("drawn", [False, True])
def test_verify_temperatures(temperature, drawn):
    for seed in range(3):
        _check_verify(1000, (4, 4), "f32", drawn, temperature=1.0, temps=(temperature, 0.7), uniform=True, seed=seed)


@gpu
def test_verify_many_shapes():
    accepted = set()
    for seed, counts in enumerate(itertools.islice(itertools.cycle([(16,), (0,), (0, 0), (31, 1), (1,) * 40, (7, 2, 9)]), 18)):
        for (a, _, _), c in zip(_check_verify(2000, counts, "bf16", seed % 2 == 0, seed=seed, extra=seed % 3 * 2)[0], counts):
            accepted.add((a == c, a == 0))
    assert len(accepted) == 4  # kept whole, refused at once, and between were all met


@gpu
def test_verify_greedy_ties_take_the_lowest_index():
    def edit(torch, t, dl, tok, au, su):
        t[:, 100] = 50.0
        t[:, 7] = 50.0
        t[:, 999] = 50.0
        tok[0], tok[1], tok[2] = 7, 100, 7
    res, got = _check_verify(1000, (3,), "f32", False, temperature=0.0, edit=edit)
    assert got[0] == (1, 7)


@gpu
def test_verify_masked_and_special_logits():
    inf, nan = float("inf"), float("nan")

    def rows(**at):
        def edit(torch, t, dl, tok, au, su):
            for r, f in at.items():
                f(torch, t[int(r[1:])], dl, tok)
        return edit

    for drawn in (False, True):
        for T in (0.0, 0.9):
            # most of the vocabulary masked; a row with nothing left; NaN; an infinite logit (two of them)
            _check_verify(500, (2, 2), "f32", drawn, T, edit=lambda torch, t, dl, tok, au, su: t[:, 3:].fill_(-inf))
            _check_verify(500, (2, 2), "bf16", drawn, T,
                          edit=lambda torch, t, dl, tok, au, su: t[:, ::2].fill_(torch.finfo(t.dtype).min))
            res, got = _check_verify(500, (2, 2), "f32", drawn, T, edit=rows(r0=lambda torch, r, dl, tok: r.fill_(-inf),
                                                                            r5=lambda torch, r, dl, tok: r.fill_(nan)))
            assert got[0] == (0, -1)
            _check_verify(500, (2, 2), "f32", drawn, T, edit=rows(r1=lambda torch, r, dl, tok: r[40:90].fill_(nan)))
            _check_verify(500, (2, 2), "f32", drawn, T, edit=rows(r0=lambda torch, r, dl, tok: r[8:301:292].fill_(inf)))
            # drafts outside the vocabulary, a drafter without probability, a draft the drafter could not make
            def odd(torch, t, dl, tok, au, su):
                tok[0], tok[3] = -1, 500
                dl[1] = -inf
                dl[2, int(tok[2])] = -inf
            _check_verify(500, (2, 2), "f32", drawn, T, edit=odd)
            # the drafter is the target: every draft stays; numbers of 0 and just under 1
            def same(torch, t, dl, tok, au, su):
                dl[0], dl[1], dl[2], dl[3] = t[0], t[1], t[3], t[4]
                au.fill_(1 - 2.0 ** -24)
                su[0], su[1] = 0.0, 1 - 2.0 ** -24
            res, got = _check_verify(500, (2, 2), "f32", drawn, T, edit=same)
            if drawn and T:
                assert [g[0] for g in got] == [2, 2]


@gpu
def test_verify_bad_starts_stay_inside():
    torch, dfl = _torch(), _dfl()
    rng = np.random.default_rng(0)
    n, d, V = 3, 6, 100
    t = torch.from_numpy(rng.standard_normal((n + d, V)).astype(np.float32)).cuda()
    tok = torch.from_numpy(rng.integers(0, V, d)).cuda().to(torch.int32)
    au, su = torch.rand(d, device="cuda"), torch.rand(n, device="cuda")
    for start in ([-5, 2, 4, 99], [6, 0, 6, 2], [0, 0, 0, 0], [6, 6, 6, 6], [3, 1, 2, 5]):
        acc, nxt, prob = dfl.verify_drafts(t, tok, au, su, draft_start=_i32(torch, start))
        torch.cuda.synchronize()
        a = acc.tolist()
        for s in range(n):
            lo = min(max(start[s], 0), d)
            hi = min(max(start[s + 1], lo), d)
            assert 0 <= a[s] <= hi - lo
        # rows of no sequence are not read into a sequence that is well formed
    res, _ = O.verify(f64(t), tok.tolist(), f64(au), f64(su))
    acc, nxt, _ = dfl.verify_drafts(t, tok, au, su)
    assert [(a, x) for a, x, _ in res] == list(zip(acc.tolist(), nxt.tolist()))


@gpu
def test_verify_samples_the_target_distribution():
    """Drafts from q, kept and resampled by the rule, are distributed as p whatever q is: the first tokens' counts over
    many sequences, against the probabilities (five standard deviations)."""
    torch, dfl = _torch(), _dfl()
    g = torch.Generator("cuda").manual_seed(0)
    n, V = 60000, 7
    p = torch.tensor([0.4, 0.2, 0.15, 0.1, 0.1, 0.05, 0.0], device="cuda")
    q = torch.tensor([0.1, 0.1, 0.3, 0.1, 0.1, 0.1, 0.2], device="cuda")
    draft = torch.multinomial(q, n, replacement=True, generator=g).to(torch.int32)
    t = p.log().expand(n, 2, V).reshape(2 * n, V).contiguous()
    acc, nxt, prob = dfl.verify_drafts(t, draft, torch.rand(n, device="cuda", generator=g),
                                       torch.rand(n, device="cuda", generator=g), draft_logits=q.log().expand(n, V).contiguous())
    first = torch.where(acc > 0, draft, nxt)
    share = torch.bincount(first.long(), minlength=V).double() / n
    assert (share[:V] - p).abs().max() < 5 * (0.25 / n) ** 0.5 and share[6] == 0


# --------------------------------------------------------------------------- together
def _pass(dfl, st, **kw):
    q = dfl.paged_append(st["kc"], st["vc"], st["k"], st["v"], st["table"], st["lens"], row_start=st["start"], q=st["q"],
                         inv_freq=st["f"], **kw)
    y = dfl.paged_attention(q, st["kc"], st["vc"], st["table"], st["lens"], row_start=st["start"], **kw)
    logits = y.flatten(1) @ st["head"]
    return y, dfl.verify_drafts(logits, st["tok"], st["au"], st["su"], draft_start=st["dstart"], **kw)


def _pass_state(torch, dfl, seed=0):
    rng = np.random.default_rng(seed)
    R = lambda *s: torch.from_numpy(rng.standard_normal(s).astype(np.float32)).cuda().to(torch.bfloat16)  # noqa: E731
    rows = (4, 1, 7)
    d = sum(rows) - 3
    st = dict(kc=R(40, 16, 2, 64), vc=R(40, 16, 2, 64), q=R(12, 8, 64), k=R(12, 2, 64), v=R(12, 2, 64), head=R(512, 700),
              table=_i32(torch, rng.permutation(39).reshape(3, 13)), lens=_i32(torch, (80, 7, 200)),
              start=_i32(torch, _starts(rows)), dstart=_i32(torch, _starts([r - 1 for r in rows])),
              tok=_i32(torch, rng.integers(0, 700, d)), f=dfl.rope_inv_freq(64, 1e4)[0],
              au=torch.from_numpy(rng.random(d).astype(np.float32)).cuda(),
              su=torch.from_numpy(rng.random(3).astype(np.float32)).cuda())
    return st


@gpu
def test_pass_together_matches_the_oracle():
    torch, dfl = _torch(), _dfl()
    st = _pass_state(torch, dfl)
    k0, v0 = f64(st["kc"]), f64(st["vc"])
    y, (acc, nxt, prob) = _pass(dfl, st)
    start, table, lens = st["start"].tolist(), st["table"].tolist(), st["lens"].tolist()
    slots, q, _ = O.paged_append(f64(st["k"]), f64(st["v"]), f64(st["q"]), table, lens, 16, 40, start, f64(st["f"].double()))
    for (p, s), (k, v) in slots.items():
        k0[p, s], v0[p, s] = k, v
    ref, _, mag, _ = O.paged_attention(q, k0, v0, table, lens, start)
    # q and k are rounded to bf16 on the way here (2^-8 each, of scores whose products sum to at most |q||k| / 8 = 12):
    # a probability moves by 2 * 12 * 2^-8 at most
    assert (np.abs(f64(y) - ref) <= HALF["bf16"] * np.abs(ref) + 24 * 2.0 ** -8 * mag).all()
    res, pref = O.verify(f64((y.flatten(1) @ st["head"])), st["tok"].tolist(), f64(st["au"]), f64(st["su"]), None,
                         st["dstart"].tolist())
    for s, (a, x, margin) in enumerate(res):
        if margin > 1e-5:
            assert (acc[s].item(), nxt[s].item()) == (a, x)


@gpu
def test_pass_captured_and_replayed_with_new_contents():
    """One captured pass replayed after its buffers' contents (rows, lengths, row starts, pages) changed equals a plain
    call on the same contents; two graphs that were given one workspace, replayed in turn, agree too."""
    torch, dfl = _torch(), _dfl()
    st, other = _pass_state(torch, dfl), _pass_state(torch, dfl, 5)
    keep = {k: v.clone() for k, v in st.items()}
    _pass(dfl, st)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y, v = _pass(dfl, st)
    for src in (keep, other, keep):
        for k in st:
            st[k].copy_(src[k])
        if src is other:
            st["start"].copy_(_i32(torch, (0, 2, 2, 12)))
            st["dstart"].copy_(_i32(torch, (0, 1, 1, 9)))
            st["lens"].copy_(_i32(torch, (3, 0, 208)))
        now = {k: x.clone() for k, x in st.items()}
        g.replay()
        torch.cuda.synchronize()
        y2, v2 = _pass(dfl, now)
        torch.cuda.synchronize()
        assert torch.equal(y, y2) and all(torch.equal(a, b) for a, b in zip(v, v2))
        assert torch.equal(st["kc"], now["kc"]) and torch.equal(st["vc"], now["vc"])
    ws = torch.empty(dfl.paged_attention_workspace(st["q"], st["kc"], 3), dtype=torch.uint8, device="cuda")
    outs, graphs = [], []
    for lens in ((80, 7, 200), (208, 208, 7)):
        gg, ln = torch.cuda.CUDAGraph(), _i32(torch, lens)
        with torch.cuda.graph(gg):
            o = dfl.paged_attention(st["q"], st["kc"], st["vc"], st["table"], ln, row_start=st["start"], workspace=ws)
        outs.append((o, ln))
        graphs.append(gg)
    for _ in range(3):
        for gg in graphs:
            gg.replay()
    torch.cuda.synchronize()
    for o, ln in outs:
        assert torch.equal(o, dfl.paged_attention(st["q"], st["kc"], st["vc"], st["table"], ln, row_start=st["start"]))


@gpu
def test_drafted_block_verified_end_to_end():
    """A drafter's block, its logits and tokens handed to the verification as they are."""
    torch, dfl = _torch(), _dfl()
    import workloads as W
    g = W.WORKLOADS["small_q4"].geom
    model = dfl.Model(g, W.make_weights(g))
    seqs = []
    for i in range(2):
        s = model.new_sequence(64)
        model.ctx_append(s, 0, W.make_taps(g, 20 + i, call_id=i))
        seqs.append(s)
    n, bl = 2, g.block
    logits = torch.empty(n, bl - 1, g.vocab, device="cuda")
    toks = torch.empty(n, bl - 1, dtype=torch.int32, device="cuda")
    model.block(seqs, _i32(torch, W.make_anchors(g, 2).astype(np.int64)), [20, 21], bl, logits=logits, tokens=toks)
    gen = torch.Generator("cuda").manual_seed(1)
    target = torch.cat((logits, torch.randn(n, 1, g.vocab, device="cuda", generator=gen)), 1)
    target[1, 4] = torch.randn(g.vocab, device="cuda", generator=gen) - 5
    target[1, 4, 17] = 100.0
    zero = torch.zeros(n, device="cuda")
    acc, nxt, prob = dfl.verify_drafts(target.flatten(0, 1), toks, torch.rand(n * (bl - 1), device="cuda", generator=gen),
                                       torch.rand(n, device="cuda", generator=gen), temperature=zero)
    # greedy, the target agreeing with the drafter: all kept; the second block is refused where its row was changed
    # (unless that draft was token 17 itself)
    assert acc.tolist() == [bl - 1, bl - 1 if toks[1, 4].item() == 17 else 4]
    assert nxt[0].item() == target[0, -1].argmax().item() and (toks[1, 4].item() == 17 or nxt[1].item() == 17)
    # drawn: q is the drafter's own distribution, so the unchanged rows keep every draft
    acc, nxt, prob = dfl.verify_drafts(target.flatten(0, 1), toks, torch.rand(n * (bl - 1), device="cuda", generator=gen),
                                       torch.rand(n, device="cuda", generator=gen), draft_logits=logits)
    assert acc[0].item() == bl - 1 and (prob[:bl - 1] == 1).all()
    for s in seqs:
        s.close()
    model.close()
