"""The target's verification pass: operators for a caller that runs the target model beside the drafter
(include/dflash.h, "The target's verification pass").

    logits, draft_tok = model.block(seqs, anchors, ...)            # the drafter's block
    for every target layer:
        q = paged_append(k_cache, v_cache, k, v, table, kv_len, q=q, inv_freq=f)
        y = paged_attention(q, k_cache, v_cache, table, kv_len)
    accepted, token, prob = verify_drafts(target_logits, draft_tok, u, v, draft_logits=logits)

Argument marshalling only: every step runs in the library's kernels.  Arguments are torch CUDA tensors of one device
(any, current or not); calls run on that device's current stream, or on the stream whose handle is given.  A call may
be captured into a CUDA graph; outputs and workspaces that it allocates then belong to the graph's memory.
"""
from __future__ import annotations

import contextlib
import ctypes as C
import math

import numpy as np

from . import _abi

# The calls below run once a layer and step, so what they do on the host is kept to some ten microseconds: the C
# descriptors are packed in one go, attributes are asked for once, the library and torch are looked up once.
torch = None
_lib = None
_DTYPES: dict = {}
_current_device = _raw_stream = None


def _init():
    global torch, _lib, _current_device, _raw_stream
    import torch as t

    from . import lib
    _lib = lib()
    _DTYPES.update({t.float32: _abi.F32, t.bfloat16: _abi.BF16, t.float16: _abi.F16, t.float8_e4m3fn: _abi.E4M3})
    _current_device = t.cuda.current_device
    _raw_stream = getattr(t._C, "_cuda_getCurrentRawStream", None) or (lambda d: t.cuda.current_stream(d).cuda_stream)
    torch = t


def _check(rc: int) -> int:
    if rc < 0:
        from . import DFlashError
        raise DFlashError(rc, _lib.dflash_last_error(None).decode())
    return rc


def _refuse(msg: str):
    from . import DFlashError
    raise DFlashError(_abi.DFLASH_EINVAL, msg)


def _direct(dev: int, stream) -> bool:
    """Whether a call can run where it stands: on the current device, on its current stream."""
    if dev < 0:
        _refuse("tensors have to be on a CUDA device")
    return stream is None and dev == _current_device()


@contextlib.contextmanager
def _moved(dev: int, stream):
    """The call's device and stream made current.  (What a call allocates belongs to the stream that is current, so
    that it is not dealt out again before that stream is done with it.)"""
    with torch.cuda.device(dev):
        if stream is None:
            yield
        else:
            with torch.cuda.stream(torch.cuda.ExternalStream(int(stream), device=dev)):
                yield


def _same_device(dev: int, *tensors):
    for t in tensors:
        if t is not None and t.get_device() != dev:
            _refuse(f"a tensor of shape {tuple(t.shape)} is on {t.device}, not on cuda:{dev}")


def _vector(t, name: str, n: int, dtype) -> int:
    """Pointer of a contiguous vector of n elements (None: 0)."""
    if t is None:
        return 0
    if t.dtype is not dtype or t.shape != (n,) or (n > 1 and t.stride(0) != 1):
        _refuse(f"{name} has to be a contiguous vector of {n} elements of {dtype}, got {tuple(t.shape)} of {t.dtype}")
    return t.data_ptr()


def _head_rows(t, name: str, n: int, hd: int, written: bool = False) -> bytes:
    """A [n][heads][hd] tensor as a dflash_head_rows (a type it has no code for: -1, which the library refuses)."""
    shape = t.shape
    if len(shape) != 3 or shape[0] != n or shape[2] != hd:
        _refuse(f"{name} has to be [{n}][heads][{hd}], got {tuple(shape)}")
    h = shape[1]
    sr, sh, sc = t.stride()
    if sc != 1:
        _refuse(f"{name} needs contiguous columns")
    if n <= 1:  # the stride of a dimension of one element is anything
        sr = 0
    elif written and sr == 0:
        _refuse(f"{name} is written and may not be an expanded tensor")
    if h <= 1:
        sh = 0
    elif written and sh == 0:
        _refuse(f"{name} is written and may not be an expanded tensor")
    return _HEAD_ROWS(t.data_ptr(), _DTYPES.get(t.dtype, -1), h, sr, sh)


_HEAD_ROWS, _PAGED_CACHE, _PAGED_ROWS = _abi.HEAD_ROWS.pack, _abi.PAGED_CACHE.pack, _abi.PAGED_ROWS.pack


def _cache(k, v, shape, k_scale, v_scale, written: bool = False) -> bytes:
    """The two cache tensors, k of the given shape, as a dflash_paged_cache."""
    if len(shape) != 4 or v.shape != shape or v.dtype is not k.dtype:
        _refuse("k_cache and v_cache have to be [pages][page_size][kv_heads][head_dim] of one shape and type, got "
                f"{tuple(shape)} of {k.dtype} and {tuple(v.shape)} of {v.dtype}")
    n, page, heads, hd = shape
    k0, k1, k2, k3 = k.stride()
    v0, v1, v2, v3 = v.stride()
    if k3 != 1 or v3 != 1:
        _refuse("k_cache and v_cache need contiguous columns")
    if n <= 1 or page <= 1 or heads <= 1:  # the stride of a dimension of one element is anything
        k0, v0 = (0, 0) if n <= 1 else (k0, v0)
        k1, v1 = (0, 0) if page <= 1 else (k1, v1)
        k2, v2 = (0, 0) if heads <= 1 else (k2, v2)
    if written and not (k0 and k1 and k2 and v0 and v1 and v2) and (
            n > 1 and not (k0 and v0) or page > 1 and not (k1 and v1) or heads > 1 and not (k2 and v2)):
        _refuse("k_cache and v_cache are written and may not be expanded tensors")
    ks = vs = 0
    if k_scale is not None or v_scale is not None:
        ks = _vector(k_scale, "k_scale", heads, torch.float32)
        vs = _vector(v_scale, "v_scale", heads, torch.float32)
    return _PAGED_CACHE(k.data_ptr(), v.data_ptr(), _DTYPES.get(k.dtype, -1), heads, hd, page, n, k0, k1, k2, v0, v1,
                        v2, ks, vs)


def _rows(table, kv_len, row_start, n_rows: int) -> bytes:
    i32, shape = torch.int32, table.shape
    if table.dtype is not i32 or len(shape) != 2 or (shape[1] > 1 and table.stride(1) != 1):
        _refuse(f"table has to be int32 [sequences][pages] with contiguous rows, got {tuple(shape)} of {table.dtype}")
    n, width = shape
    return _PAGED_ROWS(n, width, n_rows, 0 if row_start is None else _vector(row_start, "row_start", n + 1, i32),
                       _vector(kv_len, "kv_len", n, i32), table.data_ptr(), table.stride(0) if n > 1 else width)


def rope_inv_freq(rotary: int, theta: float = 1e6, scaling: str | None = None, factor: float = 1.0,
                  trained: int | None = None, beta_fast: float = 32.0, beta_slow: float = 1.0, device=None):
    """Rotation frequencies for `paged_append` and the scale that goes with them: (float64 [rotary/2] tensor, scale).

    theta^(-2i/rotary), and for contexts `factor` times longer than trained
      "linear"  every frequency / factor
      "yarn"    frequencies that turn fewer than beta_slow times in `trained` positions / factor, those that turn more
                than beta_fast times as they are, a linear ramp over the pairs between; scale 0.1 ln(factor) + 1
    """
    if torch is None:
        _init()
    if rotary < 2 or rotary % 2 or not theta > 0 or not factor > 0:
        raise ValueError(f"rotary {rotary}, theta {theta}, factor {factor}")
    f = theta ** (-np.arange(0, rotary, 2, dtype=np.float64) / rotary)
    scale = 1.0
    if scaling == "linear":
        f = f / factor
    elif scaling == "yarn":
        if not trained or trained < 1:
            raise ValueError("yarn needs the trained length")

        def pair(turns):  # the pair that turns so many times in `trained` positions
            return rotary * math.log(trained / (turns * 2 * math.pi)) / (2 * math.log(theta))

        lo, hi = max(math.floor(pair(beta_fast)), 0), min(math.ceil(pair(beta_slow)), rotary - 1)
        ramp = np.clip((np.arange(rotary // 2) - lo) / max(hi - lo, 1e-3), 0.0, 1.0)
        f = f / factor * ramp + f * (1.0 - ramp)
        scale = 0.1 * math.log(factor) + 1.0 if factor > 1 else 1.0
    elif scaling is not None:
        raise ValueError(f"scaling {scaling!r} is not linear or yarn")
    return torch.from_numpy(f).to(device if device is not None else "cuda"), scale


def paged_append(k_cache, v_cache, k, v, table, kv_len, *, row_start=None, q=None, q_out=None, inv_freq=None,
                 interleaved: bool = False, rope_scale: float = 1.0, q_norm=None, k_norm=None, eps: float = 1e-6,
                 k_scale=None, v_scale=None, stream=None):
    """Write a pass's keys and values into a paged cache, normed and rotated on the way, and return its rotated
    queries (None without q).

    k_cache, v_cache  [pages][page_size][kv_heads][head_dim] bfloat16, float16 or float8_e4m3fn, any strides with
                      contiguous columns; k_scale, v_scale [kv_heads] float32: an 8-bit element is code * scale
    k, v, q           [rows][heads][head_dim] of one type: float32, bfloat16 or float16 (slices of a fused projection
                      fit)
    table             int32 [sequences][pages]; a page id outside the cache: not held, not written
    kv_len            int32 [sequences]: tokens in each sequence's cache with its new rows in; row i of its r rows
                      stands at position kv_len - r + i
    row_start         int32 [sequences + 1]: each sequence's rows; None: equally many
    q_out             where the queries go (default: a new tensor like q; q itself is allowed)
    inv_freq          float64 [rotary / 2] (`rope_inv_freq`); None: no rotation.  Pairs are columns (i, i + rotary/2),
                      or (2i, 2i + 1) when interleaved; columns from `rotary` on stay
    q_norm, k_norm    float32 [head_dim] gains of an RMS norm before the rotation; None: none
    """
    if torch is None:
        _init()
    dev = k_cache.get_device()
    if not _direct(dev, stream):
        with _moved(dev, stream):
            return paged_append(k_cache, v_cache, k, v, table, kv_len, row_start=row_start, q=q, q_out=q_out,
                                inv_freq=inv_freq, interleaved=interleaved, rope_scale=rope_scale, q_norm=q_norm,
                                k_norm=k_norm, eps=eps, k_scale=k_scale, v_scale=v_scale)
    _same_device(dev, v_cache, k, v, table, kv_len, row_start, q, q_out, inv_freq, q_norm, k_norm, k_scale, v_scale)
    shape, n = k_cache.shape, k.shape[0] if k.dim() else 0
    cache = _cache(k_cache, v_cache, shape, k_scale, v_scale, True)
    kv_heads, hd = shape[2], shape[3]
    kr, vr = _head_rows(k, "k", n, hd), _head_rows(v, "v", n, hd)
    qr = qo = rot = None
    if inv_freq is not None:
        f = inv_freq.numel()
        rot = _abi.ROTATION.pack(_vector(inv_freq, "inv_freq", f, torch.float64), 2 * f, 1 if interleaved else 0,
                                 rope_scale)
    if q is not None:
        qr = _head_rows(q, "q", n, hd)
        if q_out is None:
            q_out = torch.empty_like(q, memory_format=torch.contiguous_format)
        elif q_out.shape != q.shape:
            _refuse(f"q_out has to be {tuple(q.shape)}, got {tuple(q_out.shape)}")
        qo = _head_rows(q_out, "q_out", n, hd, True)
    elif q_out is not None:
        _refuse("q_out without q")
    qn = kn = 0
    if q_norm is not None:
        qn = _vector(q_norm, "q_norm", hd, torch.float32)
    if k_norm is not None:
        kn = _vector(k_norm, "k_norm", hd, torch.float32)
    rc = _lib.dflash_paged_append(cache, _rows(table, kv_len, row_start, n), kr, vr, qr, qo, qn, kn, eps, rot,
                                  _raw_stream(dev))
    if rc < 0:
        _check(rc)
    return q_out


def paged_attention(q, k_cache, v_cache, table, kv_len, *, row_start=None, scale: float | None = None, window: int = 0,
                    k_scale=None, v_scale=None, out=None, lse=None, workspace=None, stream=None):
    """Attention of a pass's rows over the paged cache, which holds their own keys and values (`paged_append`):
    returns out [rows][heads][head_dim] in q's type.

    q          [rows][heads][head_dim] of the cache's type (bfloat16 or float16 for an 8-bit cache); query head h
               reads key/value head h / (heads / kv_heads)
    scale      of the scores; None: head_dim ** -0.5
    window     > 0: the row at position p sees the positions p - window + 1 .. p; 0: all up to p
    lse        float32 [rows][heads] to fill with ln sum exp of the row's scores (-inf: the row sees nothing)
    workspace  uint8 tensor of `paged_attention_workspace` bytes for callers that may not allocate (calls that may
               overlap need one each); None: allocated for the call
    The other arguments are `paged_append`'s.
    """
    if torch is None:
        _init()
    dev = q.get_device()
    if not _direct(dev, stream):
        with _moved(dev, stream):
            return paged_attention(q, k_cache, v_cache, table, kv_len, row_start=row_start, scale=scale, window=window,
                                   k_scale=k_scale, v_scale=v_scale, out=out, lse=lse, workspace=workspace)
    _same_device(dev, k_cache, v_cache, table, kv_len, row_start, k_scale, v_scale, out, lse, workspace)
    shape, qshape = k_cache.shape, q.shape
    cache = _cache(k_cache, v_cache, shape, k_scale, v_scale)
    if len(qshape) != 3:
        _refuse(f"q has to be [rows][heads][head_dim], got {tuple(qshape)}")
    n, heads, hd = qshape[0], qshape[1], shape[3]
    qr, rows = _head_rows(q, "q", n, hd), _rows(table, kv_len, row_start, n)
    if lse is not None and (lse.dtype is not torch.float32 or lse.shape != (n, heads) or not lse.is_contiguous()):
        _refuse(f"lse has to be contiguous float32 [{n}][{heads}]")
    if out is None:
        out = torch.empty_like(q, memory_format=torch.contiguous_format)
    elif out.shape != qshape:
        _refuse(f"out has to be {tuple(qshape)}, got {tuple(out.shape)}")
    if workspace is None:
        need = _check(_lib.dflash_paged_attention_workspace(cache, table.shape[0], n, heads))
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    else:
        if not workspace.is_contiguous():
            _refuse("workspace has to be contiguous")
        need = workspace.nbytes
    rc = _lib.dflash_paged_attention(cache, rows, qr, _head_rows(out, "out", n, hd, True),
                                     0 if lse is None else lse.data_ptr(), hd ** -0.5 if scale is None else scale,
                                     window, workspace.data_ptr(), need, _raw_stream(dev))
    if rc < 0:
        _check(rc)
    return out


def paged_attention_workspace(q, k_cache, n_seqs: int) -> int:
    """Bytes of workspace that `paged_attention` needs for q's rows over n_seqs sequences."""
    if torch is None:
        _init()
    dev = q.get_device()
    if not _direct(dev, None):
        with _moved(dev, None):
            return paged_attention_workspace(q, k_cache, n_seqs)
    cache = _cache(k_cache, k_cache, k_cache.shape, None, None)
    return _check(_lib.dflash_paged_attention_workspace(cache, n_seqs, q.shape[0], q.shape[1]))


def verify_drafts(target_logits, draft_tokens, accept_u, sample_u, *, draft_logits=None, draft_start=None,
                  temperature=None, accepted=None, next_token=None, prob=None, workspace=None, stream=None):
    """Which drafted tokens the target keeps, and the token after them, from given random numbers: returns
    (accepted int32 [sequences], next_token int32 [sequences], prob float32 [drafts]).

    target_logits  [drafts + sequences][vocab] float32, bfloat16 or float16: sequence by sequence, a row for each
                   draft and one for the token after them all
    draft_tokens   int32 or uint32, `Model.block`'s tokens as they are ([sequences][drafts]) or [drafts]
    accept_u       float32 [drafts], sample_u float32 [sequences], uniform in [0, 1)
    draft_logits   float32 [..][vocab], a row a draft, `Model.block`'s logits as they are: drafts drawn from their
                   softmax; None: drafts that were chosen, not drawn (a draft stays with probability p(draft))
    draft_start    int32 [sequences + 1]: each sequence's drafts; None: equally many
    temperature    float32 [sequences], 0: greedy; None: 1 for all
    A draft stays while accept_u * q(draft) < p(draft); the next token comes from max(p - q, 0) of the first refused
    draft's row, or from p of the last row, at the running sum that passes sample_u.  prob is min(1, p / q).  A row
    without any probability yields token -1.  Sequences are refused or served alike: include/dflash.h, dflash_verify.
    """
    if torch is None:
        _init()
    dev = target_logits.get_device()
    if not _direct(dev, stream):
        with _moved(dev, stream):
            return verify_drafts(target_logits, draft_tokens, accept_u, sample_u, draft_logits=draft_logits,
                                 draft_start=draft_start, temperature=temperature, accepted=accepted,
                                 next_token=next_token, prob=prob, workspace=workspace)
    _same_device(dev, draft_tokens, accept_u, sample_u, draft_logits, draft_start, temperature, accepted, next_token,
                 prob, workspace)
    f32, i32 = torch.float32, torch.int32
    if target_logits.dim() != 2:
        _refuse(f"target_logits has to be [rows][vocab], got {tuple(target_logits.shape)}")
    n, d, (rows, vocab), (stride, one) = sample_u.numel(), draft_tokens.numel(), target_logits.shape, target_logits.stride()
    if one != 1 and vocab > 1:
        _refuse("target_logits needs contiguous rows")
    if rows != n + d:
        _refuse(f"{d} drafts of {n} sequences need {n + d} target rows, got {rows}")
    if draft_tokens.dtype is not i32 and draft_tokens.dtype is not torch.uint32 or not draft_tokens.is_contiguous():
        _refuse(f"draft_tokens has to be contiguous int32 or uint32, got {draft_tokens.dtype}")
    dl, ds = None, 0
    if draft_logits is not None:
        if draft_logits.dtype is not f32 or draft_logits.shape[-1] != vocab or draft_logits.numel() != d * vocab:
            _refuse(f"draft_logits has to be float32 [{d}][{vocab}], got {tuple(draft_logits.shape)}")
        if draft_logits.dim() == 2 and (vocab == 1 or draft_logits.stride(1) == 1):
            ds = draft_logits.stride(0) if d > 1 else vocab
        elif draft_logits.is_contiguous():
            ds = vocab
        else:
            _refuse("draft_logits needs contiguous rows (more than two dimensions: contiguous as a whole)")
        dl = draft_logits.data_ptr()
    if accepted is None:
        accepted = torch.empty(n, dtype=i32, device=target_logits.device)
    if next_token is None:
        next_token = torch.empty_like(accepted)
    if prob is None:
        prob = torch.empty_like(accept_u, memory_format=torch.contiguous_format)
    if workspace is None:
        need = _check(_lib.dflash_verify_workspace(n, d, vocab))
        workspace = torch.empty(need, dtype=torch.uint8, device=target_logits.device)
    else:
        if not workspace.is_contiguous():
            _refuse("workspace has to be contiguous")
        need = workspace.nbytes
    rc = _lib.dflash_verify(
        target_logits.data_ptr(), _DTYPES.get(target_logits.dtype, -1), stride if rows > 1 else vocab, dl, ds,
        draft_tokens.data_ptr(), _vector(draft_start, "draft_start", n + 1, i32),
        _vector(temperature, "temperature", n, f32), _vector(accept_u, "accept_u", d, f32),
        _vector(sample_u, "sample_u", n, f32), n, d, vocab, _vector(accepted, "accepted", n, i32),
        _vector(next_token, "next_token", n, i32), _vector(prob, "prob", d, f32), workspace.data_ptr(), need,
        _raw_stream(dev))
    if rc < 0:
        _check(rc)
    return accepted, next_token, prob


def verify_workspace(n_seqs: int, n_drafts: int, vocab: int) -> int:
    """Bytes of workspace that `verify_drafts` needs on the current device."""
    if torch is None:
        _init()
    return _check(_lib.dflash_verify_workspace(n_seqs, n_drafts, vocab))
