"""The target's verification pass: operators for a caller that runs the target model beside the drafter
(include/dflash.h, "The target's verification pass").

    logits, draft_tok = model.block(seqs, anchors, ...)            # the drafter's block
    for every target layer:
        q = paged_append(k_cache, v_cache, k, v, table, kv_len, q=q, inv_freq=f)
        y = paged_attention(q, k_cache, v_cache, table, kv_len)
    accepted, token, prob = verify_drafts(target_logits, draft_tok, u, v, draft_logits=logits)

A cache may be held in 4 bits (`k_block`, `v_block` in all of the paged calls) and cut back to the tokens that its
queries look at:

    y = paged_attention(q, k_cache, v_cache, table, kv_len, lse=lse)
    paged_key_weights(weights, q, k_cache, table, kv_len, lse)     # what each key received
    kv_len = paged_evict(k_cache, v_cache, weights, table, kv_len, keep, recent=64, evicted=evicted)
    q = paged_append(k_cache, v_cache, k, v, table, kv_len + rows, q=q, inv_freq=f, evicted=evicted)

Argument marshalling only: every step runs in the library's kernels.  Arguments are torch CUDA tensors of one device
(any, current or not); calls run on that device's current stream, or on the stream whose handle is given.  A call may
be captured into a CUDA graph; outputs and workspaces that it allocates then belong to the graph's memory.
"""
from __future__ import annotations

import ctypes as C
import math

import numpy as np

from . import _abi

torch = _binding = None


def _init():
    """torch, the library and the compiled half of this module (csrc/binding.cpp), on the first call."""
    global torch, _binding
    import torch as t

    from . import DFlashError, lib
    try:
        from . import _binding as b
    except ImportError as e:
        raise ImportError(f"the binding is not built, or not for this torch; run __graft_entry__.build() or "
                          f"python -m block_speculative_drafting_gb300.csrc.build ({e})") from e
    L = lib()
    names = ("dflash_paged_append_at", "dflash_paged_attention", "dflash_paged_attention_workspace", "dflash_verify",
             "dflash_verify_workspace", "dflash_last_error", "dflash_paged_read", "dflash_paged_key_weights",
             "dflash_paged_evict", "dflash_paged_evict_workspace")
    b.init(tuple(C.cast(getattr(L, n), C.c_void_p).value for n in names), DFlashError,
           t.cuda.OutOfMemoryError)
    torch, _binding = t, b


def _check(rc: int) -> int:
    if rc < 0:
        from . import DFlashError, lib
        raise DFlashError(rc, lib().dflash_last_error(None).decode())
    return rc


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
                 k_scale=None, v_scale=None, k_block=None, v_block=None, evicted=None, stream=None):
    """Write a pass's keys and values into a paged cache, normed and rotated on the way, and return its rotated
    queries (None without q).

    k_cache, v_cache  [pages][page_size][kv_heads][head_dim] bfloat16, float16 or float8_e4m3fn, any strides with
                      contiguous columns; k_scale, v_scale [kv_heads] float32: an 8-bit element is code * scale.
                      Or in 4 bits: uint8 (or float4_e2m1fn_x2) [..][head_dim / 2], two e2m1 codes a byte, the first in
                      the lower bits, with k_block, v_block float8_e4m3fn [pages][page_size][kv_heads][head_dim / 16]:
                      an element is code * block scale * head's scale
    k, v, q           [rows][heads][head_dim] of one type: float32, bfloat16 or float16 (slices of a fused projection
                      fit)
    table             int32 [sequences][pages]; a page id outside the cache: not held, not written
    kv_len            int32 [sequences]: tokens in each sequence's cache with its new rows in; row i of its r rows
                      stands at position kv_len - r + i
    row_start         int32 [sequences + 1]: each sequence's rows; None: equally many
    q_out             where the queries go (default: a new, contiguous tensor of q's shape and type; q itself is allowed)
    inv_freq          float64 [rotary / 2] (`rope_inv_freq`); None: no rotation.  Pairs are columns (i, i + rotary/2),
                      or (2i, 2i + 1) when interleaved; columns from `rotary` on stay
    q_norm, k_norm    float32 [head_dim] gains of an RMS norm before the rotation; None: none
    evicted           int32 [sequences]: tokens that `paged_evict` has taken out of each sequence's cache; a row is
                      rotated as the position of its slot + evicted (None: 0)
    """
    if torch is None:
        _init()
    return _binding.paged_append(k_cache, v_cache, k, v, table, kv_len, row_start, q, q_out, inv_freq, interleaved,
                                 rope_scale, q_norm, k_norm, eps, k_scale, v_scale, stream, k_block, v_block, evicted)


def paged_read(k_cache, v_cache, table, kv_len, rows: int, *, row_start=None, k_scale=None, v_scale=None, k_block=None,
               v_block=None, dtype=None, k_out=None, v_out=None, stream=None):
    """The keys and values that a paged cache holds for `rows` rows in all, as values: returns (k, v)
    [rows][kv_heads][head_dim] of `dtype` (float32, bfloat16 or float16; None: that of k_out or v_out, without them float16
    from a float16 cache, else bfloat16).  Rows are `paged_append`'s: the last ones of each sequence (all of them with row_start = the running sum
    of kv_len).  Positions that are not held read as zeros.  k_out, v_out: where they go, of any row and head strides.
    The other arguments are `paged_append`'s.
    """
    if torch is None:
        _init()
    given = k_out if k_out is not None else v_out
    if dtype is None and given is not None:
        dtype = given.dtype
    return _binding.paged_read(k_cache, v_cache, table, kv_len, rows, row_start, k_scale, v_scale, k_block, v_block, dtype,
                               k_out, v_out, stream)


def paged_attention(q, k_cache, v_cache, table, kv_len, *, row_start=None, scale: float | None = None, window: int = 0,
                    k_scale=None, v_scale=None, k_block=None, v_block=None, out=None, lse=None, workspace=None,
                    stream=None):
    """Attention of a pass's rows over the paged cache, which holds their own keys and values (`paged_append`):
    returns out [rows][heads][head_dim] in q's type.

    q          [rows][heads][head_dim] of the cache's type (bfloat16 or float16 for an 8-bit or 4-bit cache); query head h
               reads key/value head h / (heads / kv_heads)
    scale      of the scores; None: head_dim ** -0.5
    window     > 0: the row at position p sees the positions p - window + 1 .. p; 0: all up to p
    out        where the result goes (default: a new, contiguous tensor of q's shape and type; q itself is allowed)
    lse        float32 [rows][heads] to fill with ln sum exp of the row's scores (-inf: the row sees nothing)
    workspace  uint8 tensor of `paged_attention_workspace` bytes for callers that may not allocate (calls that may
               overlap need one each); None: allocated for the call
    The other arguments are `paged_append`'s.
    """
    if torch is None:
        _init()
    return _binding.paged_attention(q, k_cache, v_cache, table, kv_len, row_start, scale, window, k_scale, v_scale, out,
                                    lse, workspace, stream, k_block, v_block)


def paged_attention_workspace(q, k_cache, n_seqs: int) -> int:
    """Bytes of workspace that `paged_attention` needs for q's rows over n_seqs sequences."""
    if torch is None:
        _init()
    from . import lib
    n, page, heads, hd = k_cache.shape
    kind = {torch.bfloat16: _abi.BF16, torch.float16: _abi.F16, torch.float8_e4m3fn: _abi.E4M3, torch.uint8: _abi.E2M1,
            torch.float4_e2m1fn_x2: _abi.E2M1}.get(k_cache.dtype, -1)
    c = _abi.PagedCache(None, None, kind, heads, 2 * hd if kind == _abi.E2M1 else hd, page, 0)
    if not q.is_cuda:
        from . import DFlashError
        raise DFlashError(_abi.DFLASH_EINVAL, "tensors have to be on a CUDA device")
    with torch.cuda.device(q.get_device()):
        return _check(lib().dflash_paged_attention_workspace(C.byref(c), n_seqs, q.shape[0], q.shape[1]))


def paged_key_weights(weights, q, k_cache, table, kv_len, lse, *, row_start=None, scale: float | None = None,
                      window: int = 0, k_scale=None, k_block=None, stream=None):
    """Add the attention weight that each cached key receives from a pass's rows to `weights`, and return them:
    weights[s][h][j] += sum of exp(scale q . k_j - lse) over the rows that see position j and the query heads that share
    key/value head h.  A position that the pass itself brings starts at 0, whatever weights held there.

    weights    float32 [sequences][kv_heads][positions], a position for each that the table names at least; any strides
               with contiguous positions
    lse        float32 [rows][heads], `paged_attention`'s for the same rows, scale and window
    The other arguments are `paged_attention`'s.  Equal calls give equal bits.
    """
    if torch is None:
        _init()
    return _binding.paged_key_weights(weights, q, k_cache, table, kv_len, lse, row_start, scale, window, k_scale, k_block,
                                      stream)


def paged_evict(k_cache, v_cache, weights, table, kv_len, keep: int, *, first: int = 0, recent: int = 0, k_block=None,
                v_block=None, weights_out=None, new_len=None, kept=None, evicted=None, workspace=None, stream=None):
    """Cut every sequence that holds more than `keep` tokens back to that many, and return the new lengths (int32
    [sequences]).  Each key/value head keeps the `first` first tokens, the `recent` last ones and, of those between, the
    ones with the largest weights (equal ones: the lowest position; NaN counts as -inf).  They move, in order, to the
    first `keep` positions of the same pages: keys, values, block scales and weights.

    weights      float32 [sequences][kv_heads][positions] (`paged_key_weights`); weights_out: where they go (default:
                 they move in their place)
    new_len      where the new lengths go (default: a new tensor; kv_len itself is allowed)
    kept         int32 [sequences][kv_heads][keep] to fill with the position that each token had (-1: no token)
    evicted      int32 [sequences] that grows by the number of tokens taken out, for `paged_append`
    workspace    uint8 tensor of `paged_evict_workspace` bytes (calls that may overlap need one each); None: allocated
    No page may hold tokens of two sequences, and k_cache and v_cache, as k_block and v_block, are apart.  Cached keys
    keep their rotation, so a window over an evicted cache counts the tokens that are left.
    """
    if torch is None:
        _init()
    return _binding.paged_evict(k_cache, v_cache, weights, table, kv_len, keep, first, recent, k_block, v_block,
                                weights_out, new_len, kept, evicted, workspace, stream)


def paged_evict_workspace(n_seqs: int, kv_heads: int, keep: int, kept: bool = False) -> int:
    """Bytes of workspace that `paged_evict` needs; kept: whether the call is given that tensor."""
    from . import lib
    return _check(lib().dflash_paged_evict_workspace(n_seqs, kv_heads, keep, 0 if kept else 1))


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
    without any probability yields token -1.  Outputs and workspace may be given (`verify_workspace`); masked logits,
    drafts outside the vocabulary and bad starts: include/dflash.h, dflash_verify.
    """
    if torch is None:
        _init()
    return _binding.verify_drafts(target_logits, draft_tokens, accept_u, sample_u, draft_logits, draft_start, temperature,
                                  accepted, next_token, prob, workspace, stream)


def verify_workspace(n_seqs: int, n_drafts: int, vocab: int) -> int:
    """Bytes of workspace that `verify_drafts` needs on the current device."""
    from . import lib
    return _check(lib().dflash_verify_workspace(n_seqs, n_drafts, vocab))
