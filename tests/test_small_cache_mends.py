"""Calls around a target's small cache that once answered wrongly or were never made by a test."""
import ctypes as C

import pytest

from test_target_ops import _cache_struct, _dfl, _rows_struct, _torch
from test_target_small_cache import _cache4, _good, _weights_struct

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
