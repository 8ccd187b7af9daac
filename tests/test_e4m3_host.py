"""Refusals of the 8-bit cache's operators and of the adjusted logits: arguments are
checked on the host before anything is enqueued, so none of this needs a GPU."""
import ctypes

import pytest
import torch

from block_diffusion_speculative_kv_gb300 import binding, build
from test_paged_host import BAD_PAGES

P = ctypes.c_void_p(64)        # never dereferenced: every call is rejected first


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.lib()


def _pages(k=64, v=64, ks=1, vs=1, table=64, table_ld=4, n_pages=10, page=16, n_kv=2, hd=128):
    return ctypes.byref(binding.PagesE4M3Struct(k, v, ks, vs, table, table_ld, n_pages, page, n_kv, hd))


def _append(lib, pages, n_req=1, n_rows=4, off=P, pos0=P, pos=None, dtype=1, k=P, v=P, ld=256, theta=1e6):
    return lib.dflash_paged_append_e4m3(pages, n_req, n_rows, off, pos0, pos, dtype, k, v, ld, theta, None)


def _attn(lib, pages, n_req=1, n_rows=4, n_q=8, off=P, pos0=P, max_rows=4, q=P, q_ld=1024, mask=None,
          mask_ld=0, out=P, out_ld=1024, ws=None, ws_bytes=0):
    return lib.dflash_paged_attention_e4m3(pages, n_req, n_rows, n_q, off, pos0, max_rows, q, q_ld, mask, mask_ld,
                                           out, out_ld, ws, ws_bytes, None)


@pytest.mark.parametrize("bad", [b for b in BAD_PAGES if "dtype" not in b] + [dict(ks=0), dict(vs=0)])
def test_bad_pages(lib, bad):
    assert _append(lib, _pages(**bad)) == 1
    assert _attn(lib, _pages(**bad)) == 1
    assert b"e4m3" in lib.dflash_last_error()


def test_append_refusals(lib):
    ok = _pages()
    assert _append(lib, None) == 1
    assert _append(lib, ok, n_req=-1) == 1 and _append(lib, ok, n_rows=-1) == 1
    assert _append(lib, ok, ld=255) == 1 and _append(lib, ok, dtype=2) == 1 and _append(lib, ok, dtype=-1) == 1
    assert _append(lib, ok, n_req=1 << 29) == 1
    assert _append(lib, _pages(n_kv=8193), ld=1 << 24) == 1
    for theta in (-1.0, float("nan"), float("inf")):
        assert _append(lib, ok, theta=theta) == 1
    for null in ("off", "pos0", "k", "v"):
        assert _append(lib, ok, **{null: None}) == 1
    assert _append(lib, ok, n_req=0) == 0 and _append(lib, ok, n_rows=0, k=None) == 0


def test_attention_refusals(lib):
    ok = _pages()
    assert _attn(lib, None) == 1
    assert _attn(lib, ok, n_q=7) == 1 and _attn(lib, ok, n_q=0) == 1
    assert _attn(lib, ok, q_ld=1016) == 1 and _attn(lib, ok, out_ld=1016) == 1
    assert _attn(lib, ok, q_ld=1028) == 1 and _attn(lib, ok, out_ld=1028) == 1
    assert _attn(lib, ok, q=ctypes.c_void_p(72)) == 1 and _attn(lib, ok, out=ctypes.c_void_p(72)) == 1
    assert _attn(lib, ok, mask=P, mask_ld=0) == 1
    assert _attn(lib, ok, mask=P, mask_ld=1, max_rows=33) == 1
    assert _attn(lib, ok, max_rows=-1) == 1
    assert _attn(lib, ok, n_rows=1 << 27) == 1                    # rows x heads reach 2^30
    for null in ("off", "pos0", "q", "out"):
        assert _attn(lib, ok, **{null: None}) == 1
    need = lib.dflash_paged_attention_e4m3_workspace_bytes(8, 2, 128)
    assert need > 0
    assert _attn(lib, ok) == 3 and _attn(lib, ok, ws=P, ws_bytes=need - 1) == 3
    assert _attn(lib, ok, ws=ctypes.c_void_p(72), ws_bytes=need) == 1
    assert _attn(lib, ok, n_req=0) == 0 and _attn(lib, ok, n_rows=0) == 0
    for sizes in ((7, 2, 128), (0, 0, 128), (8, 2, 96), (2, 4, 128)):
        assert lib.dflash_paged_attention_e4m3_workspace_bytes(*sizes) == 0


def test_adjust_refusals(lib):
    def call(n_req=1, rows=2, vocab=100, dtype=1, x=P, ld=100, out=ctypes.c_void_p(4096), out_ld=100, off=P, hist=None,
             hist_ld=0, hist_len=None, tok=None, mask=None, mask_ld=0, bt=None, bv=None, nb=0, allowed=None, al=0):
        return lib.dflash_logits_adjust(n_req, rows, vocab, dtype, x, ld, out, out_ld, off, hist, hist_ld, hist_len, None,
                                        None, None, None, tok, mask, mask_ld, bt, bv, nb, allowed, al, None)

    for bad in (dict(n_req=-1), dict(rows=-1), dict(rows=1 << 30), dict(vocab=0), dict(vocab=101),
                dict(vocab=(1 << 22) + 1, ld=1 << 23, out_ld=1 << 23), dict(dtype=7), dict(x=None), dict(out=None),
                dict(off=None), dict(ld=99), dict(out_ld=99), dict(out=P, out_ld=104), dict(x=ctypes.c_void_p(65)),
                dict(dtype=0, x=ctypes.c_void_p(66)), dict(hist=P), dict(hist=P, hist_ld=4), dict(hist=P, hist_len=P),
                dict(mask=P, mask_ld=1), dict(mask=P, tok=P), dict(nb=-1), dict(nb=2), dict(nb=2, bt=P),
                dict(nb=(1 << 20) + 1, bt=P, bv=P), dict(allowed=P, al=3)):
        assert call(**bad) == 1, bad
        assert lib.dflash_last_error()
    assert call(rows=0) == 0 and call(n_req=0, x=None) == 0


def test_binding_refuses_wrong_tensors():
    z = torch.zeros
    u8 = dict(dtype=torch.uint8)
    table = z(1, 2, dtype=torch.int32)
    good = [z(2, 1, 16, 64, **u8), z(2, 1, 16, 64, **u8), z(2, 1, 1, **u8), z(2, 1, 1, **u8), table]
    with pytest.raises(ValueError, match="CUDA"):
        binding.PagesE4M3(*good)
    for i, t in ((0, z(2, 1, 16, 128, **u8)), (1, z(2, 1, 16, 64)), (2, z(2, 1, 2, **u8)), (3, z(2, 1, 1)),
                 (4, z(1, 2)), (0, z(1, 2, 64, 16, **u8).permute(1, 0, 3, 2))):
        with pytest.raises(ValueError):
            binding.PagesE4M3(*good[:i], t, *good[i + 1:])
    x, off = z(2, 10), z(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        binding.logits_adjust(x, x, off)
    with pytest.raises(ValueError):
        binding.logits_adjust(x, z(2, 11), off)
    with pytest.raises(ValueError):
        binding.logits_adjust(x, x, off, vocab=11)
    with pytest.raises(ValueError):
        binding.logits_adjust(x, x, z(0, dtype=torch.int32))


def test_adjust_of_an_empty_batch_needs_no_lists(lib):
    """Tensors without entries have null pointers, whatever their widths."""
    def call(n_req, rows, **kw):
        a = dict(hist=None, hist_ld=0, hist_len=None, tok=None, mask=None, mask_ld=0, bt=None, bv=None, nb=0)
        a.update(kw)
        return lib.dflash_logits_adjust(n_req, rows, 100, 1, None, 100, None, 100, None, a["hist"], a["hist_ld"],
                                        a["hist_len"], None, None, None, None, a["tok"], a["mask"], a["mask_ld"],
                                        a["bt"], a["bv"], a["nb"], None, 4, None)
    for n_req, rows in ((0, 0), (0, 5), (3, 0)):
        assert call(n_req, rows) == 0
        assert call(n_req, rows, hist_ld=8, mask_ld=2, nb=7) == 0
    assert call(0, 0, nb=-1) == 1 and call(0, 0, nb=(1 << 20) + 1) == 1


def test_adjust_refuses_histories_past_its_indexes(lib):
    def call(ld):
        return lib.dflash_logits_adjust(1, 2, 100, 1, P, 100, ctypes.c_void_p(4096), 100, None, P, ld, P, None, None, None,
                                        None, None, None, 0, None, None, 0, None, 0, None)
    for ld in ((1 << 30) + 1, (1 << 31) - 1):
        assert call(ld) == 1 and b"history" in lib.dflash_last_error()
    assert call(1 << 30) == 1 and b"null" in lib.dflash_last_error()       # (the row offsets)
