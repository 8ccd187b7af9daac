"""Refusals of the paged-cache operators and the filtered sampler: arguments are
checked on the host before anything is enqueued, so none of this needs a GPU."""
import ctypes

import pytest
import torch

from block_diffusion_speculative_kv_gb300 import binding, build

P = ctypes.c_void_p(64)        # never dereferenced: every call is rejected first


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.lib()


def _pages(k=64, v=64, table=64, table_ld=4, n_pages=10, page=16, n_kv=2, hd=128, dtype=1):
    return ctypes.byref(binding.PagesStruct(k, v, table, table_ld, n_pages, page, n_kv, hd, dtype))


BAD_PAGES = [dict(k=0), dict(v=0), dict(table=0), dict(k=72), dict(table_ld=0), dict(n_pages=0),
             dict(page=8), dict(page=24), dict(page=2048), dict(page=0), dict(page=-16), dict(n_kv=0),
             dict(hd=96), dict(hd=256), dict(dtype=5), dict(table_ld=1 << 27), dict(n_pages=1 << 30)]


def _append(lib, pages, n_req=1, n_rows=4, off=P, pos0=P, pos=None, k=P, v=P, ld=256, theta=1e6):
    return lib.dflash_paged_append(pages, n_req, n_rows, off, pos0, pos, k, v, ld, theta, None)


def _attn(lib, pages, n_req=1, n_rows=4, n_q=8, off=P, pos0=P, max_rows=4, q=P, q_ld=1024, mask=None,
          mask_ld=0, out=P, out_ld=1024, ws=None, ws_bytes=0):
    return lib.dflash_paged_attention(pages, n_req, n_rows, n_q, off, pos0, max_rows, q, q_ld, mask, mask_ld,
                                      out, out_ld, ws, ws_bytes, None)


@pytest.mark.parametrize("bad", BAD_PAGES)
def test_bad_pages(lib, bad):
    assert _append(lib, _pages(**bad)) == 1
    assert _attn(lib, _pages(**bad)) == 1
    assert lib.dflash_last_error()


def test_append_refusals(lib):
    ok = _pages()
    assert _append(lib, None) == 1
    assert _append(lib, ok, n_req=-1) == 1 and _append(lib, ok, n_rows=-1) == 1
    assert _append(lib, ok, ld=255) == 1
    for theta in (-1.0, float("nan"), float("inf")):
        assert _append(lib, ok, theta=theta) == 1
    for null in ("off", "pos0", "k", "v"):
        assert _append(lib, ok, **{null: None}) == 1
    assert _append(lib, ok, n_req=0) == 0 and _append(lib, ok, n_rows=0, k=None) == 0


def test_attention_refusals(lib):
    ok = _pages()
    assert _attn(lib, None) == 1
    assert _attn(lib, _pages(dtype=0)) == 2                       # fp32 pages: not implemented
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
    need = lib.dflash_paged_attention_workspace_bytes(8, 2, 128)
    assert need > 0
    assert _attn(lib, ok) == 3 and _attn(lib, ok, ws=P, ws_bytes=need - 1) == 3
    assert _attn(lib, ok, ws=ctypes.c_void_p(72), ws_bytes=need) == 1
    assert _attn(lib, ok, n_req=0) == 0 and _attn(lib, ok, n_rows=0) == 0
    for sizes in ((7, 2, 128), (0, 0, 128), (8, 2, 96), (2, 4, 128)):
        assert lib.dflash_paged_attention_workspace_bytes(*sizes) == 0


def test_norm_rope_refusals(lib):
    def call(n=4, n_q=2, n_kv=1, hd=128, dtype=1, gq=P, gk=P, eps=1e-6, theta=1e6, pos=P, q=P, q_ld=256, k=P,
             k_ld=128, qo=ctypes.c_void_p(4096), qo_ld=256, ko=ctypes.c_void_p(8192), ko_ld=128):
        return lib.dflash_qk_norm_rope(n, n_q, n_kv, hd, dtype, gq, gk, eps, theta, pos, q, q_ld, k, k_ld, qo,
                                       qo_ld, ko, ko_ld, None)

    for bad in (dict(n=-1), dict(n_q=-1), dict(n_kv=-2), dict(hd=32), dict(dtype=2), dict(eps=-1.0),
                dict(eps=float("nan")), dict(theta=-1.0), dict(theta=float("nan")), dict(q_ld=255),
                dict(k_ld=127), dict(qo_ld=128), dict(ko_ld=64), dict(q=None), dict(k=None), dict(qo=None),
                dict(ko=None), dict(pos=None), dict(qo=P, q_ld=512), dict(ko=P, k_ld=256)):
        assert call(**bad) == 1, bad
    assert call(n=0) == 0 and call(n_q=0, n_kv=0) == 0


def test_sample_refusals(lib):
    def call(rows=2, vocab=100, ld=100, dtype=1, x=P, u=P, tok=P, lp=P):
        return lib.dflash_logits_sample_filtered(rows, vocab, ld, dtype, x, None, None, None, None, u, tok, lp,
                                                 None)

    for bad in (dict(rows=-1), dict(vocab=0), dict(vocab=101), dict(vocab=(1 << 22) + 1, ld=1 << 23),
                dict(dtype=7), dict(x=None), dict(u=None), dict(tok=None), dict(lp=None)):
        assert call(**bad) == 1, bad
    assert call(rows=0) == 0


def test_binding_refuses_host_tensors():
    z = torch.zeros
    with pytest.raises(ValueError):
        binding.Pages(z(2, 1, 16, 64), z(2, 1, 16, 64), z(1, 2, dtype=torch.int32))
    with pytest.raises(ValueError):
        binding.Pages(z(2, 1, 16, 64), z(2, 1, 16, 128), z(1, 2, dtype=torch.int32))
    with pytest.raises(ValueError):
        binding.Pages(z(2, 1, 16, 64), z(2, 1, 16, 64), z(1, 2))
    with pytest.raises(ValueError):
        binding.qk_norm_rope(z(2, 128), None, None, None, 0.0, 0.0, None, 64)
    with pytest.raises(ValueError):
        binding.qk_norm_rope(None, None, None, None, 0.0, 0.0, None, 64)
    with pytest.raises(ValueError):
        binding.logits_sample_filtered(z(2, 10), z(2), z(2, dtype=torch.int32), z(2))


def test_slots_past_the_limit(lib):
    """A request's slots, and the rows added to them, stay within 32 bits."""
    assert _append(lib, _pages(table_ld=(1 << 26) + 1)) == 1 and _attn(lib, _pages(table_ld=(1 << 26) + 1)) == 1
    assert _append(lib, _pages(table_ld=1 << 26), n_rows=0) == 0 and _attn(lib, _pages(table_ld=1 << 26), n_rows=0) == 0


def test_heads_past_the_limit(lib):
    """Head counts whose index arithmetic would leave 32 bits."""
    def norm(n_q, n_kv, n=0):
        big = 1 << 24
        return lib.dflash_qk_norm_rope(n, n_q, n_kv, 128, 1, P, P, 1e-6, 1e6, P, P, big, P, big, P, big, P, big, None)

    assert norm(16384, 16384) == 0
    for n_q, n_kv in ((16385, 1), (1, 16385), (23171, 0), ((1 << 31) - 1, 0)):
        assert norm(n_q, n_kv) == 1 and norm(n_q, n_kv, n=4) == 1

    def append(n_kv, n_rows=0):
        return _append(lib, _pages(n_kv=n_kv), n_rows=n_rows, ld=1 << 24)

    assert append(8192) == 0
    for n_kv in (8193, 11586, 100000):
        assert append(n_kv) == 1 and append(n_kv, n_rows=4) == 1


def test_division_within_the_limit():
    """The quotient by a rounded-up reciprocal is exact for eight rows of 16384 heads,
    and one too large soon after 23170."""
    def quot(i, n):
        return i if n == 1 else (i * ((2 ** 32 + n - 1) // n)) >> 32

    for n in list(range(1, 300)) + list(range(16384 - 300, 16385)):
        for r in range(1, 9):
            for i in (r * n - 1, r * n - n):
                assert quot(i, n) == i // n
    assert any(quot(8 * n - 1, n) == 8 for n in range(23171, 33000))


def test_sample_vocab_within_the_view():
    """A view's rows may lie further apart than its columns reach: vocab is bound by the
    columns, or the last row would be read past its storage."""
    wide = torch.zeros(3, 40)
    args = torch.zeros(3), torch.zeros(3, dtype=torch.int32), torch.zeros(3)
    for view, vocab in ((wide[:, 3:], 38), (wide[:, 3:], 40), (wide[:, :10], 11), (wide[:1, :10], 40), (wide, 41)):
        n = len(view)
        with pytest.raises(ValueError, match="vocab"):
            binding.logits_sample_filtered(view, *(a[:n] for a in args), vocab=vocab)
    with pytest.raises(ValueError, match="CUDA"):              # (accepted as far as that goes)
        binding.logits_sample_filtered(wide[:, 3:], *args, vocab=37)
    with pytest.raises(ValueError, match="logits"):
        binding.logits_sample_filtered(wide[0], *args)


def test_no_requests_need_no_table(lib):
    """An empty batch: a table of no rows has a null pointer."""
    none = _pages(table=0)
    assert _append(lib, none, n_req=0) == 0 and _attn(lib, none, n_req=0) == 0
    assert _append(lib, none, n_req=1, n_rows=0) == 1 and _attn(lib, none, n_req=1, n_rows=0) == 1
