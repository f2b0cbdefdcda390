"""Refusals of the paged-cache calls on the host (no GPU: the pointers are never dereferenced)."""
import ctypes

import pytest
import torch

OK, INVALID, SHAPE, ALIGN, WS = 0, 1, 2, 3, 4
P = ctypes.c_void_p(0x100000)
MIS = ctypes.c_void_p(0x100008)


@pytest.fixture(scope="module")
def lib():
    from canvas_denoising_denoise_b200 import _lib
    return _lib.load()


APPEND = dict(k=P, v=P, ldkv=1024, q=P, ldq=2048, q_out=P, ldqo=2048, Hq=16, rope=P, rope_len=64,
              rot_dim=128, interleaved=0, k_pages=P, v_pages=P, k_exp=P, v_exp=P, n_pages=8,
              page=64, page_table=P, max_pages=4, tok_start=P, cache_len=P, max_new=0, B=1, T=1,
              Hkv=8, hd=128, stream=None)
ATTN = dict(q=P, ldq=2048, k_pages=P, v_pages=P, k_exp=P, v_exp=P, n_pages=8, page=64,
            page_table=P, max_pages=4, tok_start=P, cache_len=P, max_new=0, max_prefix=0, out=P,
            ldo=2048, lse=None, B=1, T=1, Hq=16, Hkv=8, hd=128, scale=0.1, mask=0, ws=None, wsn=0,
            stream=None)


def call(fn, base, **kw):
    assert set(kw) <= set(base)
    return fn(*{**base, **kw}.values())


def test_no_rows_is_no_work(lib):
    # max_new 0 (above) or T 0: the arguments are checked and nothing is launched
    before = lib.dg_launch_count()
    assert call(lib.dg_kv_append_e4m3, APPEND) == OK
    assert call(lib.dg_kv_append_e4m3, APPEND, max_new=5, T=0) == OK
    assert call(lib.dg_kv_append_e4m3, APPEND, q=None, q_out=None, rope=None, rot_dim=0) == OK
    assert call(lib.dg_paged_attn_e4m3, ATTN) == OK
    assert call(lib.dg_paged_attn_e4m3, ATTN, max_new=5, T=0) == OK
    assert lib.dg_launch_count() == before


@pytest.mark.parametrize("kw,status", [
    (dict(k=None), INVALID), (dict(v_exp=None), INVALID), (dict(cache_len=None), INVALID),
    (dict(q_out=None), INVALID), (dict(q=None), INVALID), (dict(Hq=0), INVALID),
    (dict(rope=None), INVALID), (dict(rot_dim=0), INVALID), (dict(rope_len=0), INVALID),
    (dict(rope=None, rot_dim=0), INVALID),  # queries without a table
    (dict(interleaved=2), INVALID), (dict(B=0), INVALID), (dict(T=-1), INVALID),
    (dict(max_new=-1), INVALID), (dict(n_pages=0), INVALID), (dict(max_pages=0), INVALID),
    (dict(rot_dim=136), SHAPE), (dict(rot_dim=24), SHAPE), (dict(hd=96), SHAPE),
    (dict(page=8), SHAPE), (dict(page=256), SHAPE), (dict(page=48), SHAPE),
    (dict(n_pages=1 << 30), SHAPE), (dict(max_pages=1 << 26), SHAPE),
    (dict(ldkv=1020), ALIGN), (dict(ldkv=1016), ALIGN), (dict(ldq=2047), ALIGN),
    (dict(ldqo=2040), ALIGN), (dict(k=MIS), ALIGN), (dict(v_pages=MIS), ALIGN),
    (dict(rope=MIS), ALIGN), (dict(q_out=MIS), ALIGN),
    (dict(max_new=1 << 30, T=1 << 30, B=64, page=16, max_pages=1 << 26), SHAPE),
])
def test_append_refuses(lib, kw, status):
    assert call(lib.dg_kv_append_e4m3, APPEND, **kw) == status
    assert b"dg_kv_append_e4m3" in lib.dg_last_error()


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), INVALID), (dict(out=None), INVALID), (dict(page_table=None), INVALID),
    (dict(Hq=12), INVALID), (dict(Hq=0), INVALID), (dict(mask=2), INVALID),
    (dict(max_prefix=-1), INVALID), (dict(scale=0.0), INVALID), (dict(scale=-1.0), INVALID),
    (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID),
    (dict(B=0), INVALID), (dict(B=65536), INVALID), (dict(hd=80), SHAPE), (dict(page=17), SHAPE),
    (dict(n_pages=1 << 30), SHAPE), (dict(max_new=1 << 30, T=1 << 30), SHAPE),
    (dict(ldq=2040), ALIGN), (dict(ldo=2052), ALIGN), (dict(q=MIS), ALIGN), (dict(out=MIS), ALIGN),
    (dict(k_pages=MIS), ALIGN), (dict(max_new=256, T=256, max_prefix=4096), WS),
    (dict(max_new=256, T=256, max_prefix=4096, ws=MIS, wsn=1 << 40), WS),
])
def test_attention_refuses(lib, kw, status):
    assert call(lib.dg_paged_attn_e4m3, ATTN, **kw) == status
    assert b"dg_paged_attn_e4m3" in lib.dg_last_error()


def test_workspace_query(lib):
    q = lib.dg_paged_attn_workspace_bytes
    assert q(1, 256, 16, 8, 128, 256, 4096) > 0
    assert q(64, 64 * 256, 16, 8, 128, 256, 0) == 0   # enough work without a split over keys
    assert q(1, 256, 16, 8, 96, 256, 4096) == 0
    assert q(1, 0, 16, 8, 128, 256, 4096) == 0
    # a bound beyond the batch's rows plans for those rows
    assert q(1, 256, 16, 8, 128, 4096, 4096) == q(1, 256, 16, 8, 128, 256, 4096)


def test_cache_object_refuses():
    import canvas_denoising_denoise_b200 as dg
    pages = torch.zeros((4, 2, 16, 64), dtype=torch.uint8)
    exps = torch.zeros((4, 2), dtype=torch.uint8)
    dg.PagedCache(pages, pages.clone(), exps, exps.clone())
    for bad in ((pages.float(), pages, exps, exps), (pages[:3], pages, exps, exps),
                (pages, pages, exps[:, :1], exps), (pages.transpose(1, 2), pages, exps, exps)):
        with pytest.raises(ValueError):
            dg.PagedCache(*bad)


@pytest.mark.parametrize("n,rot", [(5, 16), (70, 128)])
def test_rope_table_is_cos_and_sin_of_the_angles(n, rot):
    import math

    import canvas_denoising_denoise_b200 as dg
    t = dg.rope_table(n, rot, base=5000.0, device="cpu")
    assert t.shape == (n, rot // 2, 2) and t.dtype == torch.float32
    for p, i in ((0, 0), (n - 1, 0), (n - 1, rot // 2 - 1), (n // 2, 3)):
        a = p * 5000.0 ** (-2 * i / rot)
        assert abs(t[p, i, 0].item() - math.cos(a)) <= 2 ** -24
        assert abs(t[p, i, 1].item() - math.sin(a)) <= 2 ** -24
