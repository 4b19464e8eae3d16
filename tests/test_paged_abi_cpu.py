"""Argument checks of the paged-cache, verification and device-rollback calls (no GPU: a call
that passes the checks then fails for want of a device, before any launch)."""
import ctypes
import os
import re

import pytest
import torch

from sparse_attention_decode_02_b200 import build as qbuild
from sparse_attention_decode_02_b200 import qsa as Q

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, INVALID, CAPACITY, CUDA, UNSUPPORTED = 0, 1, 2, 4, 5
PTR = 1 << 20   # an aligned address that no refused call touches


@pytest.fixture(scope="module")
def lib():
    if torch.cuda.is_available():
        pytest.skip("checks that stop at the missing device")
    qbuild.build()
    return Q.load_library()


def _cache(**kw):
    base = dict(n_pages=10, page_size=16, n_kv_heads=4, head_dim=128, format=Q.QSA_PAGE_FP8, reserved=0, page_stride=0,
                scale_stride=0, k_pages=PTR, v_pages=PTR, k_scales=PTR, v_scales=PTR)
    return Q.QsaPagedKv(**{**base, **kw})


def test_descriptor_matches_header():
    with open(os.path.join(ROOT, "include", "qsa.h")) as f:
        body = re.search(r"typedef struct \{([^{}]*?)\} qsa_paged_kv;", f.read(), re.S).group(1)
    body = re.sub(r"/\*.*?\*/", "", body, flags=re.S)
    ctype = {"int32_t": ctypes.c_int32, "int64_t": ctypes.c_int64, "void*": ctypes.c_void_p}
    fields = [(n, ctype[t]) for t, n in re.findall(r"(int32_t|int64_t|void\*)\s+(\w+);", body)]
    assert fields == list(Q.QsaPagedKv._fields_)


def test_buffer_sizes(lib):
    size = lambda which, **kw: lib.qsa_paged_bytes(ctypes.byref(_cache(**kw)), which)  # noqa: E731
    rows = 10 * 4 * 16
    assert size(0, format=Q.QSA_PAGE_F16) == rows * 256 and size(1, format=Q.QSA_PAGE_F16) == 0
    assert size(0) == rows * 128 and size(1) == rows * 4
    assert size(0, format=Q.QSA_PAGE_INT4) == rows * 64 and size(1, format=Q.QSA_PAGE_INT4) == rows * 8
    assert size(0, format=Q.QSA_PAGE_INT4, head_dim=64) == rows * 32
    assert size(0, n_pages=2 ** 31 - 1) == (2 ** 31 - 1) * 4 * 16 * 128     # past 32 bits
    assert size(2) == 0 and lib.qsa_paged_bytes(None, 0) == 0
    ws = lib.qsa_paged_workspace_bytes(ctypes.byref(_cache()), 32, 1)
    assert ws > 0 and ws % 256 == 0
    assert lib.qsa_paged_workspace_bytes(ctypes.byref(_cache()), 32, 4) >= ws


BAD_SHAPES = [(dict(n_pages=0), INVALID), (dict(n_kv_heads=0), INVALID), (dict(page_size=8), UNSUPPORTED),
              (dict(page_size=48), UNSUPPORTED), (dict(page_size=512), UNSUPPORTED), (dict(head_dim=96), UNSUPPORTED),
              (dict(head_dim=256), UNSUPPORTED), (dict(format=3), UNSUPPORTED), (dict(format=-1), UNSUPPORTED)]
BAD_BUFFERS = [(dict(k_pages=None), INVALID), (dict(v_pages=PTR + 8), INVALID), (dict(k_scales=None), INVALID),
               (dict(v_scales=PTR + 4), INVALID), (dict(page_stride=4 * 16 * 128 - 16), INVALID),
               (dict(page_stride=4 * 16 * 128 + 8), INVALID), (dict(scale_stride=16), INVALID),
               (dict(page_stride=-16), INVALID)]


@pytest.mark.parametrize("bad,want", BAD_SHAPES + BAD_BUFFERS)
def test_bad_caches_are_refused(lib, bad, want):
    c = ctypes.byref(_cache(**bad))
    if (bad, want) in BAD_SHAPES:
        assert lib.qsa_paged_bytes(c, 0) == 0 and lib.qsa_paged_workspace_bytes(c, 32, 1) == 0
    assert lib.qsa_paged_write(c, PTR, PTR, 0, 1, PTR, 1, 1, PTR, PTR, None, None) == want
    assert lib.qsa_paged_read(c, PTR, PTR, 0, 1, PTR, 1, 1, PTR, PTR, None, None) == want
    assert lib.qsa_paged_attend(c, PTR, 0, 1, 32, PTR, 1, 1, PTR, 0.0, PTR, None, PTR, 1 << 30, None, None) == want


ROWS = dict(k=PTR, v=PTR, row_stride=0, n_rows=3, block_table=PTR, table_width=2, n_seqs=2, first=PTR, row_start=PTR,
            status=None, stream=None)


@pytest.mark.parametrize("bad", [dict(k=PTR + 2), dict(row_stride=504), dict(row_stride=516), dict(row_stride=-512),
                                 dict(n_rows=-1), dict(n_seqs=-1), dict(table_width=0), dict(table_width=-1),
                                 dict(block_table=None), dict(first=None), dict(row_start=None), dict(first=PTR + 2),
                                 dict(status=PTR + 1), dict(k=None)])
def test_bad_row_arguments_are_refused(lib, bad):
    c, args = ctypes.byref(_cache()), {**ROWS, **bad}
    assert lib.qsa_paged_write(c, *args.values()) == INVALID
    if bad != dict(k=None):     # a read may leave one of the two out
        assert lib.qsa_paged_read(c, *args.values()) == INVALID


def test_empty_and_good_row_arguments(lib):
    c = ctypes.byref(_cache())
    for f in (lib.qsa_paged_write, lib.qsa_paged_read):
        assert f(c, *{**ROWS, "n_rows": 0, "k": None, "v": None}.values()) == OK
        assert f(c, *{**ROWS, "n_seqs": 0, "block_table": None}.values()) == OK
        assert f(c, *ROWS.values()) == CUDA                     # passes the checks, finds no device
        assert f(c, *{**ROWS, "row_stride": 520}.values()) == CUDA
    assert lib.qsa_paged_read(c, *{**ROWS, "k": None, "v": None}.values()) == OK
    assert lib.qsa_paged_read(c, *{**ROWS, "k": None}.values()) == CUDA


ATTEND = dict(q=PTR, q_stride=0, n_queries=1, n_q_heads=32, block_table=PTR, table_width=2, n_seqs=2, seq_lens=PTR,
              sm_scale=0.0, out=PTR, lse=None, workspace=PTR, workspace_bytes=1 << 30, status=None, stream=None)


@pytest.mark.parametrize("bad,want", [
    (dict(q=None), INVALID), (dict(q=PTR + 2), INVALID), (dict(q_stride=4088), INVALID), (dict(q_stride=4100), INVALID),
    (dict(n_queries=0), INVALID), (dict(n_queries=5), UNSUPPORTED), (dict(n_q_heads=0), INVALID),
    (dict(n_q_heads=30), UNSUPPORTED), (dict(n_q_heads=36), UNSUPPORTED), (dict(table_width=0), INVALID),
    (dict(n_seqs=-1), INVALID), (dict(n_seqs=65537), UNSUPPORTED), (dict(seq_lens=None), INVALID),
    (dict(block_table=PTR + 2), INVALID), (dict(sm_scale=-1.0), INVALID), (dict(sm_scale=float("nan")), INVALID),
    (dict(sm_scale=float("inf")), INVALID), (dict(sm_scale=2e20), INVALID), (dict(out=None), INVALID), (dict(lse=PTR + 2), INVALID),
    (dict(workspace=None), INVALID), (dict(workspace=PTR + 128), INVALID), (dict(status=PTR + 2), INVALID)])
def test_bad_attend_arguments_are_refused(lib, bad, want):
    assert lib.qsa_paged_attend(ctypes.byref(_cache()), *{**ATTEND, **bad}.values()) == want


def test_empty_and_good_attend_arguments(lib):
    c = ctypes.byref(_cache())
    assert lib.qsa_paged_attend(c, *{**ATTEND, "n_seqs": 0, "q": None, "out": None, "workspace": None}.values()) == OK
    assert lib.qsa_paged_attend(c, *ATTEND.values()) == CUDA
    assert lib.qsa_paged_workspace_bytes(c, 36, 1) == 0 and lib.qsa_paged_workspace_bytes(c, 32, 5) == 0


VERIFY = dict(target=PTR, target_stride=0, draft=PTR, draft_stride=0, tokens=PTR, n_drafts=None, uniforms=PTR, n_seqs=2,
              max_drafts=3, vocab=100, n_accepted=PTR, next_token=PTR, status=None, stream=None)


@pytest.mark.parametrize("bad,want", [
    (dict(target=None), INVALID), (dict(target=PTR + 2), INVALID), (dict(target_stride=99), INVALID),
    (dict(draft_stride=99), INVALID), (dict(draft=PTR + 1), INVALID), (dict(tokens=None), INVALID),
    (dict(uniforms=None), INVALID), (dict(n_seqs=-1), INVALID), (dict(max_drafts=-1), INVALID),
    (dict(max_drafts=65), UNSUPPORTED), (dict(vocab=0), INVALID), (dict(vocab=2 ** 30 + 1), UNSUPPORTED), (dict(n_accepted=None), INVALID),
    (dict(next_token=PTR + 2), INVALID), (dict(n_drafts=PTR + 2), INVALID), (dict(status=PTR + 2), INVALID)])
def test_bad_verify_arguments_are_refused(lib, bad, want):
    assert lib.qsa_verify_drafts(*{**VERIFY, **bad}.values()) == want


def test_empty_and_good_verify_arguments(lib):
    assert lib.qsa_verify_drafts(*{**VERIFY, "n_seqs": 0, "target": None}.values()) == OK
    assert lib.qsa_verify_drafts(*VERIFY.values()) == CUDA
    assert lib.qsa_verify_drafts(*{**VERIFY, "max_drafts": 0, "tokens": None, "draft": None}.values()) == CUDA
    assert lib.qsa_rollback_rejected(None, 0, 1, PTR, None) == INVALID


def test_binding_refuses_a_cache_without_pages(lib):
    for fmt, row, kind in ((Q.QSA_PAGE_F16, 64, torch.float16), (Q.QSA_PAGE_FP8, 64, torch.uint8), (Q.QSA_PAGE_INT4, 32, torch.uint8)):
        pages, scales = torch.zeros(0, 2, 16, row, dtype=kind), torch.zeros(0, 2, 16)
        with pytest.raises(Q.QsaError):
            Q.PagedKV(pages, pages, fmt, scales, scales)


def test_binding_refuses_tensors_that_are_not_on_the_gpu():
    pages = torch.zeros(4, 2, 16, 64, dtype=torch.float16)
    with pytest.raises(ValueError):
        Q.PagedKV(pages, pages, Q.QSA_PAGE_F16)
    with pytest.raises(ValueError):
        Q.PagedKV(pages.float(), pages.float(), Q.QSA_PAGE_F16)
    with pytest.raises(ValueError):
        Q.PagedKV(pages, pages, 7)
    with pytest.raises(ValueError):
        Q.PagedKV(pages[0], pages[0], Q.QSA_PAGE_F16)
