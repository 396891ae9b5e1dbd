"""Paged key-value cache calls: refusals on the host (no GPU is touched, every
device address is fake) and the plain model of the block tables that the GPU
tests compare with."""

import ctypes
import os
import re

import pytest
import torch

from attention_predictor_gemv_b200 import binding as bd
from tests._paged import tables_model

A = 0x10000  # a 16-byte aligned fake device address (never dereferenced)
NEW = {"dv_page_tables", "dv_paged_append", "dv_paged_attn", "dv_sparse_mha_paged"}


def _kv(**kw):
    a = dict(kvdtype=bd.DV_BF16, K=A, V=A, page_stride=0, n_pages=10, page=16, h_kv=4, dh=64)
    a.update(kw)
    return bd.PagedKVC(*a.values())


def test_header_declares_the_paged_calls():
    assert NEW <= set(bd.exported_symbols_declared_in_header())


def test_workspace_sizes():
    n = bd.dv_workspace_size(bd.DV_OP_PAGE_TABLES, bd.dims())
    assert n == bd.dv_workspace_size(bd.DV_OP_PAGED_APPEND, bd.dims()) > 0
    a = bd.dv_workspace_size(bd.DV_OP_PAGED_ATTN, bd.dims(dh=64))
    assert n < a and n < bd.dv_workspace_size(bd.DV_OP_PAGED_ATTN, bd.dims(dh=128))
    for dh in (0, 4, 12, 264):
        assert bd.dv_workspace_size(bd.DV_OP_PAGED_ATTN, bd.dims(dh=dh)) == 0
    m = bd.dv_workspace_size(bd.DV_OP_SPARSE_MHA_PAGED, bd.dims(B=4, d=512, h=8, dh=64, kh_max=8))
    assert m > bd.dv_workspace_size(bd.DV_OP_SPARSE_MHA_PAGED, bd.dims(B=1, d=512, h=8, dh=64, kh_max=2)) > a
    assert bd.dv_workspace_size(bd.DV_OP_PAGED_ATTN, bd.dims(dh=256)) > bd.dv_workspace_size(bd.DV_OP_PAGED_ATTN, bd.dims(dh=128))
    assert bd.dv_workspace_size(bd.DV_OP_SPARSE_MHA_PAGED, bd.dims(B=17, d=512, h=8, dh=64, kh_max=8)) == 0
    assert bd.dv_workspace_size(bd.DV_OP_SPARSE_MHA_PAGED, bd.dims(B=1, d=512, h=8, dh=96, kh_max=8)) == 0


def _append(kv, k=A, v=A, T=3, slots=A, ws=A, wsb=1 << 20):
    return bd._lib_dv_paged_append(ctypes.byref(kv) if kv is not None else None, k, v, T, slots, ws, wsb, None)


@pytest.mark.parametrize("bad, status", [
    (dict(K=None), bd.DV_ERR_ARG), (dict(V=None), bd.DV_ERR_ARG), (dict(kvdtype=2), bd.DV_ERR_ARG),
    (dict(kvdtype=-1), bd.DV_ERR_ARG), (dict(K=A + 8), bd.DV_ERR_ALIGN), (dict(V=A + 2), bd.DV_ERR_ALIGN),
    (dict(n_pages=0), bd.DV_ERR_ARG), (dict(page=0), bd.DV_ERR_ARG), (dict(h_kv=0), bd.DV_ERR_ARG),
    (dict(dh=0), bd.DV_ERR_ARG), (dict(dh=60), bd.DV_ERR_ARG), (dict(dh=264), bd.DV_ERR_UNSUPPORTED),
    (dict(page_stride=4 * 16 * 64 - 64), bd.DV_ERR_ARG), (dict(page_stride=4 * 16 * 64 + 8), bd.DV_ERR_ARG),
    (dict(page_stride=-64), bd.DV_ERR_ARG), (dict(n_pages=2 ** 31 - 1), bd.DV_ERR_UNSUPPORTED),
    (dict(n_pages=2 ** 20, page_stride=64 * 2 ** 11), bd.DV_ERR_UNSUPPORTED),
    (dict(n_pages=2 ** 16, page=2 ** 15), bd.DV_ERR_UNSUPPORTED),
])
def test_pool_checks(bad, status):
    kv = _kv(**bad)
    assert _append(kv) == status
    assert bd._lib_dv_paged_attn(ctypes.byref(kv), A, 1, 4, A, 4, A, 0.1, None, None, 0, A, None, A, 1 << 30, None) == status


def test_append_checks():
    assert _append(None) == bd.DV_ERR_ARG
    assert _append(_kv(), k=None) == bd.DV_ERR_ARG
    assert _append(_kv(), slots=None) == bd.DV_ERR_ARG
    assert _append(_kv(), T=-1) == bd.DV_ERR_ARG
    assert _append(_kv(), v=A + 4) == bd.DV_ERR_ALIGN
    assert _append(_kv(), slots=A + 4) == bd.DV_ERR_ALIGN
    assert _append(_kv(), ws=None) == bd.DV_ERR_ARG
    assert _append(_kv(), ws=A + 8) == bd.DV_ERR_ALIGN
    assert _append(_kv(), wsb=16) == bd.DV_ERR_WORKSPACE
    assert _append(_kv(), T=0) == bd.DV_OK  # nothing to launch


def _attn(kv=None, q=A, B=1, h_q=8, table=A, W=4, lens=A, idx=None, cnt=None, kh=0, out=A, lse=None, ws=A, wsb=1 << 30):
    return bd._lib_dv_paged_attn(ctypes.byref(kv or _kv()), q, B, h_q, table, W, lens, 0.1, idx, cnt, kh, out, lse, ws, wsb,
                                 None)


def test_attn_checks():
    for kw in (dict(q=None), dict(table=None), dict(lens=None), dict(out=None), dict(B=0), dict(W=0), dict(h_q=0),
               dict(h_q=6), dict(idx=A), dict(cnt=A), dict(idx=A, cnt=A, kh=-1), dict(idx=A, cnt=A, kh=5), dict(ws=None)):
        assert _attn(**kw) == bd.DV_ERR_ARG, kw
    for kw in (dict(q=A + 8), dict(table=A + 4), dict(lens=A + 4), dict(out=A + 4), dict(lse=A + 4),
               dict(idx=A + 4, cnt=A, kh=1), dict(ws=A + 1)):
        assert _attn(**kw) == bd.DV_ERR_ALIGN, kw
    assert _attn(B=4097) == bd.DV_ERR_UNSUPPORTED
    assert _attn(W=2 ** 27) == bd.DV_ERR_UNSUPPORTED  # W * page
    assert _attn(h_q=2 ** 26) == bd.DV_ERR_UNSUPPORTED  # h_q * dh
    assert _attn(B=4096, W=2 ** 21) == bd.DV_ERR_UNSUPPORTED  # units of 16 keys of all requests and heads
    assert _attn(wsb=1 << 16) == bd.DV_ERR_WORKSPACE
    assert _attn(idx=A, cnt=A, kh=0) == bd.DV_OK  # no head: nothing to launch


def _tables(**kw):
    a = dict(want=A, R=4, page=16, n_pages=100, W=8, lens=A, lens_out=A, table=A, free_list=A, free_count=A,
             free_count_out=A, max_tokens=64, slots=A, offsets=A, granted=A, ws=A, wsb=1 << 20, st=None)
    a.update(kw)
    return bd._lib_dv_page_tables(*a.values())


def test_page_tables_checks():
    for n in ("want", "lens", "lens_out", "table", "free_list", "free_count", "free_count_out", "slots", "offsets",
              "granted", "ws"):
        assert _tables(**{n: None}) == bd.DV_ERR_ARG, n
        assert _tables(**{n: A + 4}) == bd.DV_ERR_ALIGN, n
    for kw in (dict(R=0), dict(page=0), dict(n_pages=0), dict(W=0), dict(max_tokens=-1)):
        assert _tables(**kw) == bd.DV_ERR_ARG, kw
    for kw in (dict(R=4097), dict(page=2 ** 26), dict(W=2 ** 30), dict(n_pages=2 ** 28), dict(R=1, W=1, n_pages=1, page=2 ** 30)):
        assert _tables(**kw) == bd.DV_ERR_UNSUPPORTED, kw
    assert _tables(wsb=16) == bd.DV_ERR_WORKSPACE


def _mha(kv=None, **kw):
    a = dict(y=A, B=1, d=256, Wqkv=A, bqkv=None, WOt=A, bO=None, dt=bd.DV_BF16, kv=ctypes.byref(kv or _kv()), table=A, W=4,
             lens=A, slots=A, scale=0.1, hidx=A, hcnt=A, kh=2, out=A, acc=0, exact=0, ws=A, wsb=1 << 30, st=None)
    a.update(kw)
    return bd._lib_dv_sparse_mha_paged(*a.values())


def test_sparse_mha_paged_checks():
    for n in ("y", "Wqkv", "WOt", "table", "lens", "slots", "hidx", "hcnt", "out", "ws"):
        assert _mha(**{n: None}) == bd.DV_ERR_ARG, n
        assert _mha(**{n: A + 4}) == bd.DV_ERR_ALIGN, n
    for kw in (dict(bqkv=A + 4), dict(bO=A + 4)):
        assert _mha(**kw) == bd.DV_ERR_ALIGN, kw
    for kw in (dict(B=0), dict(B=17), dict(d=60), dict(W=0), dict(kh=5), dict(kh=-1), dict(dt=9)):
        assert _mha(**kw) == bd.DV_ERR_ARG, kw
    assert _mha(dt=bd.DV_F32) == bd.DV_ERR_UNSUPPORTED  # the pools are bf16
    assert _mha(kv=_kv(dh=96)) == bd.DV_ERR_UNSUPPORTED
    assert _mha(kv=_kv(h_kv=1025)) == bd.DV_ERR_UNSUPPORTED
    assert _mha(W=2 ** 30) == bd.DV_ERR_UNSUPPORTED
    assert _mha(wsb=1 << 16) == bd.DV_ERR_WORKSPACE


def test_binding_checks_shapes_before_the_call():
    K = torch.zeros(4, 2, 8, 64)
    with pytest.raises(ValueError, match="CUDA"):
        bd.PagedKV(K, K.clone())
    with pytest.raises(ValueError, match="alike"):
        bd.PagedKV(K, torch.zeros(4, 2, 8, 32))
    with pytest.raises(ValueError, match="alike"):
        bd.PagedKV(K, torch.zeros(4, 2, 8, 64, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="contiguous"):
        bd.PagedKV(K.transpose(1, 2), K.transpose(1, 2))
    with pytest.raises(ValueError, match="empty"):
        bd.PagedKV(K[:0], K[:0])
    i = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError, match="want"):
        bd.dv_page_tables(i.long(), i, i, torch.zeros(4, 2, dtype=torch.int32), i, i[:1], i[:1], i, i, i, 16, i)


def test_tables_model_grows_shrinks_and_refuses():
    """The model that the GPU tests use, by hand: pages of 4, a stack of 3."""
    m = tables_model(want=[5, 0, 9, -1, 12], lens=[4, 6, 8, 3, 0],
                     table=[[0, -1, -1], [1, 2, -1], [3, 4, -1], [5, -1, -1], [-1, -1, -1]],
                     free=[7, 8, 9], page=4, n_pages=12, max_tokens=8)
    # freed: 1, 2 -> stack 7 8 9 1 2; row 0 takes 2, row 2 takes 1, row 4 wants three of [9 8 7] but 12 tokens do not fit 8
    assert m["granted"] == [1, 1, 1, 1, 0]
    assert m["lens"] == [5, 0, 9, 3, 0]
    assert m["table"][0] == [0, 2, -1] and m["table"][2] == [3, 4, 1]
    assert m["stack"][:3] == [7, 8, 9] and m["free_count"] == 3
    assert m["slots"] == [2 * 4, 1 * 4] + [-1] * 6 and m["offsets"] == [0, 1, 1, 2, 2, 2]


def test_the_projections_tile_list_holds_every_set():
    """A CTA's list holds its share of the most tiles that a call can have: 1000 entries, none of them a valid head, and k
    and v of all 1024 heads of 128 channels, over 148 SMs; and the host compares that very count with the list."""
    here = os.path.join(os.path.dirname(bd.__file__), "csrc")
    proj, host = (open(os.path.join(here, f)).read() for f in ("dv_paged_proj.cuh", "dv_paged.cu"))
    held = int(re.search(r"constexpr int PQ_MAX_TILES = (\d+);", proj).group(1))
    most = re.search(r"qkv_most_tiles\(.*?\{\s*return (.*?);", proj, re.S).group(1)
    for src, py in (("3ll", "3"), ("2ll", "2"), ("(all ? 2 * h : 0)", "2 * h"), ("dh / 8", "dh // 8")):
        most = most.replace(src, py)
    most_tiles = eval(most, dict(kh_max=1000, h=1024, dh=128))  # every entry invalid, exact_kv
    assert most_tiles == (3 * 1000 + 2 * 1024) * 16
    # CTA c has tiles floor(n c / 148) up to floor(n (c + 1) / 148)
    assert max(most_tiles * (c + 1) // 148 - most_tiles * c // 148 for c in range(148)) <= -(-most_tiles // 148) <= held
    assert "per_cta <= PQ_MAX_TILES" in host and "s_row[PQ_MAX_TILES]" in proj


def test_paged_kernels_take_no_read_only_loads():
    """A kernel launched with programmatic serialisation may be resident while the kernel before it still writes its inputs, so
    they are read by coherent loads: the read-only path asks for data that does not change while the kernel lives."""
    here = os.path.join(os.path.dirname(bd.__file__), "csrc")
    for f in ("dv_paged.cuh", "dv_paged_proj.cuh", "dv_paged.cu"):
        code = re.sub(r"//[^\n]*", "", open(os.path.join(here, f)).read())
        assert not re.search(r"__ldg\s*\(|ld\.global[.\w:]*\.nc", code), f


def test_attn_units_leave_room_for_rounding_up():
    """The units are rounded up to the warps of all CTAs in 31 bits: at most 8 warps of 2 CTAs on 148 SMs, under 8192."""
    wide = _kv(h_kv=64)
    assert _attn(wide, h_q=64, W=2 ** 25 - 2, wsb=16) == bd.DV_ERR_UNSUPPORTED  # 2^31 - 64 units
    assert _attn(wide, h_q=64, W=2 ** 25 - 2 - 128, wsb=16) == bd.DV_ERR_WORKSPACE  # 2^31 - 64 - 8192: past this check
    assert _mha(_kv(h_kv=64), W=2 ** 25 - 2) == bd.DV_ERR_UNSUPPORTED
    assert _mha(_kv(h_kv=64), W=2 ** 25 - 2 - 128, wsb=1 << 16) == bd.DV_ERR_WORKSPACE
