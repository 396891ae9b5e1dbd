"""Paged key-value cache on the GPU against the row-by-row models in 64 bits
(tests/_paged.py): block tables, the append, attention, the attention block,
and a run of them together.

Tolerances. Attention's scores carry fp32 sums of at most 24 chained tensor
core steps (each off by at most 2^-23 of the partial sum) plus a few fp32
roundings, so a score is off by at most 32 * 2^-23 = 2^-18 of
bound = max |scale| sum |q| |k|, a weight by twice that in relative terms (with
the normalisation), and the output by (2 * 2^-18 * bound + 2^-18) max |V|
(the last term: weights, products and sums over the keys, again below 32
steps of 2^-23 each joined in fp32). lse is off by 2^-18 bound plus one fp32
rounding of its value.
"""

import numpy as np
import pytest
import torch

from tests._helpers import f64
from tests._paged import attn_model, tables_model

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from attention_predictor_gemv_b200 import binding as bd
    from attention_predictor_gemv_b200 import workload as wl

BF16, F32 = torch.bfloat16, torch.float32


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def make_cache(lens, h, dh, page, dtype, seed, extra=3, junk=float("nan"), W=None, table_junk=2 ** 31 - 1):
    """Pools with randomly placed pages; slots past a row's length and unused
    pages hold `junk`, table entries past a row's pages `table_junk`."""
    g = gen(seed)
    n = [-(-max(0, x) // page) for x in lens]
    W = W or max(1, max(n))
    total = sum(n) + extra
    perm = torch.randperm(total, generator=g, device="cuda").tolist()
    table = np.full((len(lens), W), table_junk, dtype=np.int64)
    K = torch.full((total, h, page, dh), junk, device="cuda", dtype=dtype)
    V = torch.full((total, h, page, dh), junk, device="cuda", dtype=dtype)
    at = 0
    for b, x in enumerate(lens):
        for c in range(n[b]):
            p = perm[at]
            at += 1
            table[b, c] = p
            used = min(page, x - c * page)
            K[p, :, :used] = torch.randn(h, used, dh, generator=g, device="cuda").to(dtype)
            V[p, :, :used] = torch.randn(h, used, dh, generator=g, device="cuda").to(dtype)
    return K, V, i32(table.astype(np.int32).tolist()), i32(list(lens))


def attn_ws(dh):
    return bd.workspace(bd.DV_OP_PAGED_ATTN, bd.dims(dh=dh))


def run_attn(K, V, table, lens, q, scale, **kw):
    ws = attn_ws(K.shape[3])
    out, lse = torch.full_like(q, 7.0), torch.full(q.shape[:2], 7.0, device="cuda")
    bd.dv_paged_attn(q, bd.PagedKV(K, V), table, lens, scale, out, ws, lse=lse, **kw)
    torch.cuda.synchronize()
    return out, lse, bd.dv_read_device_status(ws)


def check_attn(out, lse, K, V, table, lens, q, scale, heads=None):
    clean = lambda t: np.nan_to_num(f64(t), nan=0.0, posinf=0.0, neginf=0.0)  # noqa: E731
    Vc = clean(V)
    want, want_lse, bound = attn_model(f64(q), clean(K), Vc, table.tolist(), lens.tolist(), scale, heads)
    tol = (2 * 2.0 ** -18 * bound + 2.0 ** -18) * np.max(np.abs(Vc), initial=1.0)
    err = np.max(np.abs(f64(out) - want), initial=0.0)
    assert err <= tol, (err, tol)
    got_lse = f64(lse)
    empty = np.isneginf(want_lse)
    assert np.array_equal(np.isneginf(got_lse), empty)
    assert np.all(np.abs(got_lse[~empty] - want_lse[~empty]) <= 2.0 ** -18 * bound + 2.0 ** -22 * np.abs(want_lse[~empty]))
    norm = np.linalg.norm(want)
    assert np.linalg.norm(f64(out) - want) <= 2e-5 * norm + 1e-30


LENS = [0, 1, 15, 16, 17, 63, 0, 300, 129, -3]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("dh", [8, 64, 72, 128, 256])
@pytest.mark.parametrize("hq, hkv, page", [(4, 4, 16), (8, 2, 5), (10, 2, 1), (16, 1, 64), (24, 2, 16), (40, 1, 48)])
def test_attention_matches_the_model(dtype, dh, hq, hkv, page):
    K, V, table, lens = make_cache(LENS, hkv, dh, page, dtype, 1000 * dh + hq)
    q = torch.randn(len(LENS), hq, dh, generator=gen(3), device="cuda")
    scale = dh ** -0.5
    out, lse, status = run_attn(K, V, table, lens, q, scale)
    assert status == 0
    check_attn(out, lse, K, V, table, lens, q, scale)
    for b, n in enumerate(LENS):
        if n <= 0:
            assert not out[b].any()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("hkv, G, n, page", [(1, 1, 70001, 16), (1, 8, 30011, 64), (2, 12, 9001, 7), (3, 1, 4096, 128)])
def test_long_rows_are_split_and_joined(dtype, hkv, G, n, page):
    K, V, table, lens = make_cache([n], hkv, 64, page, dtype, n)
    q = 2.0 * torch.randn(1, hkv * G, 64, generator=gen(4), device="cuda")
    out, lse, status = run_attn(K, V, table, lens, q, 0.125)
    assert status == 0
    check_attn(out, lse, K, V, table, lens, q, 0.125)


@pytest.mark.parametrize("B, top, hq, hkv, dh, page, dtype", [
    (300, 40, 4, 2, 64, 8, "bf16"), (1500, 9, 4, 2, 64, 8, "bf16"), (4096, 3, 4, 2, 64, 8, "bf16"), (33, 700, 4, 2, 64, 8, "bf16"),
    (40, 900, 3, 3, 128, 16, "bf16"), (60, 500, 8, 2, 128, 32, "bf16"), (24, 700, 24, 2, 128, 16, "bf16"), (20, 900, 4, 2, 256, 16, "bf16"),
    (20, 900, 3, 3, 256, 16, "f32"), (20, 700, 8, 2, 256, 16, "f32"), (30, 800, 6, 3, 128, 16, "f32"), (33, 600, 3, 3, 64, 16, "f32"),
    (30, 400, 36, 2, 64, 16, "f32"), (40, 600, 5, 5, 96, 16, "bf16"), (30, 600, 16, 2, 96, 24, "f32")])
def test_many_rows_of_different_lengths(B, top, hq, hkv, dh, page, dtype):
    lens = [(i * 7919) % (top + 1) for i in range(B)]
    K, V, table, lens_t = make_cache(lens, hkv, dh, page, BF16 if dtype == "bf16" else F32, B)
    q = torch.randn(B, hq, dh, generator=gen(5), device="cuda")
    out, lse, status = run_attn(K, V, table, lens_t, q, 0.125)
    assert status == 0
    check_attn(out, lse, K, V, table, lens_t, q, 0.125)


@pytest.mark.parametrize("G", [1, 4, 16])
def test_selected_heads_and_rows_behind_the_count(G):
    lens, h = [40, 0, 129, 200], 6
    K, V, table, lens_t = make_cache(lens, h, 128, 16, BF16, G)
    heads = [1, 2, 5]
    kh = 5
    q = torch.randn(4, kh * G, 128, generator=gen(6), device="cuda")
    out, lse, status = run_attn(K, V, table, lens_t, q, 0.09, head_idx=i32(heads + [77, -1]), head_count=i32([3]))
    assert status == 0
    check_attn(out[:, : 3 * G], lse[:, : 3 * G], K, V, table, lens_t, q[:, : 3 * G], 0.09, heads)
    assert (out[:, 3 * G:] == 7.0).all() and (lse[:, 3 * G:] == 7.0).all()
    # an empty set leaves everything; a count above the bound is clamped and flagged
    out, lse, status = run_attn(K, V, table, lens_t, q, 0.09, head_idx=i32(heads + [0, 3]), head_count=i32([0]))
    assert status == 0 and (out == 7.0).all()
    out, lse, status = run_attn(K, V, table, lens_t, q, 0.09, head_idx=i32(heads + [0, 3]), head_count=i32([9]))
    assert status == bd.DV_DEV_COUNT_CLAMPED
    check_attn(out, lse, K, V, table, lens_t, q, 0.09, heads + [0, 3])


def test_bad_pages_heads_and_lengths_are_flagged_and_left_out():
    lens = [40, 33]
    K, V, table, lens_t = make_cache(lens, 2, 64, 16, BF16, 9)
    q = torch.randn(2, 2, 64, generator=gen(7), device="cuda")
    bad = table.clone()
    bad[0, 1] = K.shape[0]  # one past the last page
    bad[1, 0] = -1
    out, lse, status = run_attn(K, V, bad, lens_t, q, 0.125)
    assert status == bd.DV_DEV_INDEX_RANGE
    # the same as a cache without those pages
    short = i32([[int(table[0, 0]), int(table[0, 2]), 0], [int(table[1, 1]), int(table[1, 2]), 0]])
    check_attn(out, lse, K, V, short, i32([24, 17]), q, 0.125)
    out, lse, status = run_attn(K, V, table, lens_t, q, 0.125, head_idx=i32([0, 2]), head_count=i32([2]))
    assert status == bd.DV_DEV_INDEX_RANGE
    assert not out[:, 1].any() and torch.isneginf(lse[:, 1]).all()
    full = table[:, :2].contiguous()  # a table too narrow for the lengths
    out, lse, status = run_attn(K, V, full, lens_t, q, 0.125)
    assert status == bd.DV_DEV_COUNT_CLAMPED
    check_attn(out, lse, K, V, full, i32([32, 32]), q, 0.125)


def test_scores_far_apart_and_scale_zero_or_negative():
    K, V, table, lens = make_cache([200, 77], 2, 64, 16, BF16, 11)
    q = torch.randn(2, 4, 64, generator=gen(8), device="cuda")
    for scale in (30.0, 0.0, -0.125):  # 30: one key takes nearly all the weight
        out, lse, status = run_attn(K, V, table, lens, q, scale)
        assert status == 0
        if scale == 30.0:  # a weight's error is that of its score, 2^-18 of 30 * 64: only the winner is sharp
            want, want_lse, bound = attn_model(f64(q), np.nan_to_num(f64(K)), np.nan_to_num(f64(V)), table.tolist(), lens.tolist(), scale)
            assert np.max(np.abs(f64(out) - want)) <= (2 * 2.0 ** -18 * bound + 2.0 ** -18) * 6
        else:
            check_attn(out, lse, K, V, table, lens, q, scale)


def test_pools_that_share_memory_and_a_page_stride():
    """K and V of two layers in one pool [pages][layer][2][h][page][dh]."""
    h, page, dh = 3, 16, 64
    lens = [50, 17]
    K0, V0, table, lens_t = make_cache(lens, h, dh, page, BF16, 13)
    pool = torch.full((K0.shape[0], 2, 2, h, page, dh), float("nan"), device="cuda", dtype=BF16)
    pool[:, 1, 0], pool[:, 1, 1] = K0, V0
    K, V = pool[:, 1, 0], pool[:, 1, 1]
    assert K.stride(0) == 4 * h * page * dh
    q = torch.randn(2, h, dh, generator=gen(9), device="cuda")
    a = run_attn(K, V, table, lens_t, q, 0.125)
    b = run_attn(K0, V0, table, lens_t, q, 0.125)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]) and a[2] == 0
    ws = bd.workspace(bd.DV_OP_PAGED_APPEND, bd.dims())
    new = torch.randn(2, h, dh, generator=gen(10), device="cuda")
    bd.dv_paged_append(bd.PagedKV(K, V), new, -new, i32([5, -1]), ws)
    torch.cuda.synchronize()
    assert torch.equal(K[0, :, 5], new[0].to(BF16)) and torch.equal(V[0, :, 5], -new[0].to(BF16))
    assert torch.isnan(pool[:, 0]).all()


def test_results_repeat_bit_for_bit_and_workspace_is_left_ready():
    K, V, table, lens = make_cache([5000, 3, 1200, 0, 64], 2, 128, 16, BF16, 17)
    q = torch.randn(5, 8, 128, generator=gen(11), device="cuda")
    kv, ws = bd.PagedKV(K, V), attn_ws(128)
    first = None
    for _ in range(20):
        out = torch.empty_like(q)
        bd.dv_paged_attn(q, kv, table, lens, 0.1, out, ws)
        torch.cuda.synchronize()
        first = out if first is None else first
        assert torch.equal(out, first)
    assert not ws[: 72 * 1024].any()  # counters and status are zero again


def test_two_streams_with_their_own_workspaces():
    K, V, table, lens = make_cache([3000, 900], 4, 64, 16, BF16, 19)
    kv = bd.PagedKV(K, V)
    qs = [torch.randn(2, 4, 64, generator=gen(20 + i), device="cuda") for i in range(2)]
    want = [run_attn(K, V, table, lens, q, 0.125)[0] for q in qs]
    streams, wss, outs = [torch.cuda.Stream() for _ in range(2)], [attn_ws(64) for _ in range(2)], [torch.empty_like(q) for q in qs]
    torch.cuda.synchronize()
    for _ in range(10):
        for s, ws, q, out in zip(streams, wss, qs, outs):
            bd.dv_paged_attn(q, kv, table, lens, 0.125, out, ws, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, want))


def test_offsets_past_32_bits():
    """Pages behind element 2^31 (and byte 2^32) of the pools."""
    h, page, dh = 4, 64, 256
    per = h * page * dh
    n_pages = (2 ** 31 + 2 ** 20) // per + 4
    K = torch.empty(n_pages, h, page, dh, device="cuda", dtype=BF16)
    V = torch.empty(n_pages, h, page, dh, device="cuda", dtype=BF16)
    lens = [130, 64]
    table = i32([[n_pages - 1, 0, n_pages - 3], [n_pages - 2, 0, 0]])
    g = gen(23)
    k, v = torch.randn(194, h, dh, generator=g, device="cuda"), torch.randn(194, h, dh, generator=g, device="cuda")
    slots = [int(table[0, s // page]) * page + s % page for s in range(130)] + [int(table[1, 0]) * page + s for s in range(64)]
    ws = bd.workspace(bd.DV_OP_PAGED_APPEND, bd.dims())
    bd.dv_paged_append(bd.PagedKV(K, V), k, v, i32(slots), ws)
    q = torch.randn(2, h, dh, generator=g, device="cuda")
    out, lse, status = run_attn(K, V, table, i32(lens), q, 1 / 16)
    assert status == 0 and bd.dv_read_device_status(ws) == 0
    keep = torch.tensor([0, n_pages - 3, n_pages - 2, n_pages - 1], device="cuda")
    small = i32([[3, 0, 1], [2, 0, 0]])
    Ks, Vs = K[keep].clone(), V[keep].clone()
    assert torch.equal(Ks[3, :, 7], k[7].to(BF16)) and torch.equal(Vs[2, :, 63], v[193].to(BF16))
    again = run_attn(Ks, Vs, small, i32(lens), q, 1 / 16)
    assert torch.equal(out, again[0])
    check_attn(out, lse, Ks, Vs, small, i32(lens), q, 1 / 16)


# ---------------------------------------------------------------------------
# append
# ---------------------------------------------------------------------------


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T, h, dh, page", [(1, 1, 8, 1), (7, 3, 64, 5), (33, 32, 128, 16), (1000, 2, 72, 48), (5, 2, 256, 3)])
def test_append_stores_rounded_rows_and_nothing_else(dtype, T, h, dh, page):
    g = gen(T)
    n_pages = -(-T // page) + 2
    K = torch.randn(n_pages, h, page, dh, generator=g, device="cuda").to(dtype)
    V = torch.randn(n_pages, h, page, dh, generator=g, device="cuda").to(dtype)
    k, v = torch.randn(T, h, dh, generator=g, device="cuda"), torch.randn(T, h, dh, generator=g, device="cuda")
    k[0, 0, 0], v[0, 0, 0] = float("inf"), float("nan")
    slots = torch.randperm(n_pages * page, generator=g, device="cuda")[:T].to(torch.int32)
    if T > 2:
        slots[1] = -1
        slots[2] = -2 ** 31
    K2, V2 = K.clone(), V.clone()
    for t, s in enumerate(slots.tolist()):
        if s >= 0:
            K2[s // page, :, s % page], V2[s // page, :, s % page] = k[t].to(dtype), v[t].to(dtype)
    ws = bd.workspace(bd.DV_OP_PAGED_APPEND, bd.dims())
    bd.dv_paged_append(bd.PagedKV(K, V), k, v, slots, ws)
    assert bd.dv_read_device_status(ws) == 0
    same = lambda x, y: torch.equal(torch.nan_to_num(x.float(), nan=9e9), torch.nan_to_num(y.float(), nan=9e9))  # noqa: E731
    assert same(K, K2) and same(V, V2)
    slots[0] = n_pages * page
    before = K.clone(), V.clone()
    bd.dv_paged_append(bd.PagedKV(K, V), k, v, torch.where(slots == n_pages * page, slots, -1), ws)
    assert bd.dv_read_device_status(ws) == bd.DV_DEV_INDEX_RANGE
    assert same(K, before[0]) and same(V, before[1])


def test_append_of_no_tokens():
    K = torch.zeros(2, 1, 4, 8, device="cuda")
    ws = bd.workspace(bd.DV_OP_PAGED_APPEND, bd.dims())
    e = torch.empty(0, 1, 8, device="cuda")
    bd.dv_paged_append(bd.PagedKV(K, K.clone()), e, e, i32([]), ws)


# ---------------------------------------------------------------------------
# block tables
# ---------------------------------------------------------------------------


def random_tables(R, W, page, seed, spare):
    r = np.random.RandomState(seed)
    lens = r.randint(0, W * page + 1, R)
    lens[r.rand(R) < 0.2] = 0
    want = np.where(r.rand(R) < 0.4, np.minimum(lens + 1, W * page + 1), r.randint(0, W * page + 2, R))
    want = np.where(r.rand(R) < 0.15, -1, np.where(r.rand(R) < 0.15, 0, want))
    n = -(-lens // page)
    free = int(spare * n.sum()) if spare else 0
    n_pages = int(n.sum()) + free + 1
    order = r.permutation(n_pages)
    table, at = np.full((R, W), -1, dtype=np.int64), 0
    for b in range(R):
        table[b, : n[b]] = order[at:at + n[b]]
        at += n[b]
    return dict(want=want.tolist(), lens=lens.tolist(), table=table.tolist(), free=order[at:at + free].tolist(), page=page,
                n_pages=n_pages)


def run_tables(m, max_tokens, alias=False):
    R, n = len(m["want"]), m["n_pages"]
    want, lens, table = i32(m["want"]), i32(m["lens"]), i32(m["table"])
    stack = i32(m["free"] + [-9] * (n - len(m["free"])))
    count = i32([len(m["free"])])
    lens_out, count_out = (lens, count) if alias else (i32([77] * R), i32([77]))
    slots, offsets, granted = i32([77] * max_tokens), i32([77] * (R + 1)), i32([77] * R)
    ws = bd.workspace(bd.DV_OP_PAGE_TABLES, bd.dims())
    bd.dv_page_tables(want, lens, lens_out, table, stack, count, count_out, slots, offsets, granted, m["page"], ws)
    status = bd.dv_read_device_status(ws)
    return dict(lens=lens_out.tolist(), table=table.tolist(), stack=stack.tolist(), free_count=count_out.item(),
                slots=slots.tolist(), offsets=offsets.tolist(), granted=granted.tolist()), status


@pytest.mark.parametrize("alias", [False, True])
@pytest.mark.parametrize("R, W, page, spare, max_tokens", [
    (1, 1, 1, 1.0, 4), (1, 4, 16, 0, 0), (5, 3, 4, 0.5, 40), (64, 7, 16, 0.3, 3001), (64, 7, 16, 3.0, 100000),
    (1025, 3, 5, 0.4, 9000), (1500, 6, 33, 0.1, 70000), (4096, 2, 8, 1.0, 20001)])
def test_page_tables_match_the_model(R, W, page, spare, max_tokens, alias):
    m = random_tables(R, W, page, R + W, spare)
    want = tables_model(**m, max_tokens=max_tokens)
    got, status = run_tables(m, max_tokens, alias)
    for n in ("granted", "lens", "offsets", "table", "free_count", "slots"):
        assert got[n] == want[n], n
    assert got["stack"][: len(want["stack"])] == want["stack"]
    assert status == (0 if all(want["granted"]) else bd.DV_DEV_REFUSED)
    # no page is held twice, none is lost
    pages = lambda n: -(-n // page)  # noqa: E731
    held = [p for r, n in zip(got["table"], got["lens"]) for p in r[: pages(n)]] + got["stack"][: got["free_count"]]
    assert len(held) == len(set(held)) == m["n_pages"] - 1


def test_page_tables_flag_what_is_not_a_length_or_a_count():
    m = dict(want=[5, 2, 3], lens=[-4, 99, 2], table=[[0, 1], [2, 3], [4, -1]], free=[5, 6], page=2, n_pages=7)
    got, status = run_tables(m, 8)
    assert status == bd.DV_DEV_INDEX_RANGE | bd.DV_DEV_REFUSED
    assert got["granted"] == [0, 0, 1] and got["lens"] == [-4, 99, 3]
    assert got["table"][2] == [4, 6] and got["slots"] == [12] + [-1] * 7 and got["free_count"] == 1


@pytest.mark.parametrize("n_pages, count", [(12, 12), (2 ** 31 - 1, 2 ** 31 - 1)])
def test_page_tables_clamp_a_free_count_that_leaves_no_room(n_pages, count):
    """More free pages than the stack holds once pages come back: flagged, nothing is pushed behind its end."""
    stack = torch.full((n_pages,), 5, dtype=torch.int32, device="cuda")
    table, free = i32([[1, 2], [-1, -1]]), i32([count])
    slots, offsets, granted, lens = i32([9, 9]), i32([9] * 3), i32([9, 9]), i32([2, 0])
    ws = bd.workspace(bd.DV_OP_PAGE_TABLES, bd.dims())
    bd.dv_page_tables(i32([0, 1]), lens, lens, table, stack, free, free, slots, offsets, granted, 1, ws)
    assert bd.dv_read_device_status(ws) == bd.DV_DEV_INDEX_RANGE
    assert lens.tolist() == [0, 1] and granted.tolist() == [1, 1] and offsets.tolist() == [0, 0, 1]
    assert free.item() == n_pages - 1 and table.tolist() == [[1, 2], [5, -1]] and slots.tolist() == [5, -1]
    assert (stack[:: max(1, n_pages // 1000)] == 5).all() and (stack[-8:] == 5).all()


def test_page_tables_repeat_from_the_same_lengths():
    m = random_tables(40, 5, 8, 3, 0.6)
    a = run_tables(m, 500)[0]
    m2 = dict(m, table=a["table"])
    b = run_tables(dict(m2, free=a["stack"][: len(m["free"])]), 500)[0]
    assert {n: a[n] for n in a if n != "stack"} == {n: b[n] for n in b if n != "stack"}


# ---------------------------------------------------------------------------
# the attention block, and all of it together
# ---------------------------------------------------------------------------


def mha_model(t, y, Kf, Vf, table, lens, slots, heads, scale, page, exact, bias):
    """Row by row in 64 bits; K, V (float64, what the pools hold) are updated."""
    Wqkv, WOt = f64(t["Wqkv"]), f64(t["WOt"])
    h, _, dh, d = Wqkv.shape
    low = t["Wqkv"].dtype == BF16
    kept = (lambda x: f64(torch.from_numpy(x).float().to(BF16))) if low else (lambda x: x)
    out = np.zeros(y.shape)
    for b in range(y.shape[0]):
        if slots[b] >= 0:
            p, o = divmod(int(slots[b]), page)
            Kf[p, :, o], Vf[p, :, o] = 0.0, 0.0
            for i in range(h) if exact else heads:
                Kf[p, i, o] = kept(Wqkv[i, 1] @ y[b] + (f64(t["bqkv"])[i, 1] if bias else 0.0))
                Vf[p, i, o] = kept(Wqkv[i, 2] @ y[b] + (f64(t["bqkv"])[i, 2] if bias else 0.0))
    q = np.stack([[Wqkv[i, 0] @ y[b] + (f64(t["bqkv"])[i, 0] if bias else 0.0) for i in heads] for b in range(y.shape[0])]) \
        if heads else np.zeros((y.shape[0], 0, dh))
    if heads:
        H, _, _ = attn_model(q, Kf, Vf, table, lens, scale, heads)
        for j, i in enumerate(heads):
            out += H[:, j] @ WOt[i]
    return out + (f64(t["bO"]) if bias else 0.0)


@pytest.mark.parametrize("wdt", ["bf16", "f32"])
@pytest.mark.parametrize("B, dh, heads, exact, acc, bias", [
    (1, 64, [0, 3], False, False, True), (1, 128, [2], True, True, False), (4, 64, [0, 1, 2, 3], False, True, True),
    (3, 128, [1, 3], True, False, True), (8, 64, [0, 2], False, False, True), (16, 64, [1], True, True, False),
    (2, 64, [], False, False, True), (2, 64, [], False, True, False), (2, 64, [], True, False, True)])
def test_sparse_mha_paged_matches_the_model(wdt, B, dh, heads, exact, acc, bias):
    d, h, page = 512, 4, 16
    s = wl.LayerShape(d=d, N=1024, r=32, h=h, dh=dh, L=8, cap=9, B=1, wdtype=wdt, kvdtype=wdt)
    t = wl.make_layer(s, 5, "cuda")
    t["bqkv"] = 0.3 * torch.randn(h, 3, dh, generator=gen(1), device="cuda")
    t["bO"] = 0.3 * torch.randn(d, generator=gen(2), device="cuda")
    lens = [(37 * (b + 1)) % 90 for b in range(B)]
    if B > 2:
        lens[1] = 0
    K, V, table, lens_t = make_cache(lens, h, dh, page, t["Wqkv"].dtype, B)
    slots = [int(table[b, (n - 1) // page]) * page + (n - 1) % page if n > 0 else -1 for b, n in enumerate(lens)]
    y = torch.randn(B, d, generator=gen(B), device="cuda")
    out0 = torch.randn(B, d, generator=gen(3), device="cuda")
    out, kh = out0.clone(), len(heads)
    ws = bd.workspace(bd.DV_OP_SPARSE_MHA_PAGED, bd.dims(B=B, d=d, h=h, dh=dh, kh_max=kh))
    Kf, Vf = np.nan_to_num(f64(K)), np.nan_to_num(f64(V))
    want = mha_model(t, f64(y), Kf, Vf, table.tolist(), lens, slots, heads, dh ** -0.5, page, exact, bias)
    for _ in range(2):  # (a second call with the same slots stores the same and gives the same)
        out.copy_(out0)
        bd.dv_sparse_mha_paged(y, t["Wqkv"], t["bqkv"] if bias else None, t["WOt"], t["bO"] if bias else None, bd.PagedKV(K, V),
                               table, lens_t, i32(slots), dh ** -0.5, i32(heads + [0] * 4), i32([kh]), kh, out, ws,
                               accumulate=acc, exact_kv=exact)
        torch.cuda.synchronize()
        assert bd.dv_read_device_status(ws) == 0
    got = f64(out) - (f64(out0) if acc else 0.0)
    # the projections' bar of the contiguous call (tests/_helpers.py): 5e-3 in the 2-norm, 2e-2 at the largest
    assert np.linalg.norm(got - want) <= 5e-3 * np.linalg.norm(want) + 1e-6
    assert np.max(np.abs(got - want)) <= 2e-2 * np.max(np.abs(want)) + 1e-6
    Kg, Vg = f64(K), f64(V)
    for b, sl in enumerate(slots):
        if sl < 0:
            continue
        p, o = divmod(sl, page)
        for i in range(h):
            if not exact and i not in heads:
                assert not Kg[p, i, o].any() and not Vg[p, i, o].any()
            for got_row, want_row in ((Kg[p, i, o], Kf[p, i, o]), (Vg[p, i, o], Vf[p, i, o])):
                scale = np.max(np.abs(want_row), initial=0.0)
                assert np.all(np.abs(got_row - want_row) <= np.abs(want_row) * 2.0 ** -7 + scale * 2.0 ** -12)


@pytest.mark.parametrize("B, d, h, heads, exact", [
    (7, 5000, 32, list(range(32)), False),  # channels in segments, weight tiles in several passes, odd blocks
    (2, 20480, 3, [0, 2], True),            # more column blocks of W^O than SMs
    (1, 12296, 40, list(range(0, 40, 2)), False), (1, 1000, 64, list(range(64)), False), (1, 4104, 40, [3, 39], True),
    (3, 264, 8, [7], True), (8, 1032, 5, [0, 1, 2, 3, 4], False), (1, 8, 2, [1], False), (5, 16, 2, [0], True)])
def test_sparse_mha_paged_at_sizes_that_do_not_divide(B, d, h, heads, exact):
    dh, page = 64, 12
    g = gen(d)
    W = (torch.randn(h, 3, dh, d, generator=g, device="cuda") * d ** -0.5).to(BF16)
    WOt = (torch.randn(h, dh, d, generator=g, device="cuda") * d ** -0.5).to(BF16)
    bqkv = 0.3 * torch.randn(h, 3, dh, generator=g, device="cuda")
    lens = [(29 * (b + 1)) % 60 + 1 for b in range(B)]
    K, V, table, lens_t = make_cache(lens, h, dh, page, BF16, B)
    pool = torch.full((K.shape[0], 2, h, page, dh), float("nan"), device="cuda", dtype=BF16)  # K and V share a pool
    pool[:, 0], pool[:, 1] = K, V
    K, V = pool[:, 0], pool[:, 1]
    slots = [int(table[b, (n - 1) // page]) * page + (n - 1) % page for b, n in enumerate(lens)]
    y = torch.randn(B, d, generator=g, device="cuda")
    out = torch.full((B, d), 7.0, device="cuda")
    Kf, Vf = torch.nan_to_num(K.double()), torch.nan_to_num(V.double())
    qkv = torch.einsum("bd,hmcd->bhmc", y.double(), W.double()) + bqkv.double()
    ws = bd.workspace(bd.DV_OP_SPARSE_MHA_PAGED, bd.dims(B=B, d=d, h=h, dh=dh, kh_max=len(heads)))
    bd.dv_sparse_mha_paged(y, W, bqkv, WOt, None, bd.PagedKV(K, V), table, lens_t, i32(slots), 0.125, i32(heads), i32([len(heads)]),
                           len(heads), out, ws, exact_kv=exact)
    torch.cuda.synchronize()
    assert bd.dv_read_device_status(ws) == 0
    want = torch.zeros(B, d, dtype=torch.float64, device="cuda")
    for b, sl in enumerate(slots):
        p, o = divmod(sl, page)
        Kf[p, :, o], Vf[p, :, o] = 0, 0
        for i in range(h) if exact else heads:
            # a stored value is the product's, rounded once: half a step of bf16, and the fp32 sum's error of 2^-18 of its terms
            for pool, dst, m in ((K, Kf, 1), (V, Vf, 2)):
                ref = qkv[b, i, m]
                mag = (y[b].double().abs() * W[i, m].double().abs()).sum(1) + bqkv[i, m].double().abs()
                assert ((pool[p, i, o].double() - ref).abs() <= ref.abs() * 2.0 ** -8 + mag * 2.0 ** -18).all()
                dst[p, i, o] = pool[p, i, o].double()  # (the attention reads what the pages hold)
        if not exact:
            for i in set(range(h)) - set(heads):
                assert not K[p, i, o].any() and not V[p, i, o].any()
        for i in heads:
            pages = table[b, : -(-lens[b] // page)].long()
            k, v = (t[pages, i].reshape(-1, dh)[: lens[b]] for t in (Kf, Vf))
            want[b] += (torch.softmax((k @ qkv[b, i, 0]) * 0.125, 0) @ v) @ WOt[i].double()
    # 64 len(heads) terms a sum, each of fp32 operands in three bf16 terms: far inside 2^-16 of the result's norm
    assert (out.double() - want).norm() <= 2.0 ** -16 * want.norm()


def block_case(B, d, h, dh, heads, lens, seed, page=8, dtype=BF16, bias=True):
    """Inputs of the attention block over pages, in one dict; the pool's slots past the lengths hold NaN."""
    g = gen(seed)
    K, V, table, lens_t = make_cache(lens, h, dh, page, dtype, seed)
    return dict(
        y=torch.randn(B, d, generator=g, device="cuda"), Wqkv=(torch.randn(h, 3, dh, d, generator=g, device="cuda") * d ** -0.5).to(dtype),
        WOt=(torch.randn(h, dh, d, generator=g, device="cuda") * d ** -0.5).to(dtype),
        bqkv=0.3 * torch.randn(h, 3, dh, generator=g, device="cuda") if bias else None,
        bO=0.3 * torch.randn(d, generator=g, device="cuda") if bias else None, K=K, V=V, table=table, lens=lens_t, page=page, heads=heads,
        slots=i32([int(table[b, (n - 1) // page]) * page + (n - 1) % page if n > 0 else -1 for b, n in enumerate(lens)]))


def run_block(c, ws=None, exact=False, accumulate=False, out=None, idx=None, count=None, kh=None):
    B, d = c["y"].shape
    h, dh = c["K"].shape[1], c["K"].shape[3]
    idx = c["heads"] if idx is None else idx
    kh = len(idx) if kh is None else kh
    ws = bd.workspace(bd.DV_OP_SPARSE_MHA_PAGED, bd.dims(B=B, d=d, h=h, dh=dh, kh_max=kh)) if ws is None else ws
    out = torch.full((B, d), 7.0, device="cuda") if out is None else out
    bd.dv_sparse_mha_paged(c["y"], c["Wqkv"], c["bqkv"], c["WOt"], c["bO"], bd.PagedKV(c["K"], c["V"]), c["table"], c["lens"], c["slots"],
                           dh ** -0.5, i32(list(idx) + [0]), i32([len(idx) if count is None else count]), kh, out, ws, accumulate=accumulate,
                           exact_kv=exact)
    torch.cuda.synchronize()
    return out, bd.dv_read_device_status(ws)


def block_sums(c):
    """(q, k, v) of every head [B][h][3][dh] in 64 bits, bias included, and the sum of their terms' magnitudes."""
    y, W = c["y"].double(), c["Wqkv"].double()
    s, m = torch.einsum("bd,hmcd->bhmc", y, W), torch.einsum("bd,hmcd->bhmc", y.abs(), W.abs())
    return (s, m) if c["bqkv"] is None else (s + c["bqkv"].double(), m + c["bqkv"].double().abs())


def block_out(c, q):
    """The block's output in 64 bits, from q [B][h][dh] and the keys and values that the pages hold now."""
    out = torch.zeros_like(c["y"], dtype=torch.float64)
    for b, n in enumerate(c["lens"].tolist()):
        if n > 0:
            pages = c["table"][b, : -(-n // c["page"])].long()
            for i in c["heads"]:
                k, v = (c[x][pages, i].reshape(-1, q.shape[2])[:n].double() for x in "KV")
                out[b] += (torch.softmax((k @ q[b, i]) * q.shape[2] ** -0.5, 0) @ v) @ c["WOt"][i].double()
    return out if c["bO"] is None else out + c["bO"].double()


@pytest.mark.parametrize("B, d, h, dh, n", [(1, 4096, 32, 128, 2), (1, 2048, 32, 64, 1), (2, 2048, 24, 64, 3), (3, 4096, 32, 128, 2),
                                            (4, 4096, 20, 128, 4), (5, 1000, 40, 64, 8), (8, 2048, 32, 64, 2), (1, 12296, 12, 128, 5)])
@pytest.mark.parametrize("seed", range(4))
def test_a_block_stores_what_the_exact_sums_round_to(B, d, h, dh, n, seed):
    """With few keys one bf16 step of one stored value moves the output by more than all its fp32 sums' errors, so the
    stored values must not depend on how a sum was formed: they are the 64-bit sums rounded to fp32, then to bf16, every
    one. (Only a sum within 2^-40 of its terms of an fp32 border that decides might not be: one in 10^9.)"""
    c = block_case(B, d, h, dh, list(range(h)), [max(1, n - b % 2) for b in range(B)], 100 * seed + B + d)
    sums, _ = block_sums(c)
    out, status = run_block(c)
    assert status == 0
    want = sums.float().to(BF16)
    for b, sl in enumerate(c["slots"].tolist()):
        p, o = divmod(sl, c["page"])
        assert torch.equal(c["K"][p, :, o], want[b, :, 1]) and torch.equal(c["V"][p, :, o], want[b, :, 2])
    # and so the output is within fp32 rounding of the definition's: chains of at most 24 tensor core steps, the scores' and
    # the weights' a few more, each off by 2^-23 of its partial sum at most: 64 of them
    ref = block_out(c, sums[:, :, 0])
    assert (out.double() - ref).norm() <= 64 * 2.0 ** -23 * ref.norm()


@pytest.mark.parametrize("B, d", [(1, 64), (2, 64), (3, 8), (8, 136), (1, 520), (4, 640)])
def test_a_block_of_few_channels_stores_what_the_exact_sums_round_to(B, d):
    """Few channels: one warp or two have all of a sum's terms, and a value may be far smaller than they are."""
    h, dh = 512, 128
    c = block_case(B, d, h, dh, list(range(h)), [2] * B, d + B)
    sums, _ = block_sums(c)
    _, status = run_block(c)
    assert status == 0
    want = sums.float().to(BF16)
    for b, sl in enumerate(c["slots"].tolist()):
        p, o = divmod(sl, c["page"])
        assert torch.equal(c["K"][p, :, o], want[b, :, 1]) and torch.equal(c["V"][p, :, o], want[b, :, 2])


@pytest.mark.parametrize("B, h", [(1, 128), (8, 40), (5, 128)])
def test_a_block_whose_sums_all_lie_at_a_border(B, h):
    """Every k and v is 257, half way between two bf16 values, or 2^-12 to either side of it."""
    d, dh = 64, 128
    c = block_case(B, d, h, dh, list(range(h)), [3] * B, 5, bias=False)
    c["y"].fill_(0.0)
    c["y"][:, :3] = torch.tensor([2.0, 0.5, 2.0 ** -6], device="cuda")
    c["y"] *= torch.where(torch.arange(B, device="cuda") % 2 == 0, 1.0, -1.0)[:, None]
    c["Wqkv"][..., 0], c["Wqkv"][..., 1] = 128.0, 2.0
    c["Wqkv"][..., 2] = (torch.randint(-1, 2, (h, 3, dh), generator=gen(6), device="cuda") * 2.0 ** -6).to(BF16)
    sums, _ = block_sums(c)
    assert set(sums.abs().unique().tolist()) == {257 - 2.0 ** -12, 257.0, 257 + 2.0 ** -12}
    _, status = run_block(c)
    assert status == 0
    want = sums.float().to(BF16)
    for b, sl in enumerate(c["slots"].tolist()):
        p, o = divmod(sl, c["page"])
        assert torch.equal(c["K"][p, :, o], want[b, :, 1]) and torch.equal(c["V"][p, :, o], want[b, :, 2])


@pytest.mark.parametrize("B", [1, 2, 8])
@pytest.mark.parametrize("bad", [5000, -1])
def test_a_block_of_many_heads_whose_set_names_none(B, bad):
    """The largest tile list: 1000 entries out of range, k and v of all 1024 heads stored."""
    h, dh, d = 1024, 128, 64
    c = block_case(B, d, h, dh, [], [1 + b % 2 for b in range(B)], B, page=1)
    out, status = run_block(c, exact=True, idx=[bad] * 1000)
    assert status == bd.DV_DEV_INDEX_RANGE
    sums, _ = block_sums(c)
    want = sums.float().to(BF16)
    for b, p in enumerate(c["slots"].tolist()):
        assert torch.equal(c["K"][p, :, 0], want[b, :, 1]) and torch.equal(c["V"][p, :, 0], want[b, :, 2])
    assert torch.equal(out, c["bO"].expand(B, d))


def check_block(c, out, exact=False, out0=None):
    """The block's output and the rows that it stored against 64 bits.

    A stored value is its sum rounded once: half a step of the pool's type (bf16 2^-8, fp32 2^-24), and the sum's error: fp32
    chains of at most 64 steps, 2^-18 of the terms' magnitudes. The output is compared with the attention over what the pages
    hold, and 64 chained steps of 2^-23 make 2^-17 of its norm, with the scores' and weights' 2^-16. From nine requests on, with
    bf16 weights, y and the attention's result enter as two bf16 terms: each value off by 2^-18, independently, so q by
    2^-18 of its norm, scores by 2^-18 |q| |k| scale <= 2^-15 here, weights by 2^-14, the output by less than 2^-13."""
    two = c["K"].dtype == BF16 and c["y"].shape[0] > 8
    sums, mags = block_sums(c)
    half = 2.0 ** -8 if c["K"].dtype == BF16 else 2.0 ** -24
    n = c["K"].shape[0] * c["page"]
    for b, sl in enumerate(c["slots"].tolist()):
        if not 0 <= sl < n:
            continue
        p, o = divmod(sl, c["page"])
        for i in range(c["K"].shape[1]):
            for pool, m in (("K", 1), ("V", 2)):
                got = c[pool][p, i, o].double()
                if not exact and i not in c["heads"]:
                    assert not got.any()
                else:
                    ref, mag = sums[b, i, m], mags[b, i, m]
                    assert ((got - ref).abs() <= ref.abs() * half + mag * (2.0 ** -17 if two else 2.0 ** -18)).all()
    ref = block_out(c, sums[:, :, 0])
    got = out.double() - (0 if out0 is None else out0.double())
    err = (got - ref).norm() - (0 if out0 is None else 2.0 ** -24 * out.double().norm())  # (one fp32 addition more)
    assert err <= (2.0 ** -13 if two else 2.0 ** -16) * ref.norm()


KINDS = [(BF16, 1), (BF16, 4), (BF16, 8), (BF16, 9), (BF16, 13), (BF16, 16), (F32, 1), (F32, 4), (F32, 16)]


def kind_case(dtype, B, heads, seed=0, top=60):
    return block_case(B, 512, 6, 64, heads, [(23 * (b + 1)) % top + (b != 2) for b in range(B)], 10 * B + seed, dtype=dtype)


@pytest.mark.parametrize("exact, acc", [(False, False), (True, False), (False, True)])
@pytest.mark.parametrize("dtype, B", KINDS)
def test_a_block_in_every_form(dtype, B, exact, acc):
    c = kind_case(dtype, B, [0, 2, 3, 5])
    out0 = torch.randn(B, 512, generator=gen(4), device="cuda")
    for _ in range(2):
        out, status = run_block(c, exact=exact, accumulate=acc, out=out0.clone())
        assert status == 0
        check_block(c, out, exact=exact, out0=out0 if acc else None)


@pytest.mark.parametrize("exact", [False, True])
@pytest.mark.parametrize("dtype, B", KINDS)
def test_a_block_skips_and_flags_what_is_out_of_range(dtype, B, exact):
    # heads out of range between valid ones: as without them
    c = kind_case(dtype, B, [1, 4], 1)
    out, status = run_block(c, exact=exact, idx=[-1, 1, 6, 4, 2 ** 31 - 1], kh=5)
    assert status == bd.DV_DEV_INDEX_RANGE
    check_block(c, out, exact=exact)
    # a count above the bound, and below zero: clamped
    c = kind_case(dtype, B, [0, 3], 2)
    out, status = run_block(c, exact=exact, idx=[0, 3, 5], count=3, kh=2)
    assert status == bd.DV_DEV_COUNT_CLAMPED
    check_block(c, out, exact=exact)
    c = kind_case(dtype, B, [], 3)
    out, status = run_block(c, exact=exact, idx=[0, 3], count=-7)
    assert status == bd.DV_DEV_COUNT_CLAMPED
    check_block(c, out, exact=exact)
    # a slot outside the pools, and a negative one: nothing is stored, the pages hold what they held
    c = kind_case(dtype, B, [2, 5], 4)
    c["slots"][0] = c["K"].shape[0] * c["page"]
    if B > 1:
        c["slots"][1] = -5
    held = c["K"].clone(), c["V"].clone()
    out, status = run_block(c, exact=exact)
    assert status == bd.DV_DEV_INDEX_RANGE
    check_block(c, out, exact=exact)
    mine = torch.ones(c["K"].shape[0], c["page"], dtype=torch.bool, device="cuda")
    for sl in c["slots"].tolist():
        if 0 <= sl < mine.numel():
            mine[sl // c["page"], sl % c["page"]] = False
    for now, before in zip((c["K"], c["V"]), held):
        same = (now == before) | (now.isnan() & before.isnan())
        assert same.transpose(1, 2)[mine].all()
    # a page out of range: its keys are left out; the new token's slot is another request's page, which stays whole
    c = kind_case(dtype, B, [0, 1, 2], 5, 100)
    c["lens"][0], c["slots"][0] = 20, -1
    pages = c["table"][0].clone()
    c["table"][0, 1] = c["K"].shape[0]
    out, status = run_block(c, exact=exact)
    assert status == bd.DV_DEV_INDEX_RANGE
    c["table"][0, 1], c["lens"][0] = pages[2], 12  # the keys of pages 0 and 2
    check_block(c, out, exact=exact)


@pytest.mark.parametrize("dtype, B", [(BF16, 1), (BF16, 5), (BF16, 12), (F32, 3)])
def test_blocks_on_two_streams_and_in_two_graphs(dtype, B):
    """Two layers' blocks at once, each with its own workspace: eager on two streams, then two graphs replayed on them."""
    cs = [kind_case(dtype, B, [0, 2, 3], 7 + i) for i in range(2)]
    want = [run_block(c)[0] for c in cs]
    # fp32 weights add their partial sums by float atomics: at most 3 * 64 terms in any order, 2^-24 each of a partial sum
    near = lambda a, b: torch.equal(a, b) if dtype == BF16 else (a - b).norm() <= 192 * 2.0 ** -24 * 192 ** 0.5 * b.norm()  # noqa: E731
    wss = [bd.workspace(bd.DV_OP_SPARSE_MHA_PAGED, bd.dims(B=B, d=512, h=6, dh=64, kh_max=3)) for _ in cs]
    kvs, outs = [bd.PagedKV(c["K"], c["V"]) for c in cs], [torch.empty(B, 512, device="cuda") for _ in cs]
    idx, cnt = i32([0, 2, 3]), i32([3])
    streams, graphs = [torch.cuda.Stream() for _ in cs], [torch.cuda.CUDAGraph() for _ in cs]

    def call(i, stream=None):
        c = cs[i]
        bd.dv_sparse_mha_paged(c["y"], c["Wqkv"], c["bqkv"], c["WOt"], c["bO"], kvs[i], c["table"], c["lens"], c["slots"], 0.125, idx, cnt, 3,
                               outs[i], wss[i], stream=stream)

    torch.cuda.synchronize()
    for _ in range(10):
        for i, s in enumerate(streams):
            call(i, s)
    torch.cuda.synchronize()
    assert all(near(a, b) for a, b in zip(outs, want))
    for i, s in enumerate(streams):
        with torch.cuda.graph(graphs[i], stream=s):
            for _ in range(3):
                call(i)
        outs[i].fill_(9.0)
    torch.cuda.synchronize()
    for _ in range(5):
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    assert all(near(a, b) for a, b in zip(outs, want)) and all(bd.dv_read_device_status(ws) == 0 for ws in wss)


def test_a_block_captured_and_replayed_follows_its_inputs():
    """One captured dv_sparse_mha_paged, replayed after the lengths, slots, set and input changed in place."""
    d, h, dh, page, B = 512, 6, 64, 8, 3
    g = gen(77)
    W = (torch.randn(h, 3, dh, d, generator=g, device="cuda") * d ** -0.5).to(BF16)
    WOt = (torch.randn(h, dh, d, generator=g, device="cuda") * d ** -0.5).to(BF16)
    full = [70, 9, 33]
    K, V, table, lens = make_cache(full, h, dh, page, BF16, 5, junk=0.0)
    kv, kh = bd.PagedKV(K, V), 4
    y, out = torch.randn(B, d, generator=g, device="cuda"), torch.empty(B, d, device="cuda")
    slots, idx, cnt = i32([-1] * B), i32([0, 1, 2, 3]), i32([4])
    wss = [bd.workspace(bd.DV_OP_SPARSE_MHA_PAGED, bd.dims(B=B, d=d, h=h, dh=dh, kh_max=kh)) for _ in range(2)]

    def call(o, ws):
        bd.dv_sparse_mha_paged(y, W, None, WOt, None, kv, table, lens, slots, 0.125, idx, cnt, kh, o, ws)

    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call(out, wss[0])
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=side):
            call(out, wss[0])
    torch.cuda.current_stream().wait_stream(side)
    for it, (ln, heads) in enumerate([([70, 9, 33], [0, 1, 2, 3]), ([12, 0, 33], [2, 5]), ([1, 8, 17], [4]), ([64, 9, 0], [])]):
        lens.copy_(i32(ln))
        slots.copy_(i32([int(table[b, (n - 1) // page]) * page + (n - 1) % page if n else -1 for b, n in enumerate(ln)]))
        idx[: len(heads)] = i32(heads)
        cnt.copy_(i32([len(heads)]))
        y.copy_(torch.randn(B, d, generator=g, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        again = torch.empty_like(out)
        call(again, wss[1])
        torch.cuda.synchronize()
        assert torch.equal(out, again)  # the same sums in the same order, whatever the launch
        if not heads:
            assert not out.any()
    assert all(bd.dv_read_device_status(ws) == 0 for ws in wss)


def test_paged_block_equals_the_contiguous_one():
    """Equal lengths, the same values: dv_sparse_mha_paged against dv_sparse_mha."""
    B, d, h, dh, page, L = 2, 1024, 8, 128, 16, 100
    s = wl.LayerShape(d=d, N=1024, r=32, h=h, dh=dh, L=L, cap=L + 4, B=B)
    t = wl.make_layer(s, 6, "cuda")
    t["K"][:, :, L], t["V"][:, :, L] = 0, 0
    W = -(-(L + 1) // page)
    table = i32([[b * W + c for c in range(W)] for b in range(B)])
    K = torch.zeros(B * W, h, page, dh, device="cuda", dtype=BF16)
    V = torch.zeros_like(K)
    for b in range(B):
        for p in range(L):
            K[b * W + p // page, :, p % page], V[b * W + p // page, :, p % page] = t["K"][b, :, p], t["V"][b, :, p]
    y = wl.make_input(s, 6, "cuda")
    idx, cnt = i32([1, 4, 6]), i32([3])
    a, b2 = torch.empty(B, d, device="cuda"), torch.empty(B, d, device="cuda")
    bd.dv_sparse_mha(y, t["Wqkv"], None, t["WOt"], None, t["K"], t["V"], L, dh ** -0.5, idx, cnt, 3, a,
                     bd.workspace(bd.DV_OP_SPARSE_MHA, bd.dims(B=B, d=d, h=h, dh=dh, cap=s.cap, kh_max=3)))
    slots = i32([int(table[b, L // page]) * page + L % page for b in range(B)])
    bd.dv_sparse_mha_paged(y, t["Wqkv"], None, t["WOt"], None, bd.PagedKV(K, V), table, i32([L + 1] * B), slots, dh ** -0.5, idx,
                           cnt, 3, b2, bd.workspace(bd.DV_OP_SPARSE_MHA_PAGED, bd.dims(B=B, d=d, h=h, dh=dh, kh_max=3)))
    torch.cuda.synchronize()
    # both are fp32 sums of the same bf16 values: 24 chained roundings of 2^-23 each side, in either order
    assert (a - b2).norm() <= 2 * 24 * 2.0 ** -23 * a.norm()
    for i in (1, 4, 6):
        for b in range(B):
            assert torch.equal(K[int(slots[b]) // page, i, L % page], t["K"][b, i, L])


def test_a_serving_loop_of_tables_append_and_blocks():
    """Requests join, grow, finish and reuse pages: dv_page_tables, a prompt's
    dv_paged_append, and decode steps of two layers' blocks in one captured
    graph, against per-request contiguous caches kept in 64 bits."""
    R, d, h, dh, page, n_pages, W, layers = 4, 256, 4, 64, 4, 24, 8, 2
    g = gen(31)
    ts = []
    for l in range(layers):
        t = wl.make_layer(wl.LayerShape(d=d, N=512, r=16, h=h, dh=dh, L=4, cap=5, B=1), 40 + l, "cuda")
        t["bqkv"], t["bO"] = torch.zeros(h, 3, dh, device="cuda"), torch.zeros(d, device="cuda")
        ts.append(t)
    pools = [(torch.full((n_pages, h, page, dh), float("nan"), device="cuda", dtype=BF16),
              torch.full((n_pages, h, page, dh), float("nan"), device="cuda", dtype=BF16)) for _ in range(layers)]
    kvs = [bd.PagedKV(*p) for p in pools]
    lens, table = i32([0] * R), i32([[-1] * W] * R)
    stack, count = i32(list(range(n_pages))), i32([n_pages])
    want, offsets, granted = i32([-1] * R), i32([0] * (R + 1)), i32([0] * R)
    ws_t = bd.workspace(bd.DV_OP_PAGE_TABLES, bd.dims())
    ws_m = bd.workspace(bd.DV_OP_SPARSE_MHA_PAGED, bd.dims(B=R, d=d, h=h, dh=dh, kh_max=h))
    heads, scale = [0, 2, 3], dh ** -0.5
    idx, cnt = i32(heads), i32([len(heads)])
    held = [[(np.zeros((0, h, dh)), np.zeros((0, h, dh))) for _ in range(R)] for _ in range(layers)]  # per layer and request
    x, slots = torch.zeros(R, d, device="cuda"), i32([-1] * R)
    outs = [torch.zeros(R, d, device="cuda") for _ in range(layers)]

    def step():
        bd.dv_page_tables(want, lens, lens, table, stack, count, count, slots, offsets, granted, page, ws_t)
        # a request's slot by its row (a row that does not grow has none)
        n = offsets[1:] - offsets[:-1]
        mine = torch.where(n > 0, slots[offsets[:-1].clamp(max=R - 1).long()], -1)
        for l in range(layers):
            bd.dv_sparse_mha_paged(x, ts[l]["Wqkv"], None, ts[l]["WOt"], None, kvs[l], table, lens, mine, scale, idx, cnt,
                                   len(heads), outs[l], ws_m)

    def prompt(r, n):
        w = i32([-1] * R)
        w[r] = n
        sl = i32([0] * n)
        bd.dv_page_tables(w, lens, lens, table, stack, count, count, sl, offsets, granted, page, ws_t)
        assert granted.tolist() == [1] * R
        for l in range(layers):
            k, v = torch.randn(n, h, dh, generator=g, device="cuda"), torch.randn(n, h, dh, generator=g, device="cuda")
            bd.dv_paged_append(kvs[l], k, v, sl, ws_t)
            held[l][r] = (f64(k.to(BF16)), f64(v.to(BF16)))

    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()  # (want is -1 everywhere: nothing changes)
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=side):
            step()
    torch.cuda.current_stream().wait_stream(side)
    prompt(0, 9)
    prompt(2, 4)
    alive = {0, 2}
    for it in range(14):
        if it == 4:
            prompt(1, 13)
            alive.add(1)
        if it == 7:  # request 0 ends and its pages go to the next one
            w = i32([-1] * R)
            w[0] = 0
            bd.dv_page_tables(w, lens, lens, table, stack, count, count, slots, offsets, granted, page, ws_t)
            alive.discard(0)
            for l in range(layers):
                held[l][0] = (np.zeros((0, h, dh)), np.zeros((0, h, dh)))
            prompt(3, 18)
            alive.add(3)
        now = lens.tolist()
        want.copy_(i32([now[r] + 1 if r in alive else -1 for r in range(R)]))
        x.copy_(torch.randn(R, d, generator=g, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        assert granted.tolist() == [1] * R
        for l in range(layers):
            Wq, Wo = f64(ts[l]["Wqkv"]), f64(ts[l]["WOt"])
            for r in range(R):
                if r not in alive:
                    assert not outs[l][r].any()
                    continue
                k, v = np.zeros((1, h, dh)), np.zeros((1, h, dh))
                for i in heads:
                    k[0, i], v[0, i] = Wq[i, 1] @ f64(x)[r], Wq[i, 2] @ f64(x)[r]
                rb = lambda z: f64(torch.from_numpy(z).float().to(BF16))  # noqa: E731
                held[l][r] = (np.concatenate([held[l][r][0], rb(k)]), np.concatenate([held[l][r][1], rb(v)]))
                n = held[l][r][0].shape[0]
                assert n == lens[r].item()
                q = np.stack([Wq[i, 0] @ f64(x)[r] for i in heads])[None]
                H, _, _ = attn_model(q, held[l][r][0].transpose(1, 0, 2)[None], held[l][r][1].transpose(1, 0, 2)[None], [[0]], [n], scale, heads)
                ref = sum(H[0, j] @ Wo[i] for j, i in enumerate(heads))
                assert np.linalg.norm(f64(outs[l])[r] - ref) <= 5e-3 * np.linalg.norm(ref)
    assert bd.dv_read_device_status(ws_t) == 0 and bd.dv_read_device_status(ws_m) == 0


def test_binding_refuses_wrong_tensors():
    K, V, table, lens = make_cache([20], 2, 64, 16, BF16, 1)
    kv, ws, q = bd.PagedKV(K, V), attn_ws(64), torch.zeros(1, 2, 64, device="cuda")
    out = torch.empty_like(q)
    for bad in (dict(q=q.to(BF16)), dict(q=q[:, :, :32]), dict(table=table.long()), dict(table=table.cpu()), dict(lens=lens[:0]),
                dict(out=out.cpu()), dict(out=torch.empty(1, 2, 128, device="cuda")[:, :, ::2]), dict(lse=torch.empty(1, 3, device="cuda")),
                dict(head_idx=i32([0])), dict(q=torch.zeros(1, 3, 64, device="cuda")), dict(ws=ws.cpu()), dict(ws=ws.float())):
        a = dict(q=q, table=table, lens=lens, out=out, ws=ws, lse=None, head_idx=None)
        a.update(bad)
        with pytest.raises(ValueError):
            bd.dv_paged_attn(a["q"], kv, a["table"], a["lens"], 0.1, a["out"], a["ws"], lse=a["lse"], head_idx=a["head_idx"])
    with pytest.raises(bd.DvError) as e:
        bd.dv_paged_attn(q, kv, table, lens, 0.1, out, ws[: 1 << 16])
    assert e.value.status == bd.DV_ERR_WORKSPACE
