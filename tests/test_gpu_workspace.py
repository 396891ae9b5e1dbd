"""One workspace, sized for the largest call and zeroed once, for calls of
other sizes in any order: what a serving loop does whose batch changes from
step to step. Every result equals that of a fresh workspace: bit for bit where
the call's sums have a fixed order. The contiguous calls at one and two rows
add partial sums by float atomics: at most 4096 terms in any order, each step
off by 2^-24 of a partial sum, and the terms' magnitudes add to at most
sqrt(4096) times the 2-norm of independent ones, so 2^-24 * 4096 * 64 = 2^-6
of the result's norm at the very most (stale sums are off by their own size)."""

import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from attention_predictor_gemv_b200 import binding as bd

BF16 = torch.bfloat16
D, H, DH, N = 2048, 16, 128, 4096


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.fixture(scope="module")
def weights():
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    return dict(Wqkv=(r(H, 3, DH, D) * D ** -0.5).to(BF16), WOt=(r(H, DH, D) * D ** -0.5).to(BF16), W1=(r(N, D) * D ** -0.5).to(BF16),
                W2=(r(N, D) * D ** -0.5).to(BF16), b1=r(N), At=(r(64, D) * D ** -0.5).to(BF16), Bm=r(N, 64).to(BF16), g=g)


def mha(w, B, kh):
    K, V = torch.randn(2, B, H, 40, DH, generator=w["g"], device="cuda").to(BF16)
    y = torch.randn(B, D, generator=w["g"], device="cuda")

    def call(ws):
        out = torch.zeros(B, D, device="cuda")
        bd.dv_sparse_mha(y, w["Wqkv"], None, w["WOt"], None, K, V, 33, DH ** -0.5, i32(list(range(kh)) + [0]), i32([kh]), kh, out, ws)
        return out

    return call, bd.dv_workspace_size(bd.DV_OP_SPARSE_MHA, bd.dims(B=B, d=D, h=H, dh=DH, cap=40, kh_max=kh))


def mlp(w, B, k):
    y = torch.randn(B, D, generator=w["g"], device="cuda")
    idx = torch.sort(torch.randperm(N, generator=w["g"], device="cuda")[: max(k, 1)])[0].to(torch.int32)

    def call(ws):
        out = torch.zeros(B, D, device="cuda")
        bd.dv_sparse_mlp(y, w["W1"], w["b1"], w["W2"], None, idx, i32([k]), k, out, ws)
        return out

    return call, bd.dv_workspace_size(bd.DV_OP_SPARSE_MLP, bd.dims(B=B, d=D, N=N, k_max=k))


def predict(w, B, k):
    y = torch.randn(B, D, generator=w["g"], device="cuda")

    def call(ws):
        scores, idx, count = torch.empty(B, N, device="cuda"), i32([0] * N), i32([0])
        bd.dv_predict_mlp(y, w["At"], w["Bm"], w["b1"], k, scores, idx, count, ws)
        return scores

    return call, bd.dv_workspace_size(bd.DV_OP_PREDICT_MLP, bd.dims(B=B, d=D, N=N, r=64, k_max=N))


def paged(w, B, kh, block=True):
    page, W = 8, 6
    K, V = torch.randn(2, B * W, H, page, DH, generator=w["g"], device="cuda").to(BF16)
    y, q = torch.randn(B, D, generator=w["g"], device="cuda"), torch.randn(B, H, DH, generator=w["g"], device="cuda")
    table, lens = i32([[b * W + c for c in range(W)] for b in range(B)]), i32([(7 * b) % 40 + 1 for b in range(B)])
    slots = i32([b * W * page + (7 * b) % 40 for b in range(B)])
    kv = bd.PagedKV(K, V)

    def call(ws):
        if not block:
            out = torch.zeros(B, H, DH, device="cuda")
            bd.dv_paged_attn(q, kv, table, lens, DH ** -0.5, out, ws)
            return out
        out = torch.zeros(B, D, device="cuda")
        bd.dv_sparse_mha_paged(y, w["Wqkv"], None, w["WOt"], None, kv, table, lens, slots, DH ** -0.5, i32(list(range(kh)) + [0]), i32([kh]), kh,
                               out, ws)
        return out

    op, d = (bd.DV_OP_SPARSE_MHA_PAGED, bd.dims(B=B, d=D, h=H, dh=DH, kh_max=kh)) if block else (bd.DV_OP_PAGED_ATTN, bd.dims(dh=DH))
    return call, bd.dv_workspace_size(op, d)


def attn(w, B, _):
    return paged(w, B, 0, block=False)


RUNS = {
    "mha": [(mha, 16, 12), (mha, 9, 12), (mha, 16, 12), (mha, 5, 3), (mha, 12, 0), (mha, 1, 16), (mha, 16, 5)],
    "mlp": [(mlp, 16, 4096), (mlp, 9, 1000), (mlp, 16, 4096), (mlp, 6, 130), (mlp, 2, 4096), (mlp, 16, 0), (mlp, 11, 700)],
    "paged": [(paged, 16, 12), (paged, 9, 12), (paged, 8, 12), (paged, 16, 12), (attn, 16, 0), (paged, 10, 4), (paged, 3, 16), (paged, 16, 0),
              (paged, 16, 16), (attn, 5, 0), (paged, 13, 16)],
    "mixed": [(predict, 16, 100), (paged, 16, 16), (mlp, 7, 4096), (mha, 16, 9), (predict, 4, 100), (paged, 8, 16), (mlp, 16, 2000), (attn, 9, 0),
              (mha, 6, 16), (predict, 16, 300), (paged, 12, 7), (mlp, 16, 4096)],
}


@pytest.mark.parametrize("run", RUNS)
def test_calls_of_other_sizes_share_a_workspace(weights, run):
    calls = [f(weights, B, n) for f, B, n in RUNS[run]]
    want = [call(torch.zeros(size, dtype=torch.uint8, device="cuda")) for call, size in calls]
    shared = torch.zeros(max(size for _, size in calls), dtype=torch.uint8, device="cuda")
    for _ in range(2):
        for (call, _), ref, what in zip(calls, want, RUNS[run]):
            out = call(shared)
            torch.cuda.synchronize()
            assert bd.dv_read_device_status(shared) == 0
            if what[0] in (mha, mlp) and what[1] <= 2:
                assert (out - ref).norm() <= 2.0 ** -6 * ref.norm(), what
            else:
                assert torch.equal(out, ref), what
