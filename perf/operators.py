"""Cases, plain forms and exact values of the paged key-value cache operators.

Four operators of one decode step over a paged cache, in the order a serving
loop calls them:

* ``tables``: block tables, slot maps and the free-page stack, built on the GPU
  from the requests' current and wanted lengths (``dv_page_tables``);
* ``append``: the keys and values of new tokens stored into their slots
  (``dv_paged_append``);
* ``attn``: attention of one new token per request over its pages, for every
  head or for a selected set of heads (``dv_paged_attn``);
* ``mha``: the head-sparse attention block over the paged cache: q, k, v of the
  selected heads, the append, the attention and W^O (``dv_sparse_mha_paged``).

``run`` computes them in plain torch (32-bit arithmetic) while ``own`` is
false and through the library while it is true.
"""

import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------


def listed():
    return [
        # a decode step of 16 running requests: each grows by one token (latency of the smallest call)
        dict(name="tables_decode_16", kind="tables", decode=16, prefill=0, release=0, idle=0, prompt=0, L=2176, page=16, spare=1.5),
        # a large serving batch in one step: running requests, new prompts, finished and idle rows; the
        # free pages do not cover the last prompts, which are refused
        dict(name="tables_mixed_1024", kind="tables", decode=700, prefill=120, release=150, idle=54, prompt=1024, L=4096, page=16, spare=0.95),
        # one decode token per request into an fp32 cache (the smallest append)
        dict(name="append_decode_f32", kind="append", T=16, h=32, dh=64, page=16, dtype="f32", holes=2),
        # the prompt tokens of one prefill step into a bf16 cache (OPT-6.7B heads)
        dict(name="append_prefill_bf16", kind="append", T=16384, h=32, dh=128, page=16, dtype="bf16", holes=37),
        # few requests of OPT-1.3B heads at its cache length, fp32 cache
        dict(name="attn_small_f32", kind="attn", B=4, hq=32, hkv=32, dh=64, L=520, page=16, dtype="f32", ragged=True, sel=0),
        # one request with a short context (latency of the smallest call)
        dict(name="attn_one_short", kind="attn", B=1, hq=32, hkv=32, dh=128, L=65, page=16, dtype="bf16", ragged=False, sel=0),
        # a batch of OPT-6.7B heads, lengths from none to the whole cache
        dict(name="attn_mha_b16", kind="attn", B=16, hq=32, hkv=32, dh=128, L=2176, page=16, dtype="bf16", ragged=True, sel=0),
        # grouped queries, a large ragged batch, pages of 64
        dict(name="attn_gqa_b64", kind="attn", B=64, hq=64, hkv=8, dh=128, L=8192, page=64, dtype="bf16", ragged=True, sel=0),
        # one request with a very long context: work only in the cache's length
        dict(name="attn_long_b1", kind="attn", B=1, hq=32, hkv=8, dh=128, L=131071, page=32, dtype="bf16", ragged=False, sel=0),
        # 14 selected heads of 96 (OPT-175B heads), one full-length batch
        dict(name="attn_selected_b8", kind="attn", B=8, hq=96, hkv=96, dh=128, L=2048, page=16, dtype="bf16", ragged=False, sel=14),
        # the attention block of one OPT-175B layer step, 14 of 96 heads
        dict(name="mha_opt175b_b1", kind="mha", B=1, d=12288, h=96, dh=128, L=2049, page=16, dtype="bf16", ragged=False, sel=14),
        # the attention block of an OPT-6.7B layer step, four requests of different lengths, 6 heads each
        dict(name="mha_opt6.7b_b4", kind="mha", B=4, d=4096, h=32, dh=128, L=2049, page=16, dtype="bf16", ragged=True, sel=20),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["tables", "append", "attn", "attn", "attn", "mha"])
    page = rng.choice([1, 5, 8, 16, 16, 24, 32, 48, 64, 100, 128])
    if kind == "tables":
        rows = _log_int(rng, 1, 2048)
        prefill = rng.randint(0, max(1, rows // 6))
        release = rng.randint(0, rows // 6)
        idle = rng.randint(0, rows // 8)
        prompt = _log_int(rng, 1, max(1, min(4096, 120000 // max(1, prefill))))
        return dict(kind="tables", decode=max(0, rows - prefill - release - idle), prefill=prefill, release=release, idle=idle,
                    prompt=prompt, L=_log_int(rng, 64, 4096), page=max(page, 8), spare=rng.choice([0.5, 0.9, 1.0, 1.5]))
    if kind == "append":
        h, dh = rng.choice([1, 4, 8, 12, 32]), rng.choice([64, 80, 96, 128, 256])
        T = _log_int(rng, 1, max(1, min(16384, 60_000_000 // (h * dh))))
        return dict(kind="append", T=T, h=h, dh=dh, page=page, dtype=rng.choice(["bf16", "f32"]), holes=rng.randint(0, T // 8))
    if kind == "attn":
        hkv = rng.choice([1, 2, 4, 8, 8, 32, 32, 96])
        G = rng.choice([1, 1, 1, 2, 4, 5, 8, 16]) if hkv <= 8 else 1
        dh = rng.choice([64, 64, 80, 96, 128, 128, 128, 256])
        dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
        B = _log_int(rng, 1, 128)
        keys = 260_000_000 // (hkv * dh * max(G // 8, 2 if dtype == "f32" else 1))  # keys in all, of every request
        L = max(1, min(_log_int(rng, 1, 131072), keys // B))
        sel = rng.choice([0, 0, max(1, hkv // 6)])
        return dict(kind="attn", B=B, hq=hkv * G, hkv=hkv, dh=dh, L=L, page=page, dtype=dtype, ragged=rng.random() < 0.6, sel=sel)
    d, h, dh = rng.choice([(2048, 32, 64), (4096, 32, 128)])
    return dict(kind="mha", B=rng.randint(1, 4), d=d, h=h, dh=dh, L=_log_int(rng, 2, 2176), page=page, dtype="bf16",
                ragged=rng.random() < 0.5, sel=rng.randint(1, h))


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------


def _lengths(case):
    """The requests' lengths in a fixed order (a permutation of them is drawn): from 0 to L where ragged."""
    B, L = case["B"], case["L"]
    return [(i * L) // (B - 1) for i in range(B)] if case["ragged"] and B > 1 else [L] * B


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _perm(n, g):
    return torch.randperm(n, generator=g, device="cuda")


def _set_of(n, k, g):
    """k of n heads, ascending."""
    return torch.sort(_perm(n, g)[:k])[0].to(torch.int32)


def _cache(case, hkv, dh, g):
    """Lengths, block tables over randomly placed pages, and the pools."""
    page, B = case["page"], case["B"]
    lens = torch.tensor(_lengths(case), device="cuda", dtype=torch.int64)[_perm(B, g)]
    n = (lens + page - 1) // page
    W = -(-case["L"] // page)
    n_pages = int(n.sum()) + 3
    at = torch.cumsum(n, 0) - n
    cols = torch.arange(W, device="cuda")
    order = _perm(n_pages, g)
    table = torch.where(cols[None, :] < n[:, None], order[(at[:, None] + cols[None, :]).clamp(max=n_pages - 1)], -1)
    K = torch.randn(n_pages, hkv, page, dh, generator=g, device="cuda").to(DT[case["dtype"]])
    V = torch.randn(n_pages, hkv, page, dh, generator=g, device="cuda").to(DT[case["dtype"]])
    return dict(lens=lens.to(torch.int32), table=table.to(torch.int32).contiguous(), K=K, V=V)


def _prepare_tables(case, g):
    page, L = case["page"], case["L"]
    R = case["decode"] + case["prefill"] + case["release"] + case["idle"]
    W = -(-(L + case["prompt"] + 1) // page)
    kind = torch.tensor([0] * case["decode"] + [1] * case["prefill"] + [2] * case["release"] + [3] * case["idle"], device="cuda")
    lens = 1 + (torch.arange(R, device="cuda") * 7919) % L  # spread over 1 to L
    lens = torch.where(kind == 1, 0, lens)  # a new prompt starts from nothing
    mix = _perm(R, g)
    kind, lens = kind[mix], lens[mix]
    want = torch.where(kind == 0, lens + 1, torch.where(kind == 1, case["prompt"], torch.where(kind == 2, 0, -1)))
    n = (lens + page - 1) // page
    goal = torch.where(want < 0, lens, want)
    need = ((goal + page - 1) // page - n).clamp(min=0).sum()
    gone = (n - (goal + page - 1) // page).clamp(min=0).sum()
    held = int(n.sum())
    free = max(0, int(int(need) * case["spare"]) - int(gone))
    n_pages = held + free + 1
    order = _perm(n_pages, g).to(torch.int32)
    at = torch.cumsum(n, 0) - n
    cols = torch.arange(W, device="cuda")
    table = torch.where(cols[None, :] < n[:, None], order[(at[:, None] + cols[None, :]).clamp(max=n_pages - 1)], -1).to(torch.int32)
    free_list = torch.full((n_pages,), -1, device="cuda", dtype=torch.int32)
    free_list[:free] = order[held:held + free]
    tokens = case["decode"] + case["prefill"] * case["prompt"]
    i32 = dict(device="cuda", dtype=torch.int32)
    return dict(want=want.to(torch.int32), lens=lens.to(torch.int32), lens_out=torch.zeros(R, **i32), table=table.contiguous(),
                free_list=free_list, free_count=torch.tensor([free], **i32), free_count_out=torch.zeros(1, **i32),
                slots=torch.zeros(max(1, tokens), **i32), offsets=torch.zeros(R + 1, **i32), granted=torch.zeros(R, **i32))


def prepare(case, seed):
    g = _gen(seed)
    kind = case["kind"]
    if kind == "tables":
        s = _prepare_tables(case, g)
    elif kind == "append":
        T, h, dh, page = case["T"], case["h"], case["dh"], case["page"]
        n_pages = -(-T // page) + 5
        slots = _perm(n_pages * page, g)[:T].to(torch.int32)
        slots[_perm(T, g)[:case["holes"]]] = -1  # padding tokens
        s = dict(k=torch.randn(T, h, dh, generator=g, device="cuda"), v=torch.randn(T, h, dh, generator=g, device="cuda"), slots=slots,
                 K=torch.randn(n_pages, h, page, dh, generator=g, device="cuda").to(DT[case["dtype"]]),
                 V=torch.randn(n_pages, h, page, dh, generator=g, device="cuda").to(DT[case["dtype"]]))
    elif kind == "attn":
        hkv, dh, G = case["hkv"], case["dh"], case["hq"] // case["hkv"]
        s = _cache(case, hkv, dh, g)
        rows = case["sel"] or hkv
        s["q"] = torch.randn(case["B"], rows * G, dh, generator=g, device="cuda")
        s["out"], s["lse"] = torch.empty_like(s["q"]), torch.empty(case["B"], rows * G, device="cuda")
        s["scale"] = dh ** -0.5
        if case["sel"]:
            s["head_idx"] = _set_of(hkv, case["sel"], g)
            s["head_count"] = torch.tensor([case["sel"]], device="cuda", dtype=torch.int32)
    else:
        d, h, dh, B = case["d"], case["h"], case["dh"], case["B"]
        s = _cache(case, h, dh, g)
        lens = s["lens"].long()
        last = (lens - 1).clamp(min=0)
        slot = s["table"].long().gather(1, (last // case["page"])[:, None])[:, 0] * case["page"] + last % case["page"]
        s["slots"] = torch.where(lens > 0, slot, -1).to(torch.int32)  # where the new token of each request goes
        s["y"] = torch.randn(B, d, generator=g, device="cuda")
        s["Wqkv"] = torch.randn(h, 3, dh, d, generator=g, device="cuda").mul_(d ** -0.5).to(DT[case["dtype"]])
        s["WOt"] = torch.randn(h, dh, d, generator=g, device="cuda").mul_(d ** -0.5).to(DT[case["dtype"]])
        s["bqkv"] = torch.randn(h, 3, dh, generator=g, device="cuda").mul_(0.1)
        s["bO"] = torch.randn(d, generator=g, device="cuda").mul_(0.1)
        s["head_idx"] = _set_of(h, case["sel"], g)
        s["head_count"] = torch.tensor([case["sel"]], device="cuda", dtype=torch.int32)
        s["out"], s["scale"] = torch.empty(B, d, device="cuda"), dh ** -0.5
    s["case"] = dict(case)
    if own:
        from attention_predictor_gemv_b200 import binding as bd

        if kind != "tables":
            s["kv"] = bd.PagedKV(s["K"], s["V"])
        s["ws"] = {
            "tables": lambda: bd.workspace(bd.DV_OP_PAGE_TABLES, bd.dims()),
            "append": lambda: bd.workspace(bd.DV_OP_PAGED_APPEND, bd.dims()),
            "attn": lambda: bd.workspace(bd.DV_OP_PAGED_ATTN, bd.dims(h=case.get("hq", 0), dh=case.get("dh", 0))),
            "mha": lambda: bd.workspace(bd.DV_OP_SPARSE_MHA_PAGED, bd.dims(B=case.get("B"), d=case.get("d"), h=case.get("h"), dh=case.get("dh"), kh_max=case.get("sel"))),
        }[kind]()
    return s


# ---------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------


def _plain_tables(s):
    """Lengths to block tables: pages that shrunk rows hold no more are pushed on the free stack (rows, then pages, in
    order); rows that grow take pages from its top, in row order, as long as the running need is covered."""
    page = s["case"]["page"]
    table, free_list, W, T = s["table"], s["free_list"], s["table"].shape[1], s["slots"].shape[0]
    lens, want, count = s["lens"].long(), s["want"].long(), s["free_count"].long()
    goal = torch.where(want < 0, lens, want)
    fits = goal <= W * page
    goal = torch.where(fits, goal, lens)
    old_p, new_p = (lens + page - 1) // page, (goal + page - 1) // page
    gone, need, add = (old_p - new_p).clamp(min=0), (new_p - old_p).clamp(min=0), (goal - lens).clamp(min=0)
    avail = count + gone.sum()
    ok = fits & ((need == 0) | (torch.cumsum(need, 0) <= avail)) & ((add == 0) | (torch.cumsum(add, 0) <= T))
    need, add = torch.where(ok, need, 0), torch.where(ok, add, 0)
    goal = torch.where(ok, goal, lens)
    cols = torch.arange(W, device=table.device)[None, :]
    freed = table[(cols >= new_p[:, None]) & (cols < old_p[:, None])]
    free_list[count + torch.arange(freed.shape[0], device=table.device)] = freed
    grow = (cols >= old_p[:, None]) & (cols < (old_p + need)[:, None])
    taken = need.sum()
    table[grow] = free_list[avail - 1 - torch.arange(int(taken), device=table.device)]
    offsets = torch.cat([torch.zeros_like(add[:1]), torch.cumsum(add, 0)])
    row = torch.repeat_interleave(torch.arange(add.shape[0], device=table.device), add)
    pos = lens[row] + torch.arange(row.shape[0], device=table.device) - offsets[row]
    s["slots"].fill_(-1)
    s["slots"][: row.shape[0]] = (table[row, pos // page].long() * page + pos % page).to(torch.int32)
    s["lens_out"].copy_(goal)
    s["offsets"].copy_(offsets)
    s["granted"].copy_(ok)
    s["free_count_out"].copy_(avail - taken)


def _plain_store(K, V, k, v, slots, page):
    at = slots.long()
    at, src = at[at >= 0], at >= 0
    K[at // page, :, at % page] = k[src].to(K.dtype)
    V[at // page, :, at % page] = v[src].to(V.dtype)


def _plain_attn(q, K, V, table, lens, scale, heads, page):
    """Softmax attention of q [B][heads][G][dh] over each row's pages, in 32 bits; 0 and -inf for an empty row."""
    B, L = table.shape[0], table.shape[1] * page
    pos = torch.arange(L, device=q.device)
    pages = table.long()[:, pos // page].clamp(min=0)
    rows = (pages * K.shape[1])[:, None, :] + heads[None, :, None]
    rows = rows * page + (pos % page)[None, None, :]  # [B][heads][L] rows of the pools
    keys, values = K.reshape(-1, K.shape[3])[rows].float(), V.reshape(-1, V.shape[3])[rows].float()
    inside = (pos[None, :] < lens[:, None])[:, None, :, None]
    score = torch.matmul(keys, q.transpose(2, 3)) * scale  # [B][heads][L][G]
    score = torch.where(inside, score, -math.inf)
    top = score.amax(2, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = torch.exp(score - top)
    total = p.sum(2, keepdim=True)
    out = torch.matmul(p.transpose(2, 3), torch.where(inside, values, 0.0))  # [B][heads][G][dh]
    out = torch.where(total.transpose(2, 3) > 0, out / total.transpose(2, 3), 0.0)
    lse = (top + torch.log(total))[:, :, 0]
    return out, lse


def _plain_mha(s):
    y, h, dh, page = s["y"], s["case"]["h"], s["case"]["dh"], s["case"]["page"]
    heads = s["head_idx"].long()
    qkv = torch.matmul(s["Wqkv"][heads].float().reshape(-1, y.shape[1]), y.t()).t().reshape(y.shape[0], -1, 3, dh) + s["bqkv"][heads]
    k, v = torch.zeros(y.shape[0], h, dh, device=y.device), torch.zeros(y.shape[0], h, dh, device=y.device)
    k[:, heads], v[:, heads] = qkv[:, :, 1], qkv[:, :, 2]  # an unselected head's slot holds zeros
    _plain_store(s["K"], s["V"], k, v, s["slots"], page)
    H, _ = _plain_attn(qkv[:, :, :1], s["K"], s["V"], s["table"], s["lens"], s["scale"], heads, page)
    s["out"].copy_(torch.matmul(H.reshape(y.shape[0], -1), s["WOt"][heads].float().reshape(-1, y.shape[1])) + s["bO"])


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------


def _tables_out(s):
    return {n: s[n] for n in ("lens_out", "table", "free_list", "free_count_out", "slots", "offsets", "granted")}


def run(s):
    kind = s["case"]["kind"]
    if own:
        from attention_predictor_gemv_b200 import binding as bd

        if kind == "tables":
            bd.dv_page_tables(s["want"], s["lens"], s["lens_out"], s["table"], s["free_list"], s["free_count"], s["free_count_out"],
                              s["slots"], s["offsets"], s["granted"], s["case"]["page"], s["ws"])
        elif kind == "append":
            bd.dv_paged_append(s["kv"], s["k"], s["v"], s["slots"], s["ws"])
        elif kind == "attn":
            bd.dv_paged_attn(s["q"], s["kv"], s["table"], s["lens"], s["scale"], s["out"], s["ws"], lse=s["lse"],
                             head_idx=s.get("head_idx"), head_count=s.get("head_count"))
        else:
            bd.dv_sparse_mha_paged(s["y"], s["Wqkv"], s["bqkv"], s["WOt"], s["bO"], s["kv"], s["table"], s["lens"], s["slots"], s["scale"],
                                   s["head_idx"], s["head_count"], s["case"]["sel"], s["out"], s["ws"])
    elif kind == "tables":
        _plain_tables(s)
    elif kind == "append":
        _plain_store(s["K"], s["V"], s["k"], s["v"], s["slots"], s["case"]["page"])
    elif kind == "attn":
        c = s["case"]
        heads = s["head_idx"].long() if c["sel"] else torch.arange(c["hkv"], device="cuda")
        out, lse = _plain_attn(s["q"].reshape(c["B"], heads.shape[0], -1, c["dh"]), s["K"], s["V"], s["table"], s["lens"], s["scale"], heads, c["page"])
        s["out"].copy_(out.reshape(s["out"].shape))
        s["lse"].copy_(lse.reshape(s["lse"].shape))
    else:
        _plain_mha(s)
    if kind == "tables":
        return _tables_out(s)
    if kind == "append":
        return {"K": s["K"], "V": s["V"]}
    if kind == "attn":
        return {"out": s["out"], "lse": s["lse"]}
    return {"out": s["out"], "K": s["K"], "V": s["V"]}


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------


def work(case):
    kind = case["kind"]
    size = 4 if case.get("dtype") == "f32" else 2
    if kind == "tables":
        page, R = case["page"], case["decode"] + case["prefill"] + case["release"] + case["idle"]
        tokens = case["decode"] + case["prefill"] * case["prompt"]
        taken = case["decode"] / page + case["prefill"] * -(-case["prompt"] // page)
        freed = case["release"] * (case["L"] / 2 + page) / page
        # want, lens in; lens, offsets, granted out; slots out; each page moved read and written once
        return {"bytes": 20 * R + 4 * tokens + 8 * (taken + freed) + 4 * case["decode"], "flops": 0}
    if kind == "append":
        T = case["T"] - case["holes"]
        return {"bytes": 4 * case["T"] + 2 * T * case["h"] * case["dh"] * (4 + size), "flops": 0}
    keys = sum(_lengths(case))
    pages = sum(-(-n // case["page"]) for n in _lengths(case))
    if kind == "attn":
        rows = case["sel"] or case["hkv"]
        G = case["hq"] // case["hkv"]
        return {"bytes": 2 * keys * rows * case["dh"] * size + 4 * pages + case["B"] * rows * G * (8 * case["dh"] + 4),
                "flops": 4 * keys * rows * G * case["dh"]}
    B, d, dh, sel = case["B"], case["d"], case["dh"], case["sel"]
    store = 2 * sum(n > 0 for n in _lengths(case)) * case["h"] * dh * size
    weights = 4 * sel * dh * d * size
    return {"bytes": weights + 2 * keys * sel * dh * size + store + 4 * pages + 8 * B * d + 4 * d + 12 * sel * dh,
            "flops": 8 * B * sel * dh * d + 4 * keys * sel * dh}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------


def _exact_rows(q, K, V, table, lens, scale, heads, page):
    """Row by row: gather the row's keys and values in order, softmax in 64 bits."""
    G = q.shape[1] // len(heads)
    out = torch.zeros(q.shape, device="cuda", dtype=torch.float64)
    lse = torch.full(q.shape[:2], -math.inf, device="cuda", dtype=torch.float64)
    for b, n in enumerate(lens.tolist()):
        if n == 0:
            continue
        pages = table[b, : -(-n // page)].long()
        for j, i in enumerate(heads):
            k = K[pages, i].reshape(-1, K.shape[3])[:n].double()
            v = V[pages, i].reshape(-1, V.shape[3])[:n].double()
            z = (q[b, j * G:(j + 1) * G] @ k.t()) * scale
            lse[b, j * G:(j + 1) * G] = torch.logsumexp(z, 1)
            out[b, j * G:(j + 1) * G] = torch.softmax(z, 1) @ v
    return out, lse


def exact(case, seed):
    kind = case["kind"]
    if kind == "tables":
        return None  # whole numbers
    s = prepare(case, seed)
    page = case["page"]
    if kind == "append":
        slots = s["slots"].long().cpu()
        K, V = s["K"].double(), s["V"].double()
        use = (slots >= 0).nonzero()[:, 0].cuda()
        at = s["slots"].long()[use]
        for pool, new in ((K, s["k"]), (V, s["v"])):
            flat = pool.transpose(1, 2).reshape(-1, case["h"], case["dh"]).clone()
            flat[at] = new[use].double()
            pool.copy_(flat.reshape(pool.shape[0], page, case["h"], case["dh"]).transpose(1, 2))
        return {"K": K, "V": V}
    if kind == "attn":
        heads = s["head_idx"].tolist() if case["sel"] else list(range(case["hkv"]))
        if case["B"] * len(heads) > 20000:
            return None
        out, lse = _exact_rows(s["q"].double(), s["K"], s["V"], s["table"], s["lens"], s["scale"], heads, page)
        return {"out": out, "lse": lse}
    heads = s["head_idx"].tolist()
    y, h, dh = s["y"].double(), case["h"], case["dh"]
    K, V = s["K"].double(), s["V"].double()
    kept = s["K"].dtype
    q = torch.zeros(case["B"], len(heads), dh, device="cuda", dtype=torch.float64)
    live = [b for b, n in enumerate(s["lens"].tolist()) if n > 0]
    for b in live:
        p, o = divmod(int(s["slots"][b]), page)
        K[p, :, o], V[p, :, o] = 0.0, 0.0
    newK, newV = K.clone(), V.clone()  # unrounded, as the definition has them; the attention reads what the cache holds
    for j, i in enumerate(heads):
        w, bias = s["Wqkv"][i].double(), s["bqkv"][i].double()
        q[:, j] = y @ w[0].t() + bias[0]
        k, v = y @ w[1].t() + bias[1], y @ w[2].t() + bias[2]
        for b in live:
            p, o = divmod(int(s["slots"][b]), page)
            newK[p, i, o], newV[p, i, o] = k[b], v[b]
            K[p, i, o], V[p, i, o] = k[b].to(kept).double(), v[b].to(kept).double()
    H, _ = _exact_rows(q, K, V, s["table"], s["lens"], s["scale"], heads, page)
    W = torch.stack([s["WOt"][i].double() for i in heads])
    return {"out": torch.einsum("bjc,jcd->bd", H, W) + s["bO"].double(), "K": newK, "V": newV}
