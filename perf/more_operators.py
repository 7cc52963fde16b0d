"""The operators of a step that verifies drafted tokens, as cases to measure.

``norm_rope``: norms of the query and key heads and their rotary positions in one pass;
``masks``: what each node of a drafted tree sees, and its position, from the nodes' parents;
``tree``: attention of the nodes of such trees over the 4-bit cache;
``compact``: the accepted nodes' tokens moved together in their pages (4-bit and E4M3 cache);
``pages``: requests forked (whole pages shared, the last one copied) and given up again.

With ``own`` false every operator runs in plain torch operations in 32 bits (angles in 64).
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
K_GLOBAL, V_GLOBAL = 0.75, 1.25  # global scales of the 4-bit cache


# ---- the cases ---------------------------------------------------------------
def _norm_rope(tokens, hq, hkv, dim, rotary, interleaved, pos_hi, dtype="bf16", offset=0.0,
               weight="bf16", base=10000.0, factor=1.0, orig=0, attn=1.0):
    return {"op": "norm_rope", "tokens": tokens, "hq": hq, "hkv": hkv, "dim": dim,
            "rotary": rotary, "interleaved": interleaved, "pos_hi": pos_hi, "dtype": dtype,
            "offset": offset, "weight": weight, "base": base, "factor": factor, "orig": orig,
            "attn": attn}


def _masks(batch, nodes_lo, nodes_hi, kv_hi):
    return {"op": "masks", "batch": batch, "new_lo": nodes_lo, "new_hi": nodes_hi,
            "kv_lo": nodes_hi, "kv_hi": max(kv_hi, nodes_hi)}


def _tree(batch, kv, nodes, hq, hkv, dk, dv, page=16, layout="HND", out="bf16"):
    return {"op": "tree", "batch": batch, "kv_lo": kv[0], "kv_hi": kv[1], "new_lo": nodes[0],
            "new_hi": nodes[1], "hq": hq, "hkv": hkv, "dk": dk, "dv": dv, "page": page,
            "layout": layout, "out": out}


def _compact(cache, batch, kv, nodes, kept, hkv, dk, dv, page=16, layout="HND"):
    return {"op": "compact", "cache": cache, "batch": batch, "kv_lo": kv[0], "kv_hi": kv[1],
            "new_lo": nodes[0], "new_hi": nodes[1], "kept": kept, "hkv": hkv, "dk": dk, "dv": dv,
            "page": page, "layout": layout}


def _forks(batch, kv, copies, hkv, dk, dv, page=16, layout="HND"):
    return {"op": "pages", "batch": batch, "kv_lo": kv[0], "kv_hi": kv[1], "copies": copies,
            "hkv": hkv, "dk": dk, "dv": dv, "page": page, "layout": layout}


def listed():
    return [
        # the drafted nodes of a few requests: a quarter of wide heads turns in pairs, weights
        # around 0 that 1 is added to, f16
        dict(_norm_rope(211, 16, 2, 256, 64, True, 32768, "f16", 1.0, "f32"),
             name="norm_rope_drafts_pairs"),
        # a long prompt: 32 query and 8 kv heads of 128
        dict(_norm_rope(16384, 32, 8, 128, 128, False, 131072, "bf16", 0.0, "bf16", 500000.0),
             name="norm_rope_long_prompt"),
        # small trees of a running batch: latency counts
        dict(_masks(16, 5, 16, 4096), name="masks_small_trees"),
        # a full server, large trees of odd sizes
        dict(_masks(1000, 31, 130, 32771), name="masks_full_server"),
        # two short requests: the smallest attention call
        dict(_tree(2, (37, 100), (5, 7), 4, 1, 128, 128), name="tree_tiny"),
        # a batch of ordinary lengths, 16 nodes each
        dict(_tree(16, (512, 4096), (16, 16), 32, 8, 128, 128), name="tree_batched"),
        # few requests, long histories, larger trees: work split over the tokens
        dict(_tree(4, (32771, 32771), (26, 26), 32, 8, 128, 128), name="tree_long"),
        # query and key heads of 512, values of 256, slots before heads in memory, f16 out
        dict(_tree(8, (2048, 8192), (6, 11), 16, 2, 512, 256, 16, "NHD", "f16"),
             name="tree_wide_heads"),
        # a few accepted nodes of each request of a running batch, 4-bit cache
        dict(_compact("nvfp4", 16, (512, 4096), (16, 16), 6, 8, 128, 128),
             name="compact_batched"),
        # long accepted paths over several pages, E4M3 cache: scales of pages meet
        dict(_compact("e4m3", 256, (40, 1000), (40, 64), 38, 8, 128, 128),
             name="compact_long_paths_e4m3"),
        # every request of a batch tries one more continuation
        dict(_forks(16, (512, 4096), 1, 8, 128, 128), name="pages_fork_batched"),
        # many continuations of long requests
        dict(_forks(64, (500, 16384), 8, 8, 128, 128), name="pages_fork_many"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm_rope", "norm_rope", "masks", "tree", "tree", "tree", "compact",
                     "pages"])
    page = rng.choice([16, 16, 16, 1])
    if op == "norm_rope":
        dim = rng.choice([64, 128, 128, 256, 512])
        rotary = rng.choice([dim, dim, dim // 2, 2 * rng.randint(1, dim // 2)])
        hkv = rng.choice([1, 2, 8])
        scaled = rng.random() < 0.5
        dtype = rng.choice(["bf16", "f16"])
        return _norm_rope(_log_int(rng, 1, 4096), hkv * rng.choice([1, 4, 5]), hkv, dim, rotary,
                          rng.random() < 0.5, _log_int(rng, 64, 1 << 20), dtype,
                          rng.choice([0.0, 1.0]), rng.choice([dtype, "f32"]),
                          rng.choice([10000.0, 500000.0]),
                          rng.uniform(1.5, 40.0) if scaled else 1.0,
                          rng.choice([0, 4096, 8192]) if scaled else 0, rng.choice([1.0, 1.25]))
    if op == "masks":
        hi = _log_int(rng, 1, 256)
        return _masks(_log_int(rng, 1, 500), rng.randint(1, hi), hi, _log_int(rng, 1, 131071))
    hkv = rng.choice([1, 2, 8])
    dk, dv = rng.choice([(64, 64), (128, 128), (128, 128), (256, 256), (256, 128), (512, 256)])
    layout = rng.choice(["HND", "NHD"])
    if op == "pages":
        batch = _log_int(rng, 1, 64)
        hi = _log_int(rng, 1, min(16384 if page == 16 else 2048, 300000 // batch))
        return _forks(batch, (rng.randint(1, hi), hi), rng.randint(1, 8), hkv, dk, dv, page,
                      layout)
    if op == "compact":
        batch, hi = _log_int(rng, 1, 256), _log_int(rng, 1, 64)
        kv = _log_int(rng, hi, max(hi, min(4000, 200000 // batch)))
        return _compact(rng.choice(["nvfp4", "e4m3"]), batch, (hi, kv), (rng.randint(1, hi), hi),
                        rng.randint(1, hi), hkv, dk, dv, page, layout)
    batch = _log_int(rng, 1, 16)
    nodes = rng.choice([rng.randint(1, 8), rng.randint(2, 32), _log_int(rng, 8, 100)])
    hi = _log_int(rng, max(nodes, 16), max(nodes, min(32771, 100000000 // (batch * hkv * (dk + dv)))))
    return _tree(batch, (rng.randint(nodes, hi), hi), (rng.choice([1, nodes]), nodes),
                 hkv * rng.choice([1, 4, 5, 8]), hkv, dk, dv, page, layout,
                 rng.choice(["bf16", "bf16", "f16"]))


def _ragged(n, lo, hi):
    """n lengths over [lo, hi], the same for every seed: both ends and what lies between."""
    if n == 1:
        return [hi]
    f = [(0.6180339887498949 * i) % 1.0 for i in range(n)]
    f[0], f[-1] = 0.0, 1.0
    return [lo + int((hi - lo) * x + 0.5) for x in f]


def _lengths(case):
    """(tokens held, drafted nodes among them) of every request."""
    kv = _ragged(case["batch"], case["kv_lo"], case["kv_hi"])
    new = _ragged(case["batch"], case["new_lo"], case["new_hi"])[::-1]
    return kv, [min(n, a) for n, a in zip(new, kv)]


def _kept(case, new):
    """Accepted nodes of every request: from none to the case's most."""
    return [min(k, n) for k, n in zip(_ragged(len(new), 0, case["kept"]), new)]


def _pages(n, page):
    return -(-n // page)


def _row_bytes(dim, cache="nvfp4"):
    return dim if cache == "e4m3" else dim // 2 + dim // 16


def work(case):
    op = case["op"]
    if op == "norm_rope":
        n = case["tokens"] * (case["hq"] + case["hkv"]) * case["dim"]
        return {"bytes": 4 * n + 4 * case["tokens"], "flops": 4 * n}
    page = case.get("page", 16)
    if op == "pages":
        kv = _ragged(case["batch"], case["kv_lo"], case["kv_hi"])
        row = case["hkv"] * (_row_bytes(case["dk"]) + _row_bytes(case["dv"]))
        forks = case["copies"] * case["batch"]
        entries = case["copies"] * sum(_pages(n, page) for n in kv)
        copied = case["copies"] * sum(1 for n in kv if n % page)
        # a parent's entry read, the child's written and read, the page's owners counted up
        # and down; the copied pages read and written
        return {"bytes": 28 * entries + 2 * copied * row * page + 24 * forks, "flops": entries}
    kv, new = _lengths(case)
    if op == "masks":
        words = _pages(max(new), 32)
        return {"bytes": sum(new) * (8 + 4 * words) + 8 * len(new), "flops": sum(new) * words}
    if op == "compact":
        row = case["hkv"] * (_row_bytes(case["dk"], case["cache"])
                             + _row_bytes(case["dv"], case["cache"]))
        kept = sum(_kept(case, new))
        return {"bytes": 2 * row * kept + 8 * kept + 16 * len(kv), "flops": kept}
    rows = sum(new)
    pages = sum(_pages(a, page) for a in kv)
    row = case["hkv"] * (_row_bytes(case["dk"]) + _row_bytes(case["dv"]))
    seen = sum((a - n + 1) * n for a, n in zip(kv, new))
    return {"bytes": row * sum(kv) + 4 * pages + rows * (case["hq"] * (2 * case["dk"]
                                                         + 2 * case["dv"] + 4)
                                                         + 4 * _pages(max(new), 32)),
            "flops": 2 * (case["dk"] + case["dv"]) * case["hq"] * seen}


# ---- what a program has in hand ------------------------------------------------
def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _indptr(counts):
    return _i32([0] + list(np.cumsum(counts)))


def _buffer(fill, pages, heads, page, row, layout):
    """[pages, heads, slots, bytes] in memory in the given layout; fill makes it of a shape."""
    if layout == "HND":
        return fill((pages, heads, page, row))
    return fill((pages, page, heads, row)).transpose(1, 2)


def _nvfp4_pool(case, gen, pages):
    """Codes of every kind; block scales (E4M3) around a quarter, so that values are near 1."""
    def codes(shape):
        return torch.randint(0, 256, shape, generator=gen, device=DEV, dtype=torch.uint8)

    def scales(shape):
        return torch.randint(0x24, 0x34, shape, generator=gen, device=DEV, dtype=torch.uint8)
    out = {}
    for n, dim in (("k", case["dk"]), ("v", case["dv"])):
        out[n + "_data"] = _buffer(codes, pages, case["hkv"], case["page"], dim // 2,
                                   case["layout"])
        out[n + "_sf"] = _buffer(scales, pages, case["hkv"], case["page"], dim // 16,
                                 case["layout"])
    return out


def _e4m3_pool(case, gen, pages):
    """Codes near 64 at scales near 2^-6 that vary from page to page."""
    def codes(shape):
        x = torch.randn(shape, generator=gen, device=DEV, dtype=torch.float16).mul_(64.0)
        return x.clamp_(-448, 448).to(torch.float8_e4m3fn)
    out = {}
    for n, dim in (("k", case["dk"]), ("v", case["dv"])):
        out[n + "_data"] = _buffer(codes, pages, case["hkv"], case["page"], dim, case["layout"])
        out[n + "_scale"] = torch.exp2(torch.randint(-8, -3, (pages, case["hkv"]), generator=gen,
                                                     device=DEV).float())
    return out


def _handle(s, case):
    import nvfp4_paged_kv_nvfp4kv_gb300 as N
    if case.get("cache") == "e4m3":
        return N.E4m3Cache(s["k_data"], s["v_data"], s["k_scale"], s["v_scale"])
    bufs = [s[n] for n in ("k_data", "v_data", "k_sf", "v_sf")]
    strides = {n: (s[n].stride(0), s[n].stride(2), s[n].stride(1))
               for n in ("k_data", "v_data", "k_sf", "v_sf")}
    return N.PagedCache(*bufs, strides, bufs[0].shape[0], case["hkv"], case["dk"], case["dv"],
                        K_GLOBAL, V_GLOBAL, case["page"])


def _page_lists(gen, kv, page):
    npages = [_pages(a, page) for a in kv]
    total = max(1, sum(npages))
    perm = torch.randperm(total, generator=gen, device=DEV).to(torch.int32)
    last = [a - (n - 1) * page if n else 0 for a, n in zip(kv, npages)]
    return {"kv_indices": perm, "kv_indptr": _indptr(npages), "last_page_len": _i32(last),
            "max_pages": max(npages), "total": total}


def _parents(gen, new):
    """Trees in one list: node 0 of each request is a root, node i hangs below one of 0 .. i-1."""
    i = torch.cat([torch.arange(n, device=DEV) for n in new])
    u = torch.rand(i.numel(), generator=gen, device=DEV, dtype=torch.float64)
    return torch.where(i > 0, torch.minimum((u.sqrt() * i).long(), i - 1), -1).int()


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(int(seed))
    op = case["op"]
    s = {"case": dict(case)}
    if op == "norm_rope":
        t, hq, hkv, dim = case["tokens"], case["hq"], case["hkv"], case["dim"]
        dtype = DTYPES[case["dtype"]]
        qkv = torch.randn((t, hq + 2 * hkv, dim), generator=gen, device=DEV)
        # heads of different sizes, as projections make them
        qkv *= torch.exp2(torch.randint(-3, 4, (t, hq + 2 * hkv, 1), generator=gen, device=DEV))
        qkv = qkv.to(dtype)  # one projection's output: q, k and v side by side
        s["q"], s["k"] = qkv[:, :hq], qkv[:, hq:hq + hkv]
        s["positions"] = torch.randint(0, case["pos_hi"], (t,), generator=gen, device=DEV,
                                       dtype=torch.int32)
        for n in ("q_weight", "k_weight"):
            w = 1.0 - case["offset"] + 0.3 * torch.randn(dim, generator=gen, device=DEV)
            s[n] = w.to(torch.float32 if case["weight"] == "f32" else dtype)
        if own:
            from nvfp4_paged_kv_nvfp4kv_gb300 import nvfp4kv_rope_plan
            s["plan"] = nvfp4kv_rope_plan(
                dim, case["rotary"], base=case["base"], interleaved=case["interleaved"],
                factor=case["factor"], original_max_position=case["orig"],
                attention_factor=case["attn"])
        return s
    if op == "pages":
        kv = _ragged(case["batch"], case["kv_lo"], case["kv_hi"])
        page, b, copies = case["page"], case["batch"], case["copies"]
        npages = [_pages(a, page) for a in kv]
        width, forks, total = max(npages) + 1, b * copies, sum(npages)
        spare = forks + 9
        ids = torch.randperm(total + spare, generator=gen, device=DEV).to(torch.int32)
        col = torch.arange(width, device=DEV)
        n = torch.tensor(npages, device=DEV)
        at = ((torch.cumsum(n, 0) - n)[:, None] + col).clamp_(max=total - 1)
        # rows of the running requests, then empty rows for their continuations
        s["block_table"] = torch.full((b + forks, width), -1, dtype=torch.int32, device=DEV)
        s["block_table"][:b] = torch.where(col < n[:, None], ids[at], -1)
        s["parents"] = _i32([i % b for i in range(forks)])
        s["children"] = _i32([b + i for i in range(forks)])
        s["kv_len"] = _i32(kv + [0] * forks)
        s["keep_len"] = _i32(kv + [0] * forks)  # the continuations are given up
        # a few pages have more owners already (a shared prefix)
        s["page_shares"] = torch.randint(-3, 3, (total + spare,), generator=gen,
                                         device=DEV).clamp_(min=0).int()
        s["page_shares"][ids[total:].long()] = 0
        s["free_pages"], s["free_head"] = ids[total - 1:].clone(), _i32([1])
        s["free_head_mid"] = _i32([0])
        s["copy_src"], s["copy_dst"] = (torch.full((forks,), -7, dtype=torch.int32, device=DEV)
                                        for _ in range(2))
        s["entries"] = copies * total
        s.update(_nvfp4_pool(case, gen, total + spare))
        if own:
            s["cache"] = _handle(s, case)
        return s
    kv, new = _lengths(case)
    s["qo_indptr"], s["kv_len"], s["max_new"] = _indptr(new), _i32(kv), max(new)
    if op in ("masks", "tree"):
        s["parents"] = _parents(gen, new)
    if op == "masks":
        return s
    lists = _page_lists(gen, kv, case["page"])
    s.update(lists)
    if op == "compact":
        s.update((_e4m3_pool if case["cache"] == "e4m3" else _nvfp4_pool)(case, gen,
                                                                           lists["total"]))
        kept = _kept(case, new)
        # accepted nodes: some of each request's, in order
        order = torch.rand((len(new), max(new)), generator=gen, device=DEV)
        n = torch.tensor(new, device=DEV)[:, None]
        k = torch.tensor(kept, device=DEV)[:, None]
        order = torch.where(torch.arange(max(new), device=DEV) < n, order, 2.0).argsort(1)
        rank = torch.arange(max(new), device=DEV)
        path = torch.where(rank < k, order, max(new)).sort(1).values
        s["path"] = torch.where(rank < k, path, -1).int().contiguous()
        s["num_kept"] = _i32(kept)
        page = case["page"]
        s["touched"] = sum(_pages(a - m + c, page) - (a - m) // page
                           for a, m, c in zip(kv, new, kept) if c)
        if own:
            s["cache"] = _handle(s, case)
        return s
    s.update(_nvfp4_pool(case, gen, lists["total"]))
    s["q"] = torch.randn((sum(new), case["hq"], case["dk"]), generator=gen,
                         device=DEV).to(torch.bfloat16)
    s["scale"] = 1.0 / math.sqrt(case["dk"])
    s["tree_mask"], _ = _masks_plain(s)
    if own:
        from nvfp4_paged_kv_nvfp4kv_gb300 import nvfp4kv_decode_plan
        s["cache"] = _handle(s, case)
        s["plan"] = nvfp4kv_decode_plan(
            s["qo_indptr"], s["kv_indptr"], s["last_page_len"], case["hq"], case["hkv"],
            case["dk"], case["dv"], page_size=case["page"], out_dtype=DTYPES[case["out"]])
    return s


# ---- the plain forms -----------------------------------------------------------
def _norm_rope_plain(s):
    c = s["case"]
    rot = c["rotary"]
    f = c["base"] ** (-torch.arange(0, rot, 2, device=DEV, dtype=torch.float64) / rot)
    if c["orig"]:
        turns = c["orig"] * f / (2 * math.pi)
        keep = ((turns - 1.0) / 31.0).clamp(0, 1)
        f = f * (keep + (1 - keep) / c["factor"])
    else:
        f = f / c["factor"]
    angle = s["positions"].double()[:, None, None] * f
    cos, sin = (angle.cos() * c["attn"]).float(), (angle.sin() * c["attn"]).float()

    def turn(x, w):
        y = x.float()
        y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + 1e-6) * (w.float() + c["offset"])
        r = y[..., :rot]
        if c["interleaved"]:
            a, b = r[..., 0::2], r[..., 1::2]
            r = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
        else:
            a, b = r[..., : rot // 2], r[..., rot // 2:]
            r = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
        return torch.cat((r, y[..., rot:]), -1).to(x.dtype)

    return {"q": turn(s["q"], s["q_weight"]), "k": turn(s["k"], s["k_weight"])}


def _padded(s):
    """(request, index in its tree) of every row."""
    qo = s["qo_indptr"].long()
    t = torch.arange(s["parents"].numel(), device=DEV)
    rb = torch.searchsorted(qo[1:], t, right=True)
    return qo, rb, t - qo[rb]


def _masks_plain(s):
    qo, rb, ri = _padded(s)
    n, b = s["max_new"], qo.numel() - 1
    up = torch.eye(n, device=DEV).repeat(b, 1, 1)  # a node and its parent
    par = s["parents"].long()
    up[rb, ri, par.clamp(min=0)] = ((par >= 0) | (ri == 0)).float()
    # (node 0 has itself in place of a parent)
    for _ in range((n - 1).bit_length()):  # ancestors twice as far at each product
        up = (up @ up).clamp_(max=1.0)
    words = _pages(n, 32)
    seen = torch.nn.functional.pad(up, (0, 32 * words - n))[rb, ri].long()
    bit = torch.arange(32, device=DEV)
    mask = (seen.view(-1, words, 32) << bit).sum(-1).to(torch.int32)
    depth = up.sum(-1)[rb, ri].int() - 1
    new = (qo[1:] - qo[:-1]).int()
    return mask, (s["kv_len"] - new)[rb] + depth


def _e2m1(codes):
    """The values of packed 4-bit codes, low nibble first."""
    value = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=DEV)
    value = torch.cat((value, -value))
    both = torch.stack((codes & 15, codes >> 4), -1).flatten(-2)
    return value[both.int()]


def _dense(data, sf, scale, table):
    """[batch, heads, tokens, dims] in 32 bits of the pages that table lists."""
    x = _e2m1(data[table])
    x = x * sf[table].view(torch.float8_e4m3fn).float().repeat_interleave(16, -1) * scale
    b, w, h, p, d = x.shape
    return x.transpose(1, 2).reshape(b, h, w * p, d)


def _tree_plain(s):
    c = s["case"]
    page, hq, hkv = c["page"], c["hq"], c["hkv"]
    qo, rb, ri = _padded(s)
    kvp = s["kv_indptr"].long()
    new, pages = qo[1:] - qo[:-1], kvp[1:] - kvp[:-1]
    length = torch.where(pages > 0, (pages - 1) * page + s["last_page_len"], 0)
    col = torch.arange(s["max_pages"], device=DEV)
    at = (kvp[:-1, None] + col).clamp(max=s["kv_indices"].numel() - 1)
    table = torch.where(col < pages[:, None], s["kv_indices"][at], 0).long()
    k = _dense(s["k_data"], s["k_sf"], K_GLOBAL, table)
    v = _dense(s["v_data"], s["v_sf"], V_GLOBAL, table)
    b, n = new.numel(), s["max_new"]
    q = torch.zeros((b, n) + s["q"].shape[1:], device=DEV)
    q[rb, ri] = s["q"].float()
    q = q.view(b, n, hkv, hq // hkv, -1).permute(0, 2, 3, 1, 4).reshape(b, hkv, -1, c["dk"])
    x = (q @ k.transpose(2, 3)).view(b, hkv, hq // hkv, n, -1) * s["scale"]
    pos = torch.arange(x.shape[-1], device=DEV)
    # a node sees what stood before the tree, and the nodes whose bits are set
    node = pos - (length - new)[:, None]
    word = torch.zeros((b, n, s["tree_mask"].shape[1]), dtype=torch.int32, device=DEV)
    word[rb, ri] = s["tree_mask"]
    at = node.clamp(0, 32 * word.shape[2] - 1)
    bits = (word.gather(2, (at // 32)[:, None].expand(b, n, -1)) >> (at % 32)[:, None]) & 1
    seen = (node < 0)[:, None] | ((bits == 1) & (pos < length[:, None])[:, None])
    x = torch.where(seen[:, None, None], x, -math.inf)
    top = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(top == -math.inf, 0.0, top))
    total = p.sum(-1, keepdim=True)
    v = torch.where((pos < length[:, None])[:, None, :, None], v, 0.0)
    o = (p.view(b, hkv, -1, p.shape[-1]) @ v).view(b, hkv, hq // hkv, n, -1)
    o = torch.where(total > 0, o / total, 0.0)
    lse = (top + torch.log(total))[..., 0]
    o = o.permute(0, 3, 1, 2, 4).reshape(b, n, hq, -1)[rb, ri]
    return {"out": o.to(DTYPES[c["out"]]),
            "lse": lse.permute(0, 3, 1, 2).reshape(b, n, hq)[rb, ri].contiguous()}


def _tokens(s):
    """(request, rank, first drafted position, its node) of every accepted token, and a
    function that gives page and slot of a position."""
    page, kvp = s["case"]["page"], s["kv_indptr"].long()
    qo = s["qo_indptr"].long()
    start = s["kv_len"].long() - (qo[1:] - qo[:-1])
    rank = torch.arange(s["path"].shape[1], device=DEV)

    def place(b, pos):
        return s["kv_indices"][(kvp[b] + pos // page)].long(), pos % page
    return start, rank < s["num_kept"][:, None], place


def _compact_nvfp4_plain(s):
    start, kept, place = _tokens(s)
    b, i = kept.nonzero(as_tuple=True)
    sp, ss = place(b, start[b] + s["path"][b, i])
    dp, ds = place(b, start[b] + i)
    for n in ("k_data", "v_data", "k_sf", "v_sf"):
        s[n][dp, :, ds] = s[n][sp, :, ss]


def _compact_e4m3_plain(s):
    page = s["case"]["page"]
    start, kept, place = _tokens(s)
    count = s["num_kept"].long()
    first = start // page
    touched = torch.where(count > 0, (start + count - 1) // page + 1 - first, 0)
    b = torch.repeat_interleave(torch.arange(count.numel(), device=DEV), touched,
                                output_size=s["touched"])
    nth = torch.arange(s["touched"], device=DEV) - (torch.cumsum(touched, 0) - touched)[b]
    pos = ((first[b] + nth) * page)[:, None] + torch.arange(page, device=DEV)
    rank = pos - start[b][:, None]
    old, fresh = rank < 0, (rank >= 0) & (rank < count[b][:, None])
    node = s["path"][b[:, None], rank.clamp(0, s["path"].shape[1] - 1)]
    source = torch.where(fresh, start[b][:, None] + node, pos)
    source = torch.minimum(source, (s["kv_len"].long() - 1)[b][:, None])
    sp, ss = place(b[:, None].expand_as(source), source)
    pid = place(b, (first[b] + nth) * page)[0]
    takes = (old | fresh)[:, None, :]
    new_data = []
    for data, scale in ((s["k_data"], s["k_scale"]), (s["v_data"], s["v_scale"])):
        had = scale[sp].transpose(1, 2)  # [touched, heads, slots]
        now = torch.where(takes, had, 0.0).amax(2)
        codes = data.view(torch.uint8)[sp, :, ss].transpose(1, 2)
        y = codes.view(torch.float8_e4m3fn).float() * (had / now[..., None])[..., None]
        y = y.to(torch.float8_e4m3fn).view(torch.uint8)
        new_data.append((torch.where(takes[..., None], y, data.view(torch.uint8)[pid]), now))
    for (codes, now), data, scale in zip(new_data, (s["k_data"], s["v_data"]),
                                         (s["k_scale"], s["v_scale"])):
        data.view(torch.uint8)[pid] = codes
        scale[pid] = now


def _release_plain(s, keep_len, head):
    page = s["case"]["page"]
    length, keep = s["kv_len"].long(), keep_len.long()
    lo, hi = (keep + page - 1) // page, (length + page - 1) // page
    count = (hi - lo).clamp(min=0)
    n = s["entries"]
    b = torch.repeat_interleave(torch.arange(count.numel(), device=DEV), count, output_size=n)
    col = lo[b] + torch.arange(n, device=DEV) - (torch.cumsum(count, 0) - count)[b]
    pid = s["block_table"][b, col].long()
    shares = s["page_shares"].long()
    shares.index_add_(0, pid, torch.full_like(pid, -1))
    # a page whose last owner left is free: listed where it was given up first
    at = torch.full_like(shares, n).scatter_reduce_(0, pid, torch.arange(n, device=DEV), "amin")
    freed = (shares[pid] < 0) & (at[pid] == torch.arange(n, device=DEV))
    place = torch.cumsum(freed, 0)
    total = place[-1:]
    to = torch.where(freed, head.long() - total + place - 1, s["free_pages"].numel())
    listed_ = torch.cat((s["free_pages"], torch.zeros(1, dtype=torch.int32, device=DEV)))
    listed_[to] = torch.where(freed, pid, 0).int()
    s["free_pages"].copy_(listed_[:-1])
    s["page_shares"].copy_(shares.clamp(min=0))
    s["free_head"].copy_(head - total)
    s["kv_len"].copy_(torch.minimum(length, keep))


def _pages_plain(s):
    page, width = s["case"]["page"], s["block_table"].shape[1]
    par, child = s["parents"].long(), s["children"].long()
    length = s["kv_len"][par].long()
    whole, partial = length // page, (length % page > 0)
    taken = torch.cumsum(partial, 0)
    fresh = s["free_pages"][s["free_head"].long() + taken - 1]
    col = torch.arange(width, device=DEV)
    row = s["block_table"][par]
    last = row.gather(1, whole[:, None])[:, 0]
    shared = col < whole[:, None]
    s["page_shares"].index_add_(0, torch.where(shared, row, 0).long().flatten(),
                                shared.int().flatten())
    new = torch.where(shared, row, s["block_table"][child])
    new = torch.where((col == whole[:, None]) & partial[:, None], fresh[:, None], new)
    s["block_table"][child] = new
    s["kv_len"][child] = length.int()
    s["copy_src"].copy_(torch.where(partial, last, -1))
    s["copy_dst"].copy_(torch.where(partial, fresh, -1))
    head = s["free_head"] + taken[-1:]
    src, dst = s["copy_src"].long(), s["copy_dst"].long()
    some = src >= 0
    src, dst = src[some], dst[some]
    for n in ("k_data", "v_data", "k_sf", "v_sf"):
        s[n][dst] = s[n][src]
    _release_plain(s, s["keep_len"], head)


def _own(s):
    import nvfp4_paged_kv_nvfp4kv_gb300 as N
    c = s["case"]
    op = c["op"]
    if op == "norm_rope":
        q, k = N.nvfp4kv_norm_rope(s["plan"], s["q"], s["k"], s["positions"], s["q_weight"],
                                   s["k_weight"], eps=1e-6, weight_offset=c["offset"])
        return {"q": q, "k": k}
    if op == "masks":
        mask, positions = N.nvfp4kv_tree_masks(s["parents"], s["qo_indptr"], s["kv_len"],
                                               max_nodes=s["max_new"])
        return {"mask": mask, "positions": positions}
    if op == "tree":
        out, lse = N.nvfp4kv_tree_run(s["plan"], s["q"], s["cache"], s["kv_indices"],
                                      s["tree_mask"], s["scale"])
        return {"out": out, "lse": lse}
    if op == "compact":
        call = (N.nvfp4kv_e4m3_compact_tokens if c["cache"] == "e4m3"
                else N.nvfp4kv_compact_tokens)
        call(s["cache"], s["path"], s["num_kept"], s["qo_indptr"], s["kv_indptr"],
             s["kv_indices"], s["last_page_len"])
        return None
    N.nvfp4kv_fork_pages(s["parents"], s["children"], s["kv_len"], s["block_table"],
                         s["page_shares"], s["free_pages"], s["free_head"], s["free_head_mid"],
                         s["copy_src"], s["copy_dst"], page_size=c["page"])
    N.nvfp4kv_copy_pages(s["cache"], s["copy_src"], s["copy_dst"])
    N.nvfp4kv_release_pages(s["keep_len"], s["kv_len"], s["block_table"], s["page_shares"],
                            s["free_pages"], s["free_head_mid"], s["free_head"],
                            page_size=c["page"])
    return None


def _buffers(s):
    """What a call changed in place.  The 4-bit codes and their scales are moved and never
    computed: they are the bytes themselves."""
    names = ["k_data", "v_data"] + (["k_scale", "v_scale"] if "k_scale" in s else
                                    ["k_sf", "v_sf"])
    if s["case"]["op"] == "pages":
        names += ["block_table", "page_shares", "free_pages", "free_head", "kv_len", "copy_src",
                  "copy_dst"]
    return {n: s[n] for n in names}


def run(state):
    op = state["case"]["op"]
    if own:
        out = _own(state)
        return _buffers(state) if out is None else out
    if op == "norm_rope":
        return _norm_rope_plain(state)
    if op == "masks":
        mask, positions = _masks_plain(state)
        return {"mask": mask, "positions": positions}
    if op == "tree":
        return _tree_plain(state)
    if op == "pages":
        _pages_plain(state)
    elif state["case"]["cache"] == "e4m3":
        _compact_e4m3_plain(state)
    else:
        _compact_nvfp4_plain(state)
    return _buffers(state)


# ---- the definitions in 64 bits --------------------------------------------------
def _exact_norm_rope(s):
    c = s["case"]
    half = c["rotary"] // 2
    f = np.array([c["base"] ** (-(2.0 * i) / c["rotary"]) for i in range(half)])
    if c["orig"]:
        wave = 2 * np.pi / f
        g = np.clip((c["orig"] / wave - 1.0) / 31.0, 0.0, 1.0)
        f = (1 - g) * f / c["factor"] + g * f
    else:
        f = f / c["factor"]
    unit = torch.from_numpy(f).to(DEV)
    turn = torch.polar(torch.full_like(unit, c["attn"]).expand(c["tokens"], half),
                       s["positions"].double()[:, None] * unit)[:, None]
    out = {}
    for name in ("q", "k"):
        x = s[name].double()
        size = torch.linalg.vector_norm(x, dim=-1, keepdim=True) ** 2 / c["dim"] + 1e-6
        y = x / size.sqrt() * (s[name + "_weight"].double() + c["offset"])
        lo, hi = ((slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if c["interleaved"]
                  else (slice(0, half), slice(half, 2 * half)))
        z = torch.complex(y[..., lo].contiguous(), y[..., hi].contiguous()) * turn
        y[..., lo], y[..., hi] = z.real, z.imag
        out[name] = y
    return out


def _e2m1_exact(codes):
    value = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
    value = torch.from_numpy(np.concatenate((value, -value))).to(DEV)
    out = torch.empty(codes.shape[:-1] + (2 * codes.shape[-1],), dtype=torch.float64, device=DEV)
    out[..., 0::2], out[..., 1::2] = value[(codes % 16).long()], value[(codes // 16).long()]
    return out


def _e4m3_values():
    """The value of every E4M3 code: sign, 4 exponent bits (bias 7), 3 fraction bits."""
    out = np.empty(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        x = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        out[c] = (math.nan if e == 15 and m == 7 else x) * (-1 if c & 128 else 1)
    return out


def _exact_tree(s):
    c = s["case"]
    page, hkv, group = c["page"], c["hkv"], c["hq"] // c["hkv"]
    value = torch.from_numpy(_e4m3_values()).to(DEV)
    kv, new = _lengths(c)
    start = s["kv_indptr"].tolist()
    parents = s["parents"].tolist()
    outs, lses = [], []
    row = 0
    for b, (total, n) in enumerate(zip(kv, new)):
        pages = s["kv_indices"][start[b]:start[b + 1]].long()
        hide = torch.zeros((n, total), dtype=torch.bool)
        hide[:, total - n:] = True
        for i in range(n):
            j = i
            while j >= 0:  # a node sees itself and what it hangs below
                hide[i, total - n + j] = False
                j = parents[row + j]
        hide = hide.to(DEV)
        o = torch.empty((n, c["hq"], c["dv"]), dtype=torch.float64, device=DEV)
        z = torch.empty((n, c["hq"]), dtype=torch.float64, device=DEV)
        for h in range(hkv):
            kk, vv = ((_e2m1_exact(s[x + "_data"][:, h][pages])
                       * value[s[x + "_sf"][:, h][pages].long()].repeat_interleave(16, -1) * g)
                      .reshape(len(pages) * page, -1)[:total]
                      for x, g in (("k", K_GLOBAL), ("v", V_GLOBAL)))
            heads = slice(h * group, (h + 1) * group)
            q = s["q"][row:row + n, heads].double()
            score = torch.einsum("ngd,ld->ngl", q, kk) * s["scale"]
            score.masked_fill_(hide[:, None, :], -math.inf)
            z[:, heads] = torch.logsumexp(score, -1)
            o[:, heads] = torch.einsum("ngl,ld->ngd", torch.exp(score - z[:, heads, None]), vv)
        outs.append(o)
        lses.append(z)
        row += n
    return {"out": torch.cat(outs), "lse": torch.cat(lses)}


def _e4m3_round(x):
    """The nearest E4M3 value of each element, ties to the even code."""
    size = np.abs(x)
    step = 2.0 ** (np.maximum(np.frexp(size)[1] - 1, -6) - 3)
    return np.copysign(np.rint(size / step) * step, x)


def _exact_compact(s):
    c = s["case"]
    page = c["page"]
    kv, new = _lengths(c)
    kept = s["num_kept"].tolist()
    path, ids = s["path"].cpu().numpy(), s["kv_indices"].cpu().numpy()
    start = s["kv_indptr"].tolist()
    out = {}
    for n in ("k", "v"):
        codes = _e4m3_values()[s[n + "_data"].contiguous().view(torch.uint8).cpu().numpy()]
        scale = s[n + "_scale"].double().cpu().numpy()
        for b in range(len(kv)):
            base = kv[b] - new[b]
            first = base // page
            for at in range(first, _pages(base + kept[b], page) if kept[b] else 0):
                p = ids[start[b] + at]
                lo = max(base - at * page, 0)
                hi = min(base + kept[b] - at * page, page)
                src = [base + path[b, at * page + x - base] for x in range(lo, hi)]
                from_ = [(ids[start[b] + x // page], x % page) for x in src]
                moved = np.stack([codes[q, :, z] * scale[q][:, None] for q, z in from_], 1)
                now = np.max([scale[q] for q, _ in from_] + ([scale[p]] if lo else []), 0)
                codes[p, :, :lo] = _e4m3_round(codes[p, :, :lo] * (scale[p] / now)[:, None, None])
                codes[p, :, lo:hi] = _e4m3_round(moved / now[:, None, None])
                scale[p] = now
        out[n + "_data"], out[n + "_scale"] = torch.from_numpy(codes), torch.from_numpy(scale)
    return out


def exact(case, seed):
    op = case["op"]
    if op in ("masks", "pages") or case.get("cache") == "nvfp4":
        return None  # whole numbers only
    s = prepare(case, seed)
    return {"norm_rope": _exact_norm_rope, "tree": _exact_tree, "compact": _exact_compact}[op](s)
