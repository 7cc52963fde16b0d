"""The operators of a serving step beside the 4-bit attention, as cases to measure.

``tables``: the step's page table and slot maps from request lengths;
``rope``: rotary positions of the query and key heads;
``append``: new tokens into a paged cache of E4M3 codes with one scale per page and kv head;
``attend``: decode and extend attention over that cache.

With ``own`` false every operator runs in plain torch operations in 32 bits (angles in 64).
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


# ---- the cases ---------------------------------------------------------------
def _tables(batch, kv, new, page=16):
    return {"op": "tables", "batch": batch, "kv_lo": kv[0], "kv_hi": kv[1], "new_lo": new[0],
            "new_hi": new[1], "page": page}


def _rope(tokens, hq, hkv, dim, rotary, interleaved, pos_hi, dtype="bf16", base=10000.0,
          factor=1.0, orig=0, low=1.0, high=32.0, attn=1.0):
    return {"op": "rope", "tokens": tokens, "hq": hq, "hkv": hkv, "dim": dim, "rotary": rotary,
            "interleaved": interleaved, "pos_hi": pos_hi, "dtype": dtype, "base": base,
            "factor": factor, "orig": orig, "low": low, "high": high, "attn": attn}


def _append(batch, held, new, hkv, dk, dv, page=16, layout="HND", dtype="bf16"):
    return {"op": "append", "batch": batch, "held_lo": held[0], "held_hi": held[1],
            "new_lo": new[0], "new_hi": new[1], "hkv": hkv, "dk": dk, "dv": dv, "page": page,
            "layout": layout, "dtype": dtype}


def _attend(batch, kv, new, hq, hkv, dk, dv, causal, page=16, layout="HND", dtype="bf16",
            out="bf16"):
    return {"op": "attend", "batch": batch, "kv_lo": kv[0], "kv_hi": kv[1], "new_lo": new[0],
            "new_hi": new[1], "hq": hq, "hkv": hkv, "dk": dk, "dv": dv, "causal": causal,
            "page": page, "layout": layout, "dtype": dtype, "out": out}


def listed():
    return [
        # every request of a running batch makes one token: latency counts
        dict(_tables(64, (1, 8192), (1, 1)), name="tables_decode_step"),
        # a full server: long histories, a few prompts in chunks, some requests idle
        dict(_tables(1000, (0, 131071), (0, 2048)), name="tables_long_histories"),
        # one decode step of a batch: 32 query and 8 kv heads of 128
        dict(_rope(16, 32, 8, 128, 128, False, 4096), name="rope_decode_step"),
        # a prompt chunk of an odd length, neighbouring pairs, a quarter of the head, f16
        dict(_rope(8191, 16, 2, 256, 64, True, 32768, "f16"), name="rope_prompt_part_pairs"),
        # long prompts far beyond the trained length, frequencies scaled by parts
        dict(_rope(16384, 32, 8, 128, 128, False, 1 << 20, "bf16", 500000.0, 32.0, 8192, 1.0,
                   32.0, 1.3465735902799727), name="rope_long_prompt_scaled"),
        # one new token for each request of the batched decode, pages partly full
        dict(_append(16, (511, 4095), (1, 1), 8, 128, 128), name="append_decode_step"),
        # prompt chunks that begin and end inside pages
        dict(_append(7, (5, 3000), (700, 2301), 8, 128, 128), name="append_prompt_chunks"),
        # two short requests: the smallest attention call
        dict(_attend(2, (37, 100), (1, 1), 4, 1, 128, 128, False), name="attend_tiny_decode"),
        # a batch of ordinary lengths, one query row each
        dict(_attend(16, (512, 4096), (1, 1), 32, 8, 128, 128, False),
             name="attend_batched_decode"),
        # few requests, long histories with a partial last page: work split over the tokens
        dict(_attend(4, (32771, 32771), (1, 1), 32, 8, 128, 128, False),
             name="attend_long_decode"),
        # query and key heads of 512, values of 256, slots before heads in memory, f16 out
        dict(_attend(8, (2048, 8192), (1, 1), 16, 2, 512, 256, False, 16, "NHD", "bf16", "f16"),
             name="attend_wide_heads_decode"),
        # 16 new rows behind a long prefix: the extend of a prefix cache
        dict(_attend(32, (2000, 16000), (16, 16), 32, 8, 128, 128, True),
             name="attend_prefix_extend"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tables", "rope", "append", "attend", "attend"])
    page = rng.choice([16, 16, 16, 1])
    if op == "tables":
        hi = _log_int(rng, 16, 131071 if page == 16 else 4095)
        return _tables(_log_int(rng, 1, 1000), (rng.choice([0, 1, hi // 3]), hi),
                       (rng.choice([0, 1]), _log_int(rng, 1, min(hi, 2048))), page)
    if op == "rope":
        dim = rng.choice([64, 128, 256])
        interleaved = rng.random() < 0.5
        rotary = rng.choice([dim, dim, dim // 2, 2 * rng.randint(1, dim // 2)])
        hkv = rng.choice([1, 2, 8])
        scaled = rng.random() < 0.5
        return _rope(_log_int(rng, 1, 8192), hkv * rng.choice([1, 4, 5]), hkv, dim, rotary,
                     interleaved, _log_int(rng, 64, 1 << 20), rng.choice(["bf16", "f16"]),
                     rng.choice([10000.0, 500000.0]), rng.uniform(1.5, 40.0) if scaled else 1.0,
                     rng.choice([0, 4096, 8192]) if scaled else 0, 1.0, rng.choice([4.0, 32.0]),
                     rng.choice([1.0, 1.25]))
    hkv = rng.choice([1, 2, 8])
    dk, dv = rng.choice([(64, 64), (128, 128), (128, 128), (256, 256), (256, 128), (512, 256)])
    layout, dtype = rng.choice(["HND", "NHD"]), rng.choice(["bf16", "bf16", "f16"])
    if op == "append":
        batch = _log_int(rng, 1, 64)
        return _append(batch, (rng.randint(0, 17), _log_int(rng, 18, 2000)),
                       (rng.choice([0, 1]), _log_int(rng, 1, 8192 // batch)), hkv, dk, dv, page,
                       layout, dtype)
    batch = _log_int(rng, 1, 32)
    hi = _log_int(rng, 16, min(32771, 500000000 // (batch * hkv * (dk + dv))))
    causal = rng.random() < 0.5
    new = rng.choice([1, 1, rng.randint(2, 16), rng.randint(17, 64)])
    return _attend(batch, (rng.randint(1, hi), hi), (rng.choice([0, 1, new]), new),
                   hkv * rng.choice([1, 4, 5, 8]), hkv, dk, dv, causal, page, layout, dtype,
                   rng.choice(["bf16", "bf16", "f16"]))


def _ragged(n, lo, hi, power=1.0):
    """n lengths over [lo, hi], the same for every seed: both ends and what lies between."""
    if n == 1:
        return [hi]
    f = [(0.6180339887498949 * i) % 1.0 for i in range(n)]
    f[0], f[-1] = 0.0, 1.0
    return [lo + int((hi - lo) * x ** power + 0.5) for x in f]


def _lengths(case):
    """(tokens held after the step, new tokens) of every request."""
    b, op = case["batch"], case["op"]
    if op == "append":
        new = _ragged(b, case["new_lo"], case["new_hi"])[::-1]
        return [h + n for h, n in zip(_ragged(b, case["held_lo"], case["held_hi"]), new)], new
    kv = _ragged(b, case["kv_lo"], case["kv_hi"])
    new = _ragged(b, case["new_lo"], case["new_hi"], 8.0 if op == "tables" else 1.0)[::-1]
    return kv, [min(n, length) for n, length in zip(new, kv)]


def _pages(n, page):
    return -(-n // page)


def work(case):
    op = case["op"]
    if op == "rope":
        heads = case["hq"] + case["hkv"]
        rot = case["tokens"] * heads * case["rotary"]
        return {"bytes": 4 * case["tokens"] * heads * case["dim"] + 4 * case["tokens"],
                "flops": 3 * rot}
    kv, new = _lengths(case)
    page = case["page"]
    if op == "tables":
        held = [_pages(a - n, page) for a, n in zip(kv, new)]
        every = [_pages(a, page) for a in kv]
        return {"bytes": 4 * sum(held) + 4 * sum(every) + 8 * (sum(every) - sum(held))
                + 16 * sum(new) + 20 * len(kv), "flops": sum(every)}
    row = case["hkv"] * (case["dk"] + case["dv"])
    if op == "append":
        touched = sum(_pages(a, page) - (a - n) // page for a, n in zip(kv, new) if n)
        return {"bytes": 3 * row * sum(new) + 8 * case["hkv"] * touched + 4 * touched,
                "flops": 2 * row * sum(new)}
    act = [(a, n) for a, n in zip(kv, new) if n]
    rows = sum(n for _, n in act)
    seen = sum(sum(a - n + i + 1 for i in range(n)) if case["causal"] else a * n for a, n in act)
    pages = sum(_pages(a, page) for a, _ in act)
    return {"bytes": row * sum(a for a, _ in act) + 8 * case["hkv"] * pages + 4 * pages
            + rows * case["hq"] * (2 * case["dk"] + 2 * case["dv"] + 4),
            "flops": 2 * (case["dk"] + case["dv"]) * case["hq"] * seen}


# ---- what a program has in hand ------------------------------------------------
def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _indptr(counts):
    return _i32([0] + list(np.cumsum(counts)))


def _pool(gen, pages, heads, page, dim, layout):
    """E4M3 codes (finite ones) in pages x heads x slots x dims, in memory in the given layout."""
    shape = (pages, heads, page, dim) if layout == "HND" else (pages, page, heads, dim)
    x = torch.randn(shape, generator=gen, device=DEV, dtype=torch.float16).mul_(64.0)
    x = x.clamp_(-448, 448).to(torch.float8_e4m3fn)
    return x if layout == "HND" else x.transpose(1, 2)


def _cache_state(case, gen, kv):
    page, hkv = case["page"], case["hkv"]
    npages = [_pages(a, page) for a in kv]
    total = max(1, sum(npages))
    k = _pool(gen, total, hkv, page, case["dk"], case["layout"])
    v = _pool(gen, total, hkv, page, case["dv"], case["layout"])
    # values near 1: codes near 64 at scales near 2^-6, that vary from page to page
    ks = torch.exp2(torch.randint(-7, -4, (total, hkv), generator=gen, device=DEV).float())
    vs = torch.exp2(torch.randint(-7, -4, (total, hkv), generator=gen, device=DEV).float())
    perm = torch.randperm(total, generator=gen, device=DEV).to(torch.int32)
    last = [a - (n - 1) * page if n else 0 for a, n in zip(kv, npages)]
    return {"k_data": k, "v_data": v, "k_scale": ks, "v_scale": vs, "kv_indices": perm,
            "kv_indptr": _indptr(npages), "last_page_len": _i32(last), "max_pages": max(npages)}


def _handle(s):
    from nvfp4_paged_kv_nvfp4kv_gb300 import E4m3Cache
    return E4m3Cache(s["k_data"], s["v_data"], s["k_scale"], s["v_scale"])


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(int(seed))
    op = case["op"]
    s = {"case": dict(case)}
    if op == "rope":
        t, hq, hkv, dim = case["tokens"], case["hq"], case["hkv"], case["dim"]
        qkv = torch.randn((t, hq + 2 * hkv, dim), generator=gen, device=DEV)
        qkv = qkv.to(DTYPES[case["dtype"]])  # one projection's output: q, k and v side by side
        s["q"], s["k"] = qkv[:, :hq], qkv[:, hq:hq + hkv]
        s["positions"] = torch.randint(0, case["pos_hi"], (t,), generator=gen, device=DEV,
                                       dtype=torch.int32)
        if own:
            from nvfp4_paged_kv_nvfp4kv_gb300 import nvfp4kv_rope_plan
            s["plan"] = nvfp4kv_rope_plan(
                dim, case["rotary"], base=case["base"], interleaved=case["interleaved"],
                factor=case["factor"], original_max_position=case["orig"],
                low_rotations=case["low"], high_rotations=case["high"],
                attention_factor=case["attn"])
        return s
    kv, new = _lengths(case)
    page = case["page"]
    if op == "tables":
        held = [_pages(a - n, page) for a, n in zip(kv, new)]
        every = [_pages(a, page) for a in kv]
        b, width = case["batch"], max(max(every), 1)
        total = max(1, sum(every))
        ids = torch.randperm(total, generator=gen, device=DEV).to(torch.int32)
        col = torch.arange(width, device=DEV)
        heldt = torch.tensor(held, device=DEV)
        start = torch.cumsum(heldt, 0) - heldt
        at = (start[:, None] + col).clamp_(max=total - 1)
        s["block_table"] = torch.where(col < heldt[:, None], ids[at], -1).contiguous()
        skip = 3  # the list's head stands behind pages that are taken already
        s["free_pages"] = torch.cat([ids[:skip], ids[sum(held):]])
        s["free_head"] = _i32([min(skip, total)])
        s["kv_len"], s["qo_len"] = _i32(kv), _i32(new)
        s["num_tokens"], s["num_pages"] = sum(new), sum(every)
        # room for more rows than this step has: they stay as they are
        tokens, pages = sum(new) + 13, sum(every) + 5
        for name, n in (("qo_indptr", b + 1), ("kv_indptr", b + 1), ("last_page_len", b),
                        ("kv_indices", pages), ("batch_idx", tokens), ("positions", tokens),
                        ("free_head_out", 1)):
            s[name] = torch.full((n,), -7, dtype=torch.int32, device=DEV)
        s["slot_map"] = torch.full((tokens,), -7, dtype=torch.int64, device=DEV)
        if own:
            from nvfp4_paged_kv_nvfp4kv_gb300 import StepTable
            s["table"] = StepTable(s["qo_indptr"], s["kv_indptr"], s["last_page_len"],
                                   s["kv_indices"], s["batch_idx"], s["positions"],
                                   s["slot_map"], s["free_head_out"])
        return s
    s.update(_cache_state(case, gen, kv))
    s["qo_indptr"] = _indptr(new)
    rows = sum(new)
    dtype = DTYPES[case["dtype"]]
    if op == "append":
        for name, dim in (("k", case["dk"]), ("v", case["dv"])):
            x = torch.randn((rows, case["hkv"], dim), generator=gen, device=DEV)
            # some tokens are larger than what their page holds, so that its scale grows
            x *= torch.exp2(torch.randint(-3, 4, (rows, 1, 1), generator=gen, device=DEV))
            s[name] = x.to(dtype)
        s["touched"] = sum(_pages(a, page) - (a - n) // page for a, n in zip(kv, new) if n)
        if own:
            s["cache"] = _handle(s)
        return s
    s["q"] = torch.randn((rows, case["hq"], case["dk"]), generator=gen, device=DEV).to(dtype)
    s["max_new"] = max(new)
    s["scale"] = 1.0 / math.sqrt(case["dk"])
    if own:
        from nvfp4_paged_kv_nvfp4kv_gb300 import nvfp4kv_decode_plan
        s["cache"] = _handle(s)
        s["plan"] = nvfp4kv_decode_plan(
            s["qo_indptr"], s["kv_indptr"], s["last_page_len"], case["hq"], case["hkv"],
            case["dk"], case["dv"], page_size=page, causal=case["causal"], kernel=5,
            out_dtype=DTYPES[case["out"]])
    return s


# ---- the plain forms -----------------------------------------------------------
def _tables_plain(s):
    page, b = s["case"]["page"], s["case"]["batch"]
    kv, new = s["kv_len"].long(), s["qo_len"].long()
    held, every = (kv - new + page - 1) // page, (kv + page - 1) // page
    taken = every - held
    zero = torch.zeros(1, dtype=torch.long, device=DEV)
    qo, kvp, fresh = (torch.cat([zero, torch.cumsum(x, 0)]) for x in (new, every, taken))
    s["qo_indptr"].copy_(qo)
    s["kv_indptr"].copy_(kvp)
    s["last_page_len"].copy_(torch.where(every > 0, kv - (every - 1) * page, 0))
    s["free_head_out"].copy_(s["free_head"] + fresh[-1])
    req = torch.arange(b, device=DEV)
    pb = torch.repeat_interleave(req, every, output_size=s["num_pages"])
    pc = torch.arange(s["num_pages"], device=DEV) - kvp[pb]
    at = s["free_head"].long() + fresh[pb] + (pc - held[pb]).clamp(min=0)
    at = at.clamp(max=s["free_pages"].numel() - 1)
    ids = torch.where(pc < held[pb], s["block_table"][pb, pc], s["free_pages"][at])
    s["block_table"][pb, pc] = ids
    s["kv_indices"][: s["num_pages"]] = ids
    tb = torch.repeat_interleave(req, new, output_size=s["num_tokens"])
    pos = torch.arange(s["num_tokens"], device=DEV) - qo[tb] + (kv - new)[tb]
    s["batch_idx"][: s["num_tokens"]] = tb.int()
    s["positions"][: s["num_tokens"]] = pos.int()
    s["slot_map"][: s["num_tokens"]] = s["block_table"][tb, pos // page].long() * page + pos % page


def _tables_out(s):
    return {n: s[n] for n in ("block_table", "qo_indptr", "kv_indptr", "last_page_len",
                              "kv_indices", "batch_idx", "positions", "slot_map",
                              "free_head_out")}


def _rope_plain(s):
    c = s["case"]
    rot = c["rotary"]
    f = c["base"] ** (-torch.arange(0, rot, 2, device=DEV, dtype=torch.float64) / rot)
    if c["orig"]:
        turns = c["orig"] * f / (2 * math.pi)
        keep = ((turns - c["low"]) / (c["high"] - c["low"])).clamp(0, 1)
        f = f * (keep + (1 - keep) / c["factor"])
    else:
        f = f / c["factor"]
    angle = s["positions"].double()[:, None, None] * f
    cos, sin = (angle.cos() * c["attn"]).float(), (angle.sin() * c["attn"]).float()

    def turn(x):
        r = x[..., :rot].float()
        if c["interleaved"]:
            a, b = r[..., 0::2], r[..., 1::2]
            y = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
        else:
            a, b = r[..., : rot // 2], r[..., rot // 2:]
            y = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
        return torch.cat((y.to(x.dtype), x[..., rot:]), -1)

    return {"q": turn(s["q"]), "k": turn(s["k"])}


def _append_plain(s):
    page = s["case"]["page"]
    qo, kvp = s["qo_indptr"].long(), s["kv_indptr"].long()
    new = qo[1:] - qo[:-1]
    pages = kvp[1:] - kvp[:-1]
    length = torch.where(pages > 0, (pages - 1) * page + s["last_page_len"], 0)
    first = (length - new) // page
    count = torch.where(new > 0, pages - first, 0)
    b = torch.repeat_interleave(torch.arange(new.numel(), device=DEV), count,
                                output_size=s["touched"])
    nth = torch.arange(s["touched"], device=DEV) - (torch.cumsum(count, 0) - count)[b]
    pid = s["kv_indices"][kvp[b] + first[b] + nth].long()
    pos = ((first[b] + nth) * page)[:, None] + torch.arange(page, device=DEV)
    begin = (length - new)[b][:, None]
    old = (pos < begin)[:, None, :, None]
    fresh = ((pos >= begin) & (pos < length[b][:, None]))[:, None, :, None]
    row = (qo[b][:, None] + pos - begin).clamp(0, max(s["k"].shape[0] - 1, 0))
    for x, data, scale in ((s["k"], s["k_data"], s["k_scale"]), (s["v"], s["v_data"], s["v_scale"])):
        new_x = x[row].transpose(1, 2).float()
        size = torch.where(fresh & new_x.isfinite(), new_x.abs(), 0.0).amax((2, 3))
        frac, e = torch.frexp(size)
        e = torch.where(size > 0, e - 8 - (frac <= 0.875).int(), -64).clamp(-64, 64)
        want = torch.ldexp(torch.ones_like(size), e)
        had = scale[pid]
        now = torch.where(old[:, :, 0, 0], torch.maximum(had, want), want)
        codes = data[pid]
        y = torch.where(fresh, new_x / now[..., None, None],
                        codes.float() * (had / now)[..., None, None]).clamp(-448, 448)
        y = torch.where(fresh | old, y.to(torch.float8_e4m3fn).view(torch.uint8),
                        codes.view(torch.uint8))
        data.view(torch.uint8)[pid] = y
        scale[pid] = now


def _dense(data, scale, table):
    """[batch, heads, tokens, dims] in 32 bits of the pages that table lists."""
    x = data[table].float() * scale[table][..., None, None]
    b, w, h, p, d = x.shape
    return x.transpose(1, 2).reshape(b, h, w * p, d)


def _attend_plain(s):
    c = s["case"]
    page, hq, hkv = c["page"], c["hq"], c["hkv"]
    qo, kvp = s["qo_indptr"].long(), s["kv_indptr"].long()
    new, pages = qo[1:] - qo[:-1], kvp[1:] - kvp[:-1]
    length = torch.where(pages > 0, (pages - 1) * page + s["last_page_len"], 0)
    col = torch.arange(s["max_pages"], device=DEV)
    at = (kvp[:-1, None] + col).clamp(max=s["kv_indices"].numel() - 1)
    table = torch.where(col < pages[:, None], s["kv_indices"][at], 0).long()
    k = _dense(s["k_data"], s["k_scale"], table)
    v = _dense(s["v_data"], s["v_scale"], table)
    b, n, rows = new.numel(), s["max_new"], s["q"].shape[0]
    i = torch.arange(n, device=DEV)
    q = s["q"][(qo[:-1, None] + i).clamp(max=rows - 1)].float()
    q = q.view(b, n, hkv, hq // hkv, -1).permute(0, 2, 3, 1, 4).reshape(b, hkv, -1, c["dk"])
    x = (q @ k.transpose(2, 3)).view(b, hkv, hq // hkv, n, -1) * s["scale"]
    pos = torch.arange(x.shape[-1], device=DEV)
    live = pos < length[:, None]
    reach = (length - new)[:, None] + i if c["causal"] else (length - 1)[:, None] + 0 * i
    seen = live[:, None, :] & (pos <= reach[..., None])
    x = torch.where(seen[:, None, None], x, -math.inf)
    top = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(top == -math.inf, 0.0, top))
    total = p.sum(-1, keepdim=True)
    v = torch.where(live[:, None, :, None], v, 0.0)
    o = (p.view(b, hkv, -1, p.shape[-1]) @ v).view(b, hkv, hq // hkv, n, -1) / total
    lse = (top + torch.log(total))[..., 0]
    t = torch.arange(rows, device=DEV)
    rb = torch.searchsorted(qo[1:], t, right=True)
    ri = t - qo[rb]
    o = o.permute(0, 3, 1, 2, 4).reshape(b, n, hq, -1)[rb, ri]
    return {"out": o.to(DTYPES[c["out"]]),
            "lse": lse.permute(0, 3, 1, 2).reshape(b, n, hq)[rb, ri].contiguous()}


def run(state):
    op = state["case"]["op"]
    if own:
        import nvfp4_paged_kv_nvfp4kv_gb300 as N
        if op == "tables":
            N.nvfp4kv_build_page_table(state["kv_len"], state["qo_len"], state["block_table"],
                                       state["free_pages"], state["free_head"], state["table"],
                                       page_size=state["case"]["page"])
            return _tables_out(state)
        if op == "rope":
            q, k = N.nvfp4kv_rope(state["plan"], state["q"], state["k"], state["positions"])
            return {"q": q, "k": k}
        if op == "append":
            N.nvfp4kv_e4m3_append(state["cache"], state["k"], state["v"], state["qo_indptr"],
                                  state["kv_indptr"], state["kv_indices"],
                                  state["last_page_len"])
            return {n: state[n] for n in ("k_data", "v_data", "k_scale", "v_scale")}
        out, lse = N.nvfp4kv_e4m3_decode_run(state["plan"], state["q"], state["cache"],
                                             state["kv_indices"], state["scale"])
        return {"out": out, "lse": lse}
    if op == "tables":
        _tables_plain(state)
        return _tables_out(state)
    if op == "rope":
        return _rope_plain(state)
    if op == "append":
        _append_plain(state)
        return {n: state[n] for n in ("k_data", "v_data", "k_scale", "v_scale")}
    return _attend_plain(state)


# ---- the definitions in 64 bits --------------------------------------------------
def _e4m3_values():
    """The value of every E4M3 code: sign, 4 exponent bits (bias 7), 3 fraction bits."""
    out = np.empty(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        x = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        out[c] = (math.nan if e == 15 and m == 7 else x) * (-1 if c & 128 else 1)
    return out


def _e4m3_round(x):
    """The nearest E4M3 value of each element, ties to the even code, at most 448 in size."""
    size = np.abs(x)
    step = 2.0 ** (np.maximum(np.frexp(size)[1] - 1, -6) - 3)
    return np.copysign(np.minimum(np.rint(size / step) * step, 448.0), x)


def _exact_rope(s):
    c = s["case"]
    half = c["rotary"] // 2
    f = np.array([c["base"] ** (-(2.0 * i) / c["rotary"]) for i in range(half)])
    if c["orig"]:
        wave = 2 * np.pi / f
        g = np.clip((c["orig"] / wave - c["low"]) / (c["high"] - c["low"]), 0.0, 1.0)
        f = (1 - g) * f / c["factor"] + g * f
    else:
        f = f / c["factor"]
    unit = torch.from_numpy(f).to(DEV)
    turn = torch.polar(torch.full_like(unit, c["attn"]).expand(c["tokens"], half),
                       s["positions"].double()[:, None] * unit)[:, None]
    out = {}
    for name in ("q", "k"):
        y = s[name].double().clone()
        lo, hi = ((slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if c["interleaved"]
                  else (slice(0, half), slice(half, 2 * half)))
        z = torch.complex(y[..., lo].contiguous(), y[..., hi].contiguous()) * turn
        y[..., lo], y[..., hi] = z.real, z.imag
        out[name] = y
    return out


def _exact_append(s):
    c = s["case"]
    page = c["page"]
    value = _e4m3_values()
    kv, new = _lengths(c)
    ids = s["kv_indices"].cpu().numpy()
    start = s["kv_indptr"].cpu().numpy()
    rows = s["qo_indptr"].cpu().numpy()
    out = {}
    for n in ("k", "v"):
        x = s[n].double().cpu().numpy()
        codes = value[s[n + "_data"].contiguous().view(torch.uint8).cpu().numpy()]
        scale = s[n + "_scale"].double().cpu().numpy()
        for b, (total, fresh) in enumerate(zip(kv, new)):
            begin = total - fresh
            for at in range(begin // page, _pages(total, page) if fresh else 0):
                p = ids[start[b] + at]
                lo, hi = max(begin - at * page, 0), min(total - at * page, page)
                r = rows[b] + at * page + lo - begin
                block = x[r:r + hi - lo].transpose(1, 0, 2)
                size = np.abs(block).max((1, 2))
                e = [-64 if z == 0 else min(max(math.ceil(math.log2(z / 448.0)), -64), 64)
                     for z in size]
                want = np.array([2.0 ** k for k in e])
                now = np.maximum(want, scale[p]) if lo else want
                codes[p, :, :lo] = _e4m3_round(codes[p, :, :lo] * (scale[p] / now)[:, None, None])
                codes[p, :, lo:hi] = _e4m3_round(block / now[:, None, None])
                scale[p] = now
        out[n + "_data"], out[n + "_scale"] = torch.from_numpy(codes), torch.from_numpy(scale)
    return out


def _exact_attend(s):
    c = s["case"]
    page, hkv, group = c["page"], c["hkv"], c["hq"] // c["hkv"]
    value = torch.from_numpy(_e4m3_values()).to(DEV)
    kv, new = _lengths(c)
    start = s["kv_indptr"].tolist()
    outs, lses = [], []
    row = 0
    for b, (total, n) in enumerate(zip(kv, new)):
        if n == 0:
            continue
        pages = s["kv_indices"][start[b]:start[b + 1]].long()
        o = torch.empty((n, c["hq"], c["dv"]), dtype=torch.float64, device=DEV)
        z = torch.empty((n, c["hq"]), dtype=torch.float64, device=DEV)
        limit = torch.arange(total - n, total, device=DEV) if c["causal"] else \
            torch.full((n,), total - 1, device=DEV)
        hide = torch.arange(total, device=DEV)[None, :] > limit[:, None]
        for h in range(hkv):
            kk, vv = ((value[s[x + "_data"][:, h].view(torch.uint8)[pages].long()]
                       * s[x + "_scale"][pages, h].double()[:, None, None])
                      .reshape(len(pages) * page, -1)[:total] for x in ("k", "v"))
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


def exact(case, seed):
    op = case["op"]
    if op == "tables":
        return None  # whole numbers only
    s = prepare(case, seed)
    return {"rope": _exact_rope, "append": _exact_append, "attend": _exact_attend}[op](s)
