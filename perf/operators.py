"""What is measured of the chunk-step operators: their cases, inputs, plain forms and 64-bit values.

The three operators make one serving step over a paged KV cache:

  tables      block tables, page lists, positions and slots of a step, from the requests' lengths
  norm_rope   per-head RMS norms of q and k, position rotation, q written out, k and v into their pages
  chunk       attention of each request's new tokens over its pages

Every case is a dict of plain values; the request lengths of a case follow from its `lens` seed, the
values (and page orders) from the seed given to `prepare`.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # a decode step's tables: 128 requests with one new token each, pages of 16
        {"name": "tables_decode", "op": "tables", "batch": 128, "page": 16, "cached_min": 512, "cached_max": 4095,
         "new_min": 1, "new_max": 1, "prefills": 0, "prefill": 0, "pad": 0, "lens": 1002},
        # one prefill of 1024 tokens among 63 decodes, rows padded as a captured step pads them
        {"name": "tables_mixed", "op": "tables", "batch": 64, "page": 16, "cached_min": 511, "cached_max": 575,
         "new_min": 1, "new_max": 1, "prefills": 1, "prefill": 1024, "pad": 193, "lens": 1004},
        # a large server: 1000 requests of up to 32768 tokens, 64 of them bringing 1000 tokens
        {"name": "tables_large", "op": "tables", "batch": 1000, "page": 16, "cached_min": 1, "cached_max": 32768,
         "new_min": 1, "new_max": 7, "prefills": 64, "prefill": 1000, "pad": 0, "lens": 7},
        # the same decode step's queries and keys: where the call's latency counts
        {"name": "norm_rope_decode", "op": "norm_rope", "tokens": 128, "hq": 32, "hkv": 8, "dim": 128, "rope": 128,
         "interleaved": False, "page": 16, "layout": "HND", "dtype": "bf16", "far": 4096},
        # a prefill of 8 x 512 tokens, 40 heads
        {"name": "norm_rope_prefill", "op": "norm_rope", "tokens": 4096, "hq": 40, "hkv": 40, "dim": 128, "rope": 128,
         "interleaved": False, "page": 16, "layout": "HND", "dtype": "bf16", "far": 512},
        # a large chunked prefill at far positions, half of each head rotated, token-major pages
        {"name": "norm_rope_large", "op": "norm_rope", "tokens": 16384, "hq": 32, "hkv": 8, "dim": 128, "rope": 64,
         "interleaved": False, "page": 64, "layout": "NHD", "dtype": "bf16", "far": 1000000},
        # fp32, an odd token count, neighbouring pairs rotated
        {"name": "norm_rope_f32", "op": "norm_rope", "tokens": 997, "hq": 8, "hkv": 8, "dim": 64, "rope": 64,
         "interleaved": True, "page": 16, "layout": "HND", "dtype": "f32", "far": 131072},
        # the smallest call: four short requests, one token each, fp32
        {"name": "chunk_decode_f32", "op": "chunk", "batch": 4, "new_min": 1, "new_max": 1, "kv_min": 17,
         "kv_max": 255, "hq": 8, "hkv": 8, "dim": 64, "page": 16, "layout": "HND", "dtype": "f32", "window": -1,
         "lens": 1},
        # verification of a few drafted tokens for 32 requests
        {"name": "chunk_verify", "op": "chunk", "batch": 32, "new_min": 2, "new_max": 8, "kv_min": 512,
         "kv_max": 4096, "hq": 32, "hkv": 8, "dim": 128, "page": 16, "layout": "HND", "dtype": "bf16", "window": -1,
         "lens": 2},
        # the last chunk of one long prompt
        {"name": "chunk_long", "op": "chunk", "batch": 1, "new_min": 500, "new_max": 500, "kv_min": 32700,
         "kv_max": 32700, "hq": 32, "hkv": 8, "dim": 128, "page": 16, "layout": "HND", "dtype": "bf16", "window": -1,
         "lens": 3},
        # chunks of a local-attention layer, ragged, token-major pages
        {"name": "chunk_window", "op": "chunk", "batch": 8, "new_min": 300, "new_max": 1100, "kv_min": 1100,
         "kv_max": 9000, "hq": 16, "hkv": 4, "dim": 64, "page": 32, "layout": "NHD", "dtype": "bf16", "window": 1023,
         "lens": 4},
        # compute-bound chunked prefill of four requests
        {"name": "chunk_large", "op": "chunk", "batch": 4, "new_min": 2048, "new_max": 2048, "kv_min": 14000,
         "kv_max": 16384, "hq": 32, "hkv": 8, "dim": 128, "page": 16, "layout": "HND", "dtype": "bf16", "window": -1,
         "lens": 5},
    ]


def _spread(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["tables", "norm_rope", "norm_rope", "chunk", "chunk", "chunk"])
    if op == "tables":
        batch = _spread(rng, 1, 1000)
        top = _spread(rng, 16, 32768)
        prefills = rng.randint(0, min(batch, 64)) if rng.random() < 0.6 else 0
        return {"op": op, "batch": batch, "page": rng.choice([8, 16, 24, 32, 64, 128]),
                "cached_min": rng.randint(0, top // 2), "cached_max": top, "new_min": 1,
                "new_max": rng.randint(1, 7), "prefills": prefills,
                "prefill": _spread(rng, 2, 1000), "pad": rng.choice([0, 0, rng.randint(1, 300)]),
                "lens": rng.randrange(1 << 30)}
    if op == "norm_rope":
        dim = rng.choice([64, 128])
        hq, hkv = rng.choice([(8, 8), (16, 4), (28, 4), (32, 8), (40, 40), (40, 8)])
        dtype = rng.choice(["bf16", "bf16", "f32"])
        top = 16384 * 48 * 128 * 2 // ((hq + 2 * hkv) * dim * (2 if dtype == "bf16" else 4))
        return {"op": op, "tokens": _spread(rng, 1, top), "hq": hq, "hkv": hkv, "dim": dim,
                "rope": rng.choice([dim, dim, dim // 2, dim // 4]), "interleaved": rng.random() < 0.4,
                "page": rng.choice([8, 16, 24, 32, 64, 128]), "layout": rng.choice(["HND", "NHD"]), "dtype": dtype,
                "far": _spread(rng, 512, 1000000)}
    hq, hkv = rng.choice([(8, 8), (16, 4), (28, 4), (32, 8), (40, 8), (16, 16)])
    dim = rng.choice([64, 128, 128])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    most = 1e12 if dtype == "bf16" else 1e11
    while True:
        batch = _spread(rng, 1, 64)
        new = _spread(rng, 1, 2048)
        kv = _spread(rng, max(16, new), 32768)
        window = rng.choice([-1, -1, _spread(rng, 16, 4096) - 1])
        if batch * new * kv * hq * dim * 4 <= most and batch * new * kv * hq <= 2e9 and batch * kv * hkv * dim <= 5e8:
            break
    return {"op": op, "batch": batch, "new_min": max(1, new // 3), "new_max": new,
            "kv_min": max(new, kv // 4), "kv_max": kv, "hq": hq, "hkv": hkv, "dim": dim,
            "page": rng.choice([16, 16, 32, 64, 128, 24 if dtype == "f32" else 16]),
            "layout": rng.choice(["HND", "NHD"]), "dtype": dtype, "window": window, "lens": rng.randrange(1 << 30)}


def _table_lens(case):
    """(cached, new) of every request of a `tables` case."""
    r = random.Random(case["lens"])
    cached = [r.randint(case["cached_min"], case["cached_max"]) for _ in range(case["batch"])]
    new = [r.randint(case["new_min"], case["new_max"]) for _ in range(case["batch"])]
    for i in r.sample(range(case["batch"]), case["prefills"]):
        cached[i], new[i] = cached[i] // 2, case["prefill"]
    return cached, new


def _chunk_lens(case):
    """(new tokens, cached tokens with them) of every request of a `chunk` case."""
    r = random.Random(case["lens"])
    new = [r.randint(case["new_min"], case["new_max"]) for _ in range(case["batch"])]
    kv = [max(n, r.randint(case["kv_min"], case["kv_max"])) for n in new]
    return new, kv


def _pages(n, page):
    return -(-n // page)


def work(case):
    if case["op"] == "tables":
        cached, new = _table_lens(case)
        old = sum(_pages(c, case["page"]) for c in cached)
        tot = sum(_pages(c + n, case["page"]) for c, n in zip(cached, new))
        need, rows, b = tot - old, sum(new) + case["pad"], case["batch"]
        # lengths and rows, pages held, pages taken; indptrs and lengths, page list, new table entries, positions, slots
        return {"bytes": 4 * (6 * b + 4 + old + tot + 2 * need) + 12 * rows, "flops": 2 * (rows + tot)}
    es = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "norm_rope":
        t, rows, d = case["tokens"], case["hq"] + 2 * case["hkv"], case["dim"]
        n = t * (case["hq"] + case["hkv"])
        return {"bytes": 2 * t * rows * d * es + 12 * t + 2 * d * es + 2 * case["rope"],
                "flops": n * (4 * d + 3 * case["rope"])}
    new, kv = _chunk_lens(case)
    w, pairs, keys = case["window"], 0, 0
    for n, m in zip(new, kv):
        last = range(m - n, m)  # positions of the new tokens
        pairs += sum(min(p, w) + 1 if w >= 0 else p + 1 for p in last)
        keys += min(m, n + w) if w >= 0 else m
    rows = sum(new) * case["hq"]
    pages = sum(_pages(m, case["page"]) for m in kv)
    return {"bytes": 2 * rows * case["dim"] * es + 4 * rows + 2 * keys * case["hkv"] * case["dim"] * es
            + 4 * (3 * case["batch"] + 2 + pages), "flops": 4 * pairs * case["hq"] * case["dim"]}


# ----------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _normal(shape, dtype, gen):
    return torch.randn(shape, device="cuda", dtype=torch.float32, generator=gen).to(dtype)


def prepare(case, seed):
    return {"tables": _prepare_tables, "norm_rope": _prepare_norm_rope, "chunk": _prepare_chunk}[case["op"]](case, seed)


def _prepare_tables(case, seed):
    """Lengths, the block table with the pages already held, and the list of free pages."""
    gen = _gen(seed)
    cached, new = _table_lens(case)
    P, B = case["page"], case["batch"]
    old = [_pages(c, P) for c in cached]
    tot = [_pages(c + n, P) for c, n in zip(cached, new)]
    rows, cols = B + B // 4 + 1, max(tot) + 3
    num_pages = sum(tot) + 57
    ids = torch.randperm(num_pages, generator=gen, device="cuda").to(torch.int32)
    row_of = torch.randperm(rows, generator=gen, device="cuda")[:B].to(torch.int32)
    held = torch.arange(cols, device="cuda")[None, :] < torch.tensor(old, device="cuda")[:, None]
    table = torch.full((rows, cols), -1, dtype=torch.int32, device="cuda")
    part = torch.full((B, cols), -1, dtype=torch.int32, device="cuda")
    part[held] = ids[:sum(old)]
    table[row_of.long()] = part
    free = ids[sum(old):].contiguous()
    nnz, total = sum(tot), sum(new) + case["pad"]
    empty = lambda n, t=torch.int32: torch.empty(n, dtype=t, device="cuda")  # noqa: E731
    out = (empty(B + 1), empty(B), empty(B + 1), empty(nnz), empty(total), empty(total, torch.int64))
    return {"case": case, "cached": _i32(cached), "new": _i32(new), "rows": row_of, "table": table, "free": free,
            "free_count": _i32([free.numel()]), "free_left": _i32([0]), "num_pages": num_pages, "nnz": nnz,
            "total": total, "out": out}


def _prepare_norm_rope(case, seed):
    """The fused projection's rows, norm weights, rotation frequencies, positions, slots and pools."""
    gen = _gen(seed)
    dt, d, t = DTYPES[case["dtype"]], case["dim"], case["tokens"]
    hq, hkv, P = case["hq"], case["hkv"], case["page"]
    qkv = _normal((t, (hq + 2 * hkv) * d), dt, gen)
    w = lambda: (1 + 0.2 * torch.randn(d, device="cuda", generator=gen)).to(dt)  # noqa: E731
    half = case["rope"] // 2
    inv_freq = (10000.0 ** (-torch.arange(half, device="cuda", dtype=torch.float64) / half)).float()
    num_pages = _pages(t, P) + 33
    slots = torch.randperm(num_pages * P, generator=gen, device="cuda")[:t].contiguous()
    positions = torch.randint(0, case["far"], (t,), generator=gen, device="cuda", dtype=torch.int32)
    shape = (num_pages, hkv, P, d) if case["layout"] == "HND" else (num_pages, P, hkv, d)
    q, k, v = (x.view(t, -1, d) for x in qkv.split([hq * d, hkv * d, hkv * d], 1))
    return {"case": case, "q": q, "k": k, "v": v, "q_weight": w(), "k_weight": w(), "inv_freq": inv_freq,
            "positions": positions, "slots": slots, "k_pool": torch.zeros(shape, dtype=dt, device="cuda"),
            "v_pool": torch.zeros(shape, dtype=dt, device="cuda"), "eps": 1e-6,
            "q_out": torch.empty((t, hq, d), dtype=dt, device="cuda")}


def _prepare_chunk(case, seed):
    """Queries, pools with the new tokens already in them, the page table, outputs and a workspace."""
    gen = _gen(seed)
    dt, d, P = DTYPES[case["dtype"]], case["dim"], case["page"]
    new, kv = _chunk_lens(case)
    pages = [_pages(m, P) for m in kv]
    num_pages = sum(pages) + 3
    ids = torch.randperm(num_pages, generator=gen, device="cuda")[:sum(pages)].to(torch.int32)
    shape = (num_pages, case["hkv"], P, d) if case["layout"] == "HND" else (num_pages, P, case["hkv"], d)
    csum = lambda x: [sum(x[:i]) for i in range(len(x) + 1)]  # noqa: E731
    total = sum(new)
    return {"case": case, "q": _normal((total, case["hq"], d), dt, gen), "k_pool": _normal(shape, dt, gen),
            "v_pool": _normal(shape, dt, gen), "qo_indptr": _i32(csum(new)), "kv_len": _i32(kv),
            "page_indptr": _i32(csum(pages)), "page_indices": ids, "max_new": max(new), "max_kv": max(kv),
            "o": torch.empty((total, case["hq"], d), dtype=dt, device="cuda"),
            "lse": torch.empty((total, case["hq"]), dtype=torch.float32, device="cuda"),
            "workspace": torch.empty(96 << 20, dtype=torch.uint8, device="cuda")}


# --------------------------------------------------------------- one pass
def run(state):
    op = state["case"]["op"]
    if own:
        import decode_ragged_paged_gb300 as pd
        if op == "tables":
            t = pd.pd_batch_tables(state["new"], state["cached"], state["table"], page_size=state["case"]["page"],
                                   num_pages=state["num_pages"], total_qo=state["total"],
                                   max_page_indices=state["nnz"], rows=state["rows"], free_pages=state["free"],
                                   free_count=state["free_count"], free_count_out=state["free_left"],
                                   out=state["out"])
            return {"qo_indptr": t[0], "kv_len": t[1], "page_indptr": t[2], "page_indices": t[3], "positions": t[4],
                    "slot_map": t[5], "table": state["table"], "free_left": state["free_left"]}
        if op == "norm_rope":
            q = pd.pd_qk_norm_rope_append(state["q"], state["k"], state["v"], state["q_weight"], state["k_weight"],
                                          state["inv_freq"], state["positions"], state["slots"], state["k_pool"],
                                          state["v_pool"], eps=state["eps"], interleaved=state["case"]["interleaved"],
                                          q_out=state["q_out"], layout=state["case"]["layout"])
            return {"q": q, "k_pool": state["k_pool"], "v_pool": state["v_pool"]}
        o, lse = pd.pd_attn_chunk(state["q"], state["k_pool"], state["v_pool"], state["kv_len"], state["page_indptr"],
                                  state["page_indices"], state["qo_indptr"], window_left=state["case"]["window"],
                                  max_qo_len=state["max_new"], max_kv_len=state["max_kv"], o=state["o"],
                                  lse=state["lse"], workspace=state["workspace"], layout=state["case"]["layout"])
        return {"o": o, "lse": lse}
    return {"tables": _plain_tables, "norm_rope": _plain_norm_rope, "chunk": _plain_chunk}[op](state)


def _indptr(n):
    return torch.cat([n.new_zeros(1), n.cumsum(0)])


def _plain_tables(s):
    P = s["case"]["page"]
    rows = s["rows"].long()
    cached, new = s["cached"].long(), s["new"].long()
    kv = cached + new
    old, tot = (cached + P - 1) // P, (kv + P - 1) // P
    need, qo, pp = _indptr(tot - old), _indptr(new), _indptr(tot)
    # every page of the batch: its request, its place there, and the free page it takes if it is new
    at = torch.arange(s["nnz"], device="cuda")
    r = torch.searchsorted(pp, at, right=True) - 1
    j = at - pp[r]
    fresh = j >= old[r]
    took = s["free"][(s["free_count"].long() - 1 - (need[r] + j - old[r])).clamp(0, s["free"].numel() - 1)]
    s["table"][rows[r], j] = torch.where(fresh, took, s["table"][rows[r], j])
    page_indices = s["table"][rows[r], j]
    # every row of the batch: its request, position and slot; padding rows have slot -1
    at = torch.arange(s["total"], device="cuda")
    r = torch.searchsorted(qo, at, right=True) - 1
    real = r < new.numel()
    r = r.clamp(max=new.numel() - 1)
    pos = torch.where(real, cached[r] + at - qo[r], torch.zeros_like(at))
    slot = torch.where(real, s["table"][rows[r], pos // P].long() * P + pos % P, torch.full_like(at, -1))
    left = s["free_count"] - need[-1:].to(torch.int32)
    return {"qo_indptr": qo.to(torch.int32), "kv_len": kv.to(torch.int32), "page_indptr": pp.to(torch.int32),
            "page_indices": page_indices, "positions": pos.to(torch.int32), "slot_map": slot, "table": s["table"],
            "free_left": left}


def _plain_rotate(x, cos, sin, rope, interleaved):
    a, b = (x[..., 0:rope:2], x[..., 1:rope:2]) if interleaved else (x[..., :rope // 2], x[..., rope // 2:rope])
    y = torch.stack([a * cos - b * sin, a * sin + b * cos], -1 if interleaved else -2).flatten(-2)
    return torch.cat([y, x[..., rope:]], -1)


def _plain_norm_rope(s):
    c = s["case"]
    t = s["positions"].double()[:, None] * s["inv_freq"].double()[None, :]  # far positions: angles in 64 bits
    cos, sin = t.cos().float()[:, None, :], t.sin().float()[:, None, :]

    def head(x, w):
        x = x.float()
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + s["eps"]) * w.float()
        return _plain_rotate(x, cos, sin, c["rope"], c["interleaved"])

    q, k = head(s["q"], s["q_weight"]), head(s["k"], s["k_weight"])
    page, slot = s["slots"] // c["page"], s["slots"] % c["page"]
    if c["layout"] == "HND":
        s["k_pool"][page, :, slot] = k.to(s["k_pool"].dtype)
        s["v_pool"][page, :, slot] = s["v"]
    else:
        s["k_pool"][page, slot] = k.to(s["k_pool"].dtype)
        s["v_pool"][page, slot] = s["v"]
    s["q_out"].copy_(q)
    return {"q": s["q_out"], "k_pool": s["k_pool"], "v_pool": s["v_pool"]}


def _plain_chunk(s):
    c = s["case"]
    B, P, d, hkv = c["batch"], c["page"], c["dim"], c["hkv"]
    g = c["hq"] // hkv
    n = (s["qo_indptr"][1:] - s["qo_indptr"][:-1]).long()
    kv = s["kv_len"].long()
    # the batch padded to its longest chunk and cache
    i = torch.arange(s["max_new"], device="cuda")
    j = torch.arange(s["max_kv"], device="cuda")
    row = (s["qo_indptr"][:-1].long()[:, None] + i).clamp(max=s["q"].shape[0] - 1)
    page = s["page_indices"][(s["page_indptr"][:-1].long()[:, None] + j // P).clamp(max=s["page_indices"].numel() - 1)]
    page, slot = page.long(), (j % P).expand(B, -1)

    def keys(pool):  # [B, Hkv, keys, D]
        x = pool[page, :, slot] if c["layout"] == "HND" else pool[page, slot]
        return x.float().transpose(1, 2)

    q = s["q"][row].float().reshape(B, s["max_new"], hkv, g, d).permute(0, 2, 3, 1, 4).reshape(B, hkv, -1, d)
    x = (q @ keys(s["k_pool"]).transpose(2, 3)).mul_(d ** -0.5).view(B, hkv, g, s["max_new"], -1)
    at = kv[:, None] - n[:, None] + i  # position of each row
    seen = (j < kv[:, None, None]) & (j <= at[:, :, None])
    if c["window"] >= 0:
        seen &= j >= at[:, :, None] - c["window"]
    x.masked_fill_(~seen[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = x.sub_(m).exp_()
    l = p.sum(-1, keepdim=True)
    o = (p.view(B, hkv, -1, s["max_kv"]) @ keys(s["v_pool"])).view(B, hkv, g, s["max_new"], d) / l
    lse = (m + l.log()).squeeze(-1)
    real = i < n[:, None]
    o = o.permute(0, 3, 1, 2, 4).reshape(B, s["max_new"], c["hq"], d)[real]
    lse = lse.permute(0, 3, 1, 2).reshape(B, s["max_new"], c["hq"])[real]
    return {"o": o.to(s["q"].dtype), "lse": lse}


# ---------------------------------------------------------------- 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "tables":
        return None
    if case["op"] == "norm_rope":
        return _exact_norm_rope(s)
    return _exact_chunk(s)


def _exact_norm_rope(s):
    c = s["case"]
    half = c["rope"] // 2
    angle = torch.outer(s["positions"].double(), s["inv_freq"].double())
    turn = torch.polar(torch.ones_like(angle), angle)[:, None, :]

    def head(x, w):
        x = x.double()
        x = x / ((x ** 2).sum(-1, keepdim=True) / c["dim"] + s["eps"]).sqrt() * w.double()
        y = x.clone()
        first = slice(0, c["rope"], 2) if c["interleaved"] else slice(0, half)
        second = slice(1, c["rope"], 2) if c["interleaved"] else slice(half, c["rope"])
        z = torch.complex(x[..., first], x[..., second]) * turn
        y[..., first], y[..., second] = z.real, z.imag
        return y

    pools = []
    for x in (head(s["k"], s["k_weight"]), s["v"].double()):
        pool = torch.zeros(s["k_pool"].shape, dtype=torch.float64, device="cuda")
        view = pool if c["layout"] == "NHD" else pool.transpose(1, 2)
        view[torch.div(s["slots"], c["page"], rounding_mode="floor"), s["slots"].remainder(c["page"])] = x
        pools.append(pool)
    return {"q": head(s["q"], s["q_weight"]), "k_pool": pools[0], "v_pool": pools[1]}


def _exact_chunk(s):
    c = s["case"]
    new, kv = _chunk_lens(c)
    P, g = c["page"], c["hq"] // c["hkv"]
    o = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(s["q"].shape[:2], dtype=torch.float64, device="cuda")
    if work(c)["flops"] > 4e12:
        return None
    row = page = 0
    for n, m in zip(new, kv):
        ids = s["page_indices"][page:page + _pages(m, P)].long()
        page += _pages(m, P)
        at = torch.arange(m - n, m, device="cuda")[:, None]
        j = torch.arange(m, device="cuda")[None, :]
        hidden = j > at
        if c["window"] >= 0:
            hidden = hidden | (at - j > c["window"])
        for h in range(c["hkv"]):
            kk, vv = (pool[ids][:, h] if c["layout"] == "HND" else pool[ids][:, :, h] for pool in
                      (s["k_pool"], s["v_pool"]))
            kk, vv = (x.reshape(-1, c["dim"])[:m].double() for x in (kk, vv))
            for e in range(h * g, h * g + g):
                x = s["q"][row:row + n, e].double() @ kk.T / math.sqrt(c["dim"])
                x[hidden] = -math.inf
                lse[row:row + n, e] = torch.logsumexp(x, -1)
                o[row:row + n, e] = torch.softmax(x, -1) @ vv
        row += n
    return {"o": o, "lse": lse}
