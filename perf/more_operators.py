"""What is measured of the operators around an 8-bit cache: their cases, inputs, plain forms and 64-bit values.

Three operators of a serving step whose paged KV cache is held in 8 bits, or whose positions have several axes:

  axes    per-head RMS norms, rotation by positions with several axes (time, height, width: each frequency
          turns by one of them), q written out, k and v into their pages
  append  new keys and values rounded to e4m3 into their pages, with a scale for each block of tokens and head
  chunk   attention of each request's new tokens, one to thousands, over such a cache

Every case is a dict of plain values; the request lengths of a case follow from its `lens` seed, the
values (and page orders) from the seed given to `prepare`.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
E4M3 = torch.float8_e4m3fn
TOP = 448.0  # e4m3's largest value


# ------------------------------------------------------------------ cases
def listed():
    return [
        # a decode step of a model that takes images: 128 requests, one text token each, where the call's latency counts
        {"name": "axes_decode", "op": "axes", "tokens": 128, "hq": 32, "hkv": 8, "dim": 128, "rope": 128, "t": 16,
         "h": 24, "mixed": False, "page": 16, "layout": "HND", "dtype": "bf16", "far": 4096},
        # prompts with images, an odd number of tokens
        {"name": "axes_images", "op": "axes", "tokens": 4099, "hq": 28, "hkv": 4, "dim": 128, "rope": 128, "t": 16,
         "h": 24, "mixed": False, "page": 16, "layout": "HND", "dtype": "bf16", "far": 8192},
        # a long video: far times, the axes' frequencies taking turns, token-major pages
        {"name": "axes_video", "op": "axes", "tokens": 16384, "hq": 32, "hkv": 8, "dim": 128, "rope": 128, "t": 24,
         "h": 20, "mixed": True, "page": 64, "layout": "NHD", "dtype": "bf16", "far": 200000},
        # a decode step: 128 requests, one new token each
        {"name": "append_decode", "op": "append", "batch": 128, "new_min": 1, "new_max": 1, "kv_min": 512,
         "kv_max": 4096, "hkv": 8, "dim": 128, "page": 16, "block": 16, "layout": "HND", "dtype": "bf16", "lens": 11},
        # prefills of 8 x 512 tokens, 40 heads
        {"name": "append_prefill", "op": "append", "batch": 8, "new_min": 512, "new_max": 512, "kv_min": 512,
         "kv_max": 512, "hkv": 40, "dim": 128, "page": 16, "block": 16, "layout": "HND", "dtype": "bf16", "lens": 12},
        # ragged fp32 chunks into token-major pages with two blocks each
        {"name": "append_ragged", "op": "append", "batch": 24, "new_min": 37, "new_max": 700, "kv_min": 700,
         "kv_max": 3000, "hkv": 8, "dim": 64, "page": 64, "block": 32, "layout": "NHD", "dtype": "f32", "lens": 13},
        # the smallest attention: four short requests, one token each
        {"name": "chunk_short", "op": "chunk", "batch": 4, "new_min": 1, "new_max": 1, "kv_min": 17, "kv_max": 255,
         "hq": 8, "hkv": 8, "dim": 64, "page": 16, "block": 16, "layout": "HND", "window": -1, "lens": 1},
        # a decode step of 128 requests
        {"name": "chunk_decode", "op": "chunk", "batch": 128, "new_min": 1, "new_max": 1, "kv_min": 512, "kv_max": 4096,
         "hq": 32, "hkv": 8, "dim": 128, "page": 16, "block": 16, "layout": "HND", "window": -1, "lens": 2},
        # verification of a few drafted tokens for 32 requests
        {"name": "chunk_verify", "op": "chunk", "batch": 32, "new_min": 2, "new_max": 8, "kv_min": 512, "kv_max": 4096,
         "hq": 32, "hkv": 8, "dim": 128, "page": 16, "block": 16, "layout": "HND", "window": -1, "lens": 2},
        # the last chunk of one long prompt
        {"name": "chunk_long", "op": "chunk", "batch": 1, "new_min": 500, "new_max": 500, "kv_min": 32700,
         "kv_max": 32700, "hq": 32, "hkv": 8, "dim": 128, "page": 16, "block": 16, "layout": "HND", "window": -1,
         "lens": 3},
        # chunks of a local-attention layer, ragged, token-major pages of 64 with two blocks each
        {"name": "chunk_window", "op": "chunk", "batch": 8, "new_min": 300, "new_max": 1100, "kv_min": 1100,
         "kv_max": 9000, "hq": 16, "hkv": 4, "dim": 64, "page": 64, "block": 32, "layout": "NHD", "window": 1023,
         "lens": 4},
        # compute-bound chunked prefill of four requests
        {"name": "chunk_large", "op": "chunk", "batch": 4, "new_min": 2048, "new_max": 2048, "kv_min": 14000,
         "kv_max": 16384, "hq": 32, "hkv": 8, "dim": 128, "page": 16, "block": 16, "layout": "HND", "window": -1,
         "lens": 5},
    ]


def _spread(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["axes", "append", "chunk", "chunk"])
    page = rng.choice([8, 16, 16, 24, 32, 64, 128])
    block = rng.choice([b for b in (8, 16, 32, 64, page) if page % b == 0])
    layout = rng.choice(["HND", "NHD"])
    if op == "axes":
        dim = rng.choice([64, 128])
        hq, hkv = rng.choice([(8, 8), (16, 4), (28, 4), (32, 8), (40, 8)])
        dtype = rng.choice(["bf16", "bf16", "f32"])
        rope = rng.choice([dim, dim, dim // 2])
        t = rng.randint(0, rope // 4)
        top = 16384 * 48 * 128 * 2 // ((hq + 2 * hkv) * dim * (2 if dtype == "bf16" else 4))
        return {"op": op, "tokens": _spread(rng, 1, top), "hq": hq, "hkv": hkv, "dim": dim, "rope": rope, "t": t,
                "h": rng.randint(0, rope // 2 - t), "mixed": rng.random() < 0.4, "page": page, "layout": layout,
                "dtype": dtype, "far": _spread(rng, 512, 200000)}
    if op == "append":
        dim, hkv = rng.choice([64, 128]), rng.choice([1, 4, 8, 8, 40])
        dtype = rng.choice(["bf16", "bf16", "f32"])
        while True:
            batch, new, kv = _spread(rng, 1, 256), _spread(rng, 1, 4096), _spread(rng, 16, 8192)
            kv = max(new, kv)
            if batch * new * hkv * dim <= 2e7 and batch * kv * hkv * dim <= 5e8:
                break
        return {"op": op, "batch": batch, "new_min": rng.randint(max(1, new // 3), new), "new_max": new,
                "kv_min": rng.randint(new, kv), "kv_max": kv, "hkv": hkv, "dim": dim, "page": page, "block": block,
                "layout": layout, "dtype": dtype, "lens": rng.randrange(1 << 30)}
    hq, hkv = rng.choice([(8, 8), (16, 4), (28, 4), (32, 8), (40, 8), (16, 16)])
    dim = rng.choice([64, 128, 128])
    while True:
        batch, new = _spread(rng, 1, 64), _spread(rng, 1, 2048)
        kv = _spread(rng, max(16, new), 32768)
        window = rng.choice([-1, -1, _spread(rng, 16, 4096) - 1])
        if batch * new * kv * hq * dim * 4 <= 1e12 and batch * new * kv * hq <= 2e9 and batch * kv * hkv * dim <= 5e8:
            break
    return {"op": op, "batch": batch, "new_min": max(1, new // 3), "new_max": new, "kv_min": max(new, kv // 4),
            "kv_max": kv, "hq": hq, "hkv": hkv, "dim": dim, "page": page, "block": block, "layout": layout,
            "window": window, "lens": rng.randrange(1 << 30)}


def _lens(case):
    """(new tokens, cached tokens with them) of every request of an `append` or `chunk` case."""
    r = random.Random(case["lens"])
    new = [r.randint(case["new_min"], case["new_max"]) for _ in range(case["batch"])]
    kv = [max(n, r.randint(case["kv_min"], case["kv_max"])) for n in new]
    return new, kv


def _freq_axis(case):
    """The axis of each frequency: the first t turn with time, h with height, the rest with width; or taking turns."""
    t, h, n = case["t"], case["h"], case["rope"] // 2
    w = n - t - h
    if not case["mixed"]:
        return bytes([0] * t + [1] * h + [2] * w)
    left, axes = [t, h, w], []
    while len(axes) < n:
        for a in range(3):
            if left[a]:
                left[a] -= 1
                axes.append(a)
    return bytes(axes)


def _pages(n, page):
    return -(-n // page)


def work(case):
    es = 2 if case.get("dtype", "bf16") == "bf16" else 4
    if case["op"] == "axes":
        t, rows, d = case["tokens"], case["hq"] + 2 * case["hkv"], case["dim"]
        n = t * (case["hq"] + case["hkv"])
        # rows read and written, three positions and a slot of each token, weights, frequencies
        return {"bytes": 2 * t * rows * d * es + 20 * t + 2 * d * es + 2 * case["rope"],
                "flops": n * (4 * d + 3 * case["rope"])}
    new, kv = _lens(case)
    if case["op"] == "append":
        values = 2 * sum(new) * case["hkv"] * case["dim"]
        S = case["block"]
        blocks = sum(_pages(m, S) - (m - n) // S for n, m in zip(new, kv))
        kept = sum((m - n) % S != 0 for n, m in zip(new, kv))  # blocks with earlier tokens: their scale is read
        return {"bytes": values * (es + 1) + 2 * 4 * case["hkv"] * (blocks + kept) + 4 * (3 * case["batch"] + 2 + blocks),
                "flops": 3 * values}
    w, pairs, keys, blocks = case["window"], 0, 0, 0
    for n, m in zip(new, kv):
        pairs += sum(min(p, w) + 1 if w >= 0 else p + 1 for p in range(m - n, m))
        k = min(m, n + w) if w >= 0 else m
        keys += k
        blocks += _pages(k, case["block"])
    rows = sum(new) * case["hq"]
    pages = sum(_pages(m, case["page"]) for m in kv)
    return {"bytes": 4 * rows * case["dim"] + 4 * rows + 2 * keys * case["hkv"] * case["dim"]
            + 8 * blocks * case["hkv"] + 4 * (3 * case["batch"] + 2 + pages), "flops": 4 * pairs * case["hq"] * case["dim"]}


# ----------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _normal(shape, dtype, gen):
    return torch.randn(shape, device="cuda", dtype=torch.float32, generator=gen).to(dtype)


def prepare(case, seed):
    return {"axes": _prepare_axes, "append": _prepare_append, "chunk": _prepare_chunk}[case["op"]](case, seed)


def _prepare_axes(case, seed):
    """The fused projection's rows, norm weights, frequencies and their axes, positions, slots and pools."""
    gen = _gen(seed)
    dt, d, t = DTYPES[case["dtype"]], case["dim"], case["tokens"]
    hq, hkv, P = case["hq"], case["hkv"], case["page"]
    qkv = _normal((t, (hq + 2 * hkv) * d), dt, gen)
    w = lambda: (1 + 0.2 * torch.randn(d, device="cuda", generator=gen)).to(dt)  # noqa: E731
    half = case["rope"] // 2
    inv_freq = (10000.0 ** (-torch.arange(half, device="cuda", dtype=torch.float64) / half)).float()
    num_pages = _pages(t, P) + 33
    slots = torch.randperm(num_pages * P, generator=gen, device="cuda")[:t].contiguous()
    # text (the three axes alike) and images (a time of their own, places of a grid)
    time = torch.randint(0, case["far"], (t,), generator=gen, device="cuda", dtype=torch.int32)
    place = torch.randint(0, 64, (2, t), generator=gen, device="cuda", dtype=torch.int32)
    text = torch.rand(t, generator=gen, device="cuda") < 0.3
    positions = torch.cat([time[None], torch.where(text, time, time // 2 + place)]).contiguous()
    shape = (num_pages, hkv, P, d) if case["layout"] == "HND" else (num_pages, P, hkv, d)
    q, k, v = (x.view(t, -1, d) for x in qkv.split([hq * d, hkv * d, hkv * d], 1))
    return {"case": case, "q": q, "k": k, "v": v, "q_weight": w(), "k_weight": w(), "inv_freq": inv_freq,
            "freq_axis": _freq_axis(case), "axis_of": torch.tensor(list(_freq_axis(case)), device="cuda"),
            "positions": positions, "slots": slots, "k_pool": torch.zeros(shape, dtype=dt, device="cuda"),
            "v_pool": torch.zeros(shape, dtype=dt, device="cuda"), "eps": 1e-6,
            "q_out": torch.empty((t, hq, d), dtype=dt, device="cuda")}


def _quantized_pool(case, num_pages, gen):
    """A pool of keys or values that the cache holds: e4m3 values and the scales of its blocks. Channels
    differ in size, as a model's do, and so do blocks."""
    P, S, hkv, d = case["page"], case["block"], case["hkv"], case["dim"]
    x = torch.randn((num_pages, hkv, P // S, S, d), device="cuda", generator=gen)
    x *= torch.exp(0.5 * torch.randn((hkv, 1, 1, d), device="cuda", generator=gen))
    x *= torch.exp(0.7 * torch.randn((num_pages, hkv, P // S, 1, 1), device="cuda", generator=gen))
    scale = torch.exp2(torch.ceil(torch.log2(x.abs().amax((3, 4)) / TOP)))
    x = (x / scale[..., None, None]).clamp_(-TOP, TOP).to(E4M3).view(num_pages, hkv, P, d)
    if case["layout"] == "NHD":
        x = x.view(torch.uint8).transpose(1, 2).contiguous().view(E4M3)
    return x, scale


def _prepare_pages(case, gen):
    """Lengths and page lists of a batch, in random page order, and the pools."""
    new, kv = _lens(case)
    P = case["page"]
    pages = [_pages(m, P) for m in kv]
    num_pages = sum(pages) + 3
    ids = torch.randperm(num_pages, generator=gen, device="cuda")[:sum(pages)].to(torch.int32)
    csum = lambda x: [sum(x[:i]) for i in range(len(x) + 1)]  # noqa: E731
    k_pool, k_scale = _quantized_pool(case, num_pages, gen)
    v_pool, v_scale = _quantized_pool(case, num_pages, gen)
    return {"case": case, "qo_indptr": _i32(csum(new)), "kv_len": _i32(kv), "page_indptr": _i32(csum(pages)),
            "page_indices": ids, "k_pool": k_pool, "v_pool": v_pool, "k_scale": k_scale, "v_scale": v_scale,
            "max_new": max(new), "max_kv": max(kv), "total": sum(new)}


def _prepare_append(case, seed):
    """A batch whose new tokens' keys and values are slices of a fused projection's rows."""
    gen = _gen(seed)
    s = _prepare_pages(case, gen)
    hkv, d = case["hkv"], case["dim"]
    rows = _normal((s["total"], 4 * hkv * d), DTYPES[case["dtype"]], gen)  # (two heads of queries a head of keys)
    s["k"], s["v"] = (x.view(s["total"], hkv, d) for x in rows.split([2 * hkv * d, hkv * d, hkv * d], 1)[1:])
    return s


def _prepare_chunk(case, seed):
    """Queries of a batch whose new tokens are in the pools already, outputs and a workspace."""
    gen = _gen(seed)
    s = _prepare_pages(case, gen)
    s["q"] = _normal((s["total"], case["hq"], case["dim"]), torch.bfloat16, gen)
    s["o"] = torch.empty_like(s["q"])
    s["lse"] = torch.empty((s["total"], case["hq"]), dtype=torch.float32, device="cuda")
    s["workspace"] = torch.empty(96 << 20, dtype=torch.uint8, device="cuda")
    return s


# --------------------------------------------------------------- one pass
def run(state):
    op = state["case"]["op"]
    if own:
        import decode_ragged_paged_gb300 as pd
        layout = state["case"]["layout"]
        if op == "axes":
            q = pd.pd_qk_norm_rope_axes_append(state["q"], state["k"], state["v"], state["q_weight"],
                                               state["k_weight"], state["inv_freq"], state["freq_axis"],
                                               state["positions"], state["slots"], state["k_pool"], state["v_pool"],
                                               eps=state["eps"], q_out=state["q_out"], layout=layout)
            return {"q": q, "k_pool": state["k_pool"], "v_pool": state["v_pool"]}
        if op == "append":
            pd.pd_kv_append_quant(state["k"], state["v"], state["k_pool"], state["v_pool"], state["k_scale"],
                                  state["v_scale"], state["qo_indptr"], state["kv_len"], state["page_indptr"],
                                  state["page_indices"], max_kv_len=state["max_kv"], layout=layout)
            return {n: state[n] for n in ("k_pool", "v_pool", "k_scale", "v_scale")}
        o, lse = pd.pd_attn_chunk_quant(state["q"], state["k_pool"], state["v_pool"], state["k_scale"],
                                        state["v_scale"], state["kv_len"], state["page_indptr"],
                                        state["page_indices"], state["qo_indptr"],
                                        window_left=state["case"]["window"], max_qo_len=state["max_new"],
                                        max_kv_len=state["max_kv"], o=state["o"], lse=state["lse"],
                                        workspace=state["workspace"], layout=layout)
        return {"o": o, "lse": lse}
    return {"axes": _plain_axes, "append": _plain_append, "chunk": _plain_chunk}[op](state)


def _plain_axes(s):
    c = s["case"]
    half = c["rope"] // 2
    at = s["positions"].double()[s["axis_of"]].T  # [tokens][frequencies]
    angle = at * s["inv_freq"].double()  # far positions: angles in 64 bits
    cos, sin = angle.cos().float()[:, None, :], angle.sin().float()[:, None, :]

    def head(x, w):
        x = x.float()
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + s["eps"]) * w.float()
        a, b = x[..., :half], x[..., half:2 * half]
        return torch.cat([a * cos - b * sin, a * sin + b * cos, x[..., 2 * half:]], -1)

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


def _power_for(amax):
    """The smallest power of two, at least 2^-100, that brings amax to 448 or below."""
    m, e = torch.frexp(amax)  # amax = m 2^e, m in [1/2, 1); 448 = 7/8 2^9
    return torch.ldexp(torch.ones_like(amax), torch.where(m <= 0.875, e - 9, e - 8).clamp(min=-100))


def _plain_append(s):
    c = s["case"]
    P, S, hkv, d = c["page"], c["block"], c["hkv"], c["dim"]
    n = (s["qo_indptr"][1:] - s["qo_indptr"][:-1]).long()
    have = s["kv_len"].long() - n  # tokens before the new ones
    row = torch.arange(s["total"], device="cuda")
    r = torch.searchsorted(s["qo_indptr"][1:].long(), row, right=True)
    pos = have[r] + row - s["qo_indptr"].long()[r]
    page = s["page_indices"][s["page_indptr"].long()[r] + pos // P].long()
    slot = pos % P
    block = page * (P // S) + slot // S
    # the blocks in which a request goes on: the place of their first new token, 0 if it has none before it
    going = have % S
    first_page = s["page_indices"][s["page_indptr"].long()[:-1] + (have // P).clamp(max=_pages(s["max_kv"], P) - 1)
                                   .minimum((s["page_indptr"][1:] - s["page_indptr"][:-1]).long() - 1)].long()
    first = first_page * (P // S) + have % P // S

    def store(x, pool, scale):
        x = x.float()
        rows = scale.transpose(1, 2).reshape(-1, hkv).clone()  # [block][head]
        amax = torch.zeros_like(rows).index_reduce_(0, block, x.abs().amax(-1), "amax")
        want = _power_for(amax)
        # a block that goes on keeps its scale or gets a larger one, its earlier values rounded again
        goes = torch.zeros(rows.shape[0], dtype=torch.bool, device="cuda")
        goes[first] = going > 0
        want = torch.where(goes[:, None], want.maximum(rows), want)
        touched = torch.zeros_like(goes)
        touched[block] = True
        held = pool.view(torch.uint8) if c["layout"] == "HND" else pool.view(torch.uint8).transpose(1, 2)
        place = first % (P // S) * S + torch.arange(S, device="cuda")[:, None]  # [S][request]
        place = place.T
        old = held[first_page[:, None], :, place]  # [request][S][head][dim]
        again = old.view(E4M3).float() * (rows[first] / want[first])[:, None, :, None]
        earlier = (torch.arange(S, device="cuda") < going[:, None])[:, :, None, None]
        keep = torch.where(earlier, again.to(E4M3).view(torch.uint8), old)
        held[first_page[:, None], :, place] = keep
        held[page, :, slot] = (x / want[block][:, :, None]).to(E4M3).view(torch.uint8)
        rows = torch.where(touched[:, None], want, rows)
        scale.copy_(rows.view(-1, P // S, hkv).transpose(1, 2))

    store(s["k"], s["k_pool"], s["k_scale"])
    store(s["v"], s["v_pool"], s["v_scale"])
    return {name: s[name] for name in ("k_pool", "v_pool", "k_scale", "v_scale")}


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

    def keys(pool, scale):  # [B, Hkv, keys, D]
        pool = pool.view(torch.uint8)
        x = (pool[page, :, slot] if c["layout"] == "HND" else pool[page, slot]).view(E4M3).float()
        return (x * scale[page, :, slot // c["block"]][..., None]).transpose(1, 2)

    q = s["q"][row].float().reshape(B, s["max_new"], hkv, g, d).permute(0, 2, 3, 1, 4).reshape(B, hkv, -1, d)
    x = (q @ keys(s["k_pool"], s["k_scale"]).transpose(2, 3)).mul_(d ** -0.5).view(B, hkv, g, s["max_new"], -1)
    at = kv[:, None] - n[:, None] + i  # position of each row
    seen = (j < kv[:, None, None]) & (j <= at[:, :, None])
    if c["window"] >= 0:
        seen &= j >= at[:, :, None] - c["window"]
    x.masked_fill_(~seen[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = x.sub_(m).exp_()
    l = p.sum(-1, keepdim=True)
    o = (p.view(B, hkv, -1, s["max_kv"]) @ keys(s["v_pool"], s["v_scale"])).view(B, hkv, g, s["max_new"], d) / l
    lse = (m + l.log()).squeeze(-1)
    real = i < n[:, None]
    o = o.permute(0, 3, 1, 2, 4).reshape(B, s["max_new"], c["hq"], d)[real]
    lse = lse.permute(0, 3, 1, 2).reshape(B, s["max_new"], c["hq"])[real]
    return {"o": o.to(s["q"].dtype), "lse": lse}


# ---------------------------------------------------------------- 64 bits
def exact(case, seed):
    if case["op"] == "chunk" and work(case)["flops"] > 4e12:
        return None
    return {"axes": _exact_axes, "append": _exact_append, "chunk": _exact_chunk}[case["op"]](prepare(case, seed))


def _exact_axes(s):
    c = s["case"]
    half = c["rope"] // 2
    turn = torch.empty((c["tokens"], 1, half), dtype=torch.complex128, device="cuda")
    for i, axis in enumerate(s["freq_axis"]):
        angle = s["positions"][axis].double() * s["inv_freq"][i].double()
        turn[:, 0, i] = torch.polar(torch.ones_like(angle), angle)

    def head(x, w):
        x = x.double()
        y = x / ((x ** 2).sum(-1, keepdim=True) / c["dim"] + s["eps"]).sqrt() * w.double()
        z = torch.complex(y[..., :half].contiguous(), y[..., half:2 * half].contiguous()) * turn
        y[..., :half], y[..., half:2 * half] = z.real, z.imag
        return y

    pools = []
    for x in (head(s["k"], s["k_weight"]), s["v"].double()):
        pool = torch.zeros(s["k_pool"].shape, dtype=torch.float64, device="cuda")
        view = pool if c["layout"] == "NHD" else pool.transpose(1, 2)
        view[torch.div(s["slots"], c["page"], rounding_mode="floor"), s["slots"].remainder(c["page"])] = x
        pools.append(pool)
    return {"q": head(s["q"], s["q_weight"]), "k_pool": pools[0], "v_pool": pools[1]}


def _to_e4m3(x):
    """The nearest e4m3 values (ties to even) of numbers of at most 448, in 64-bit arithmetic."""
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(x / step) * step


def _exact_append(s):
    """Request by request: all of a block's tokens, old and new, and the scale that holds them."""
    c = s["case"]
    P, S = c["page"], c["block"]
    new, kv = _lens(c)
    out = {}
    for name in ("k", "v"):
        pool, scale = s[name + "_pool"].double(), s[name + "_scale"].double()
        view = pool if c["layout"] == "HND" else pool.transpose(1, 2)  # [page][head][slot][dim]
        row = at = 0
        for n, m in zip(new, kv):
            ids = s["page_indices"][at:at + _pages(m, P)].long()
            at += _pages(m, P)
            have, lo, hi = m - n, (m - n) // S * S, _pages(m, S) * S  # whole blocks [lo, hi)
            t = torch.arange(lo, hi, device="cuda")
            pg, sl = ids[t // P], t % P
            x = torch.zeros((hi - lo, c["hkv"], c["dim"]), dtype=torch.float64, device="cuda")
            x[have - lo:m - lo] = s[name][row:row + n].double()
            row += n
            amax = x.abs().amax(-1).view(-1, S, c["hkv"]).amax(1)  # [block][head]
            need = torch.exp2(torch.ceil(torch.log2((amax / TOP).clamp(min=2.0 ** -100))))
            b_page, b_in = pg[::S], sl[::S] // S
            was = scale[b_page[0], :, b_in[0]].clone()
            if have > lo:
                need[0] = torch.maximum(need[0], was)
            codes = _to_e4m3(x / need.repeat_interleave(S, 0)[..., None])
            if have > lo:
                codes[:have - lo] = _to_e4m3(view[pg[:have - lo], :, sl[:have - lo]] * (was / need[0])[:, None])
            scale[b_page, :, b_in] = need
            view[pg[:m - lo], :, sl[:m - lo]] = codes[:m - lo]
        out[name + "_pool"], out[name + "_scale"] = pool, scale
    return out


def _exact_chunk(s):
    c = s["case"]
    new, kv = _lens(c)
    P, S, g = c["page"], c["block"], c["hq"] // c["hkv"]
    o = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(s["q"].shape[:2], dtype=torch.float64, device="cuda")
    row = page = 0
    for n, m in zip(new, kv):
        ids = s["page_indices"][page:page + _pages(m, P)].long()
        page += _pages(m, P)
        at = torch.arange(m - n, m, device="cuda")[:, None]
        j = torch.arange(m, device="cuda")[None, :]
        hidden = j > at
        if c["window"] >= 0:
            hidden = hidden | (at - j > c["window"])
        kk, vv = [], []
        for pool, scale, to in ((s["k_pool"], s["k_scale"], kk), (s["v_pool"], s["v_scale"], vv)):
            pool = pool.view(torch.uint8)[ids].view(E4M3).double()
            pool = pool if c["layout"] == "HND" else pool.transpose(1, 2)
            pool = pool * scale.double()[ids].repeat_interleave(S, 2)[..., None]
            to += [pool[:, h].reshape(-1, c["dim"])[:m] for h in range(c["hkv"])]
        for e in range(c["hq"]):
            x = s["q"][row:row + n, e].double() @ kk[e // g].T / math.sqrt(c["dim"])
            x[hidden] = -math.inf
            lse[row:row + n, e] = torch.logsumexp(x, -1)
            o[row:row + n, e] = torch.softmax(x, -1) @ vv[e // g]
        row += n
    return {"o": o, "lse": lse}
