"""64-bit plain forms of the 8-bit cache for its GPU tests, written from the definitions in include/pd.h."""
import math

import torch

import step_ref as ref

E4M3 = torch.float8_e4m3fn


def to_e4m3(x):
    """The nearest e4m3 values (ties to even) of fp64 numbers of at most 448; NaN stays."""
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(x / step) * step


def power_for(amax):
    """The smallest power of two >= max(amax / 448, 2^-100)."""
    p = 2.0 ** -100
    while p * 448.0 < amax:
        p *= 2
    return p


def heads_first(pool, layout):
    return pool if layout == "HND" else pool.transpose(1, 2)


def append(x_new, pool, scale, qo, kv, pp, px, page, block, layout):
    """The pool's e4m3 values and the scales after the append, in fp64 (pool, scale: before it). Lists are Python's."""
    pool, scale = pool.double().clone(), scale.double().clone()
    view = heads_first(pool, layout)  # [page][head][slot][dim]
    x = x_new.double()
    heads = x.shape[1]
    for r, n in enumerate(kv):
        have = n - (qo[r + 1] - qo[r])
        t = have
        while t < n:
            end = min(n, (t // block + 1) * block)
            pg, s0, b = int(px[pp[r] + t // page]), t % page, t % page // block
            new = x[qo[r] + t - have:qo[r] + end - have]  # [tokens][head][dim]
            for h in range(heads):
                y = new[:, h]
                finite = y[torch.isfinite(y)]
                s = power_for(float(finite.abs().max()) if finite.numel() else 0.0)
                first = b * block
                if s0 > first:
                    was = float(scale[pg, h, b])
                    s = max(s, was)
                    view[pg, h, first:s0] = to_e4m3(view[pg, h, first:s0] * (was / s))
                scale[pg, h, b] = s
                view[pg, h, s0:s0 + end - t] = to_e4m3(torch.where(torch.isfinite(y), y / s, torch.full_like(y, math.nan)))
            t = end
    return pool, scale


def dequant(pool, scale, layout):
    """[pages][...] fp64 values of an 8-bit pool, in its layout (scales below 2^-100 count as that)."""
    x = heads_first(pool.view(torch.uint8).view(E4M3).double(), layout)
    block = x.shape[2] // scale.shape[2]
    x = x * scale.double().clamp(min=2.0 ** -100).repeat_interleave(block, 2)[..., None]
    return heads_first(x, layout).contiguous()


def attention(q, k_pool, v_pool, k_scale, v_scale, qo, kv, pp, px, *, causal=True, window=-1, scale=None, layout="HND"):
    """step_ref.attention over the values that the cache holds, its bounds widened by what the 8-bit cache's
    tensor-core form adds (bf16 queries):
      a query value is two e4m3 terms, off by at most half of e4m3's smallest step, 2^-10, where the row's
        largest value is over 224: 2^-17 of that, times sum |k| in a score, and twice in a weight;
      weights times their keys' scales of V are fp16 whose largest is at least 2^3 (2^2 to allow for its own
        errors): half of fp16's smallest step, 2^-25, is 2^-27 of the largest, times the sum of the e4m3 sizes."""
    k, v = dequant(k_pool, k_scale, layout), dequant(v_pool, v_scale, layout)
    kw = dict(causal=causal, window=window, scale=scale, layout=layout)
    o, lse, ob, lb = ref.attention(q, k, v, qo, kv, pp, px, **kw)
    if q.dtype != torch.bfloat16:
        return o, lse, ob, lb
    sizes = ref.attention(q, k, torch.nan_to_num(v).abs(), qo, kv, pp, px, **kw)[0]
    sm = 1 / math.sqrt(q.shape[2]) if scale is None else scale
    extra = torch.zeros(q.shape[:2], dtype=torch.float64, device=q.device)
    floor = torch.zeros_like(o)
    codes = dequant(v_pool, torch.ones_like(v_scale), layout)
    spread = dequant(torch.ones_like(v_pool, dtype=torch.float32).to(E4M3), v_scale, layout)  # every slot's scale
    g = q.shape[1] // k_scale.shape[1]
    for r, n in enumerate(kv):
        a, b = qo[r], qo[r + 1]
        if b == a or n == 0:
            continue
        ids = px[pp[r]:pp[r + 1]]
        kk, cc, bb = (torch.nan_to_num(ref.gather(x, ids, n, layout)) for x in (k, codes, spread))
        extra[a:b] = sm * 2.0 ** -17 * q[a:b].double().abs().amax(-1) * kk.abs().sum(-1).amax(0).repeat_interleave(g)
        pos = torch.arange(n - (b - a), n, device=q.device)[:, None]
        j = torch.arange(n, device=q.device)[None]
        keep = (j <= pos) if causal else torch.ones(b - a, n, dtype=torch.bool, device=q.device)
        if window >= 0:
            keep = keep & (j >= pos - window)
        for h in range(q.shape[1]):
            s = torch.nan_to_num(q[a:b, h].double() @ kk[:, h // g].T * sm).masked_fill(~keep, -math.inf)
            top = (torch.softmax(s, -1).nan_to_num() * bb[:, h // g, 0]).amax(-1)  # the largest weight times its scale
            floor[a:b, h] = 2.0 ** -27 * top[:, None] * (keep.double() @ cc[:, h // g].abs())
    rel = 2 * extra
    return o, lse, ob + rel[..., None] * sizes + floor, lb + extra
