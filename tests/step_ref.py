"""64-bit plain forms of the chunk-step operators for their GPU tests, written from the definitions
in include/pd.h: dense torch in fp64 (rotation and attention) and plain Python integers (tables)."""
import math

import torch

U = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}  # half a step, relative to the value


def ceil_div(a, b):
    return -(-a // b)


# ------------------------------------------------------------------ tables
def tables(rows, cached, new, table, free, count, *, page, num_pages, total_qo, max_page_indices, pops=True):
    """Python lists in, dict of lists out; `table` (list of rows) is changed in place."""
    cols, seen = len(table[0]), set()
    qo, kv, pp, pages, pos, slot = [0], [], [0], [], [], []
    at_rows = at_pages = at_need = 0
    left = max(0, min(count, len(free)))
    avail = left
    for r, (c, n) in enumerate(zip(cached, new)):
        row = rows[r] if rows is not None else r
        ok = n >= 0 and c >= 0 and ceil_div(c + n, page) <= cols
        if 0 <= row < len(table):
            first = row not in seen
            seen.add(row)
        else:
            first = False
        ok = ok and first
        tot = ceil_div(c + n, page) if ok else 0
        need = tot - ceil_div(c, page) if ok and pops else 0
        at_rows += max(n, 0)
        at_pages += tot
        at_need += need
        ok = ok and at_rows <= total_qo and at_pages <= max_page_indices and (need == 0 or at_need <= avail)
        if ok:
            for j in range(need):
                table[row][tot - need + j] = free[avail - 1 - (at_need - need + j)]
            left -= need
            ids = table[row][:tot]
        else:
            ids = [-1] * tot
        kv.append(c + n if ok else -1)
        pages += ids
        for i in range(max(n, 0)):
            p = c + i if ok else 0
            good = ok and 0 <= ids[p // page] < num_pages
            pos.append(p)
            slot.append(ids[p // page] * page + p % page if good else -1)
        qo.append(min(at_rows, total_qo))
        pp.append(min(at_pages, max_page_indices))
    pos, slot = pos[:total_qo], slot[:total_qo]
    pad = total_qo - len(pos)
    return {"qo_indptr": qo, "kv_len": kv, "page_indptr": pp, "page_indices": pages[:max_page_indices],
            "positions": pos + [0] * pad, "slot_map": slot + [-1] * pad, "left": left}


# --------------------------------------------------------------- norm, rope
def norm_rope(x, w, inv_freq, positions, *, eps, interleaved):
    """(values, pair sizes): x [T][H][D] any type, fp64 out; the second bounds each value's own size
    before the rotation mixed it with its partner."""
    y = x.double()
    if w is not None:
        y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + eps) * w.double()
    size = y.abs().clone()
    if inv_freq is not None:
        half = inv_freq.numel()
        t = positions.double()[:, None, None] * inv_freq.double()
        a, b = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if interleaved else (slice(0, half),
                                                                                  slice(half, 2 * half))
        ya, yb = y[..., a].clone(), y[..., b].clone()
        y[..., a] = ya * t.cos() - yb * t.sin()
        y[..., b] = ya * t.sin() + yb * t.cos()
        size[..., a] = size[..., b] = torch.hypot(ya, yb)
    return y, size


def norm_rope_bound(ref, size, dtype):
    """Largest error of a result computed in fp32 and rounded once. In units of 2^-24 of the pair's
    size: the sum of squares goes through at most 2 V + 5 <= 21 additions of which the root halves the
    relative error (11), rsqrt 4, eps and mean 2, the two products with weight and factor 3, cosine
    and sine 2 ulp each (8 over the two terms), the angle 2, two products and a sum 4: 34, taken as 40."""
    return U[dtype] * ref.abs() + 40 * 2.0 ** -24 * size


# --------------------------------------------------------------- attention
def gather(pool, ids, n, layout):
    """[n][Hkv][D] fp64 of a request's pages."""
    x = pool[ids.long()]
    if layout == "HND":
        x = x.transpose(1, 2)
    return x.reshape(-1, x.shape[2], x.shape[3])[:n].double()


def attention(q, k_pool, v_pool, qo_indptr, kv_len, page_indptr, page_indices, *, causal=True, window=-1, scale=None,
              layout="HND"):
    """(o, lse, o_bound, lse_bound) in fp64 on q's device; the index lists are Python lists. Bounds:
    of a result from exact products, fp32 sums and weights and, for bf16, weights and output rounded
    to bf16 once:
      scores are off by es <= 4 D 2^-24 max_j |s|_j, with |s| the sum of the products' sizes (the
        factor 4: a truncating adder, 2^-23 a sum, and the scaled exponent's own rounding);
      weights by es twice (own and in the sum), by 2^-21 for exp2, by 2^-8 where rounded to bf16;
      the sums over n keys by n 2^-23;
      the output by half a step."""
    T, hq, D = q.shape
    hkv = k_pool.shape[1] if layout == "HND" else k_pool.shape[2]
    g = hq // hkv
    scale = 1 / math.sqrt(D) if scale is None else scale
    dev = q.device
    o = torch.zeros(T, hq, D, dtype=torch.float64, device=dev)
    lse = torch.full((T, hq), -math.inf, dtype=torch.float64, device=dev)
    ob, lb = torch.zeros_like(o), torch.zeros_like(lse)
    rounded = 2.0 ** -8 if q.dtype == torch.bfloat16 else 0.0
    for r, n in enumerate(kv_len):
        a, b = qo_indptr[r], qo_indptr[r + 1]
        if b == a or n == 0:
            continue
        ids = page_indices[page_indptr[r]:page_indptr[r + 1]]
        pos = torch.arange(n - (b - a), n, device=dev)[:, None]
        j = torch.arange(n, device=dev)[None]
        keep = torch.ones(b - a, n, dtype=torch.bool, device=dev)
        if causal:
            keep &= j <= pos
        if window >= 0:
            keep &= j >= pos - window
        some = keep.any(-1)
        k, v = (gather(x, ids, n, layout) for x in (k_pool, v_pool))
        dead = ~keep.any(0)
        k[dead], v[dead] = 0.0, 0.0  # nothing may come of keys that no row sees
        for h in range(hq):
            qh, kh, vh = q[a:b, h].double(), k[:, h // g], v[:, h // g]
            s = (qh @ kh.T) * scale
            es = 4 * D * 2.0 ** -24 * scale * ((qh.abs() @ kh.abs().T) * keep).amax(-1, keepdim=True)
            s = s.masked_fill(~keep, -math.inf)
            m = s.amax(-1, keepdim=True)
            p = torch.exp(s - torch.where(m.isinf(), torch.zeros_like(m), m))
            p = torch.where(keep, p, torch.zeros_like(p))
            l = p.sum(-1, keepdim=True)
            p = p / torch.where(l == 0, torch.ones_like(l), l)
            o[a:b, h] = p @ vh
            rel = 2 * es + 2.0 ** -20 + n * 2.0 ** -23 + rounded
            ob[a:b, h] = rel * (p @ vh.abs())
            lse[a:b, h] = torch.where(some, (m + l.log()).squeeze(-1), lse[a:b, h])
            lb[a:b, h] = (es + 2.0 ** -20 + n * 2.0 ** -23).squeeze(-1) + 2.0 ** -21 * (1 + m.abs().squeeze(-1))
    return o, lse, ob, lb


def check_attention(o, lse, ref):
    ro, rl, ob, lb = ref
    err = (o.double() - ro).abs()
    lim = ob + U[o.dtype] * (ro.abs() + ob)
    assert torch.isfinite(o.float()).all(), "non-finite output"
    assert bool((err <= lim).all()), f"o: worst error / bound {float((err / lim.clamp(min=1e-30)).max())}"
    empty = torch.isinf(rl)
    assert torch.equal(torch.isinf(lse), empty) and bool((lse[empty] < 0).all())
    assert bool((o[empty] == 0).all())
    e = (lse.double() - rl).abs()[~empty]
    assert bool((e <= lb[~empty]).all()), f"lse: worst error {float(e.max())}"
