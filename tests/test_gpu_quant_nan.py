"""pd_attn_chunk_quant where some of V's values are NaN (as pd_kv_append_quant stores what is not finite): such a
value reaches its column of the rows that see its key, and nothing of the rows that do not, whichever kernel
takes the call."""
import random

import pytest
import torch

import step_ref as ref
from test_gpu_chunk_quant import BF16, E4M3, F32, Batch

pytestmark = pytest.mark.gpu

# q's type, head dim, page, block: tensor cores (or, with few rows, the kernel for those), and the CUDA cores
TYPES = [(BF16, 128, 16, 16), (BF16, 64, 32, 8), (BF16, 128, 24, 24), (BF16, 128, 6, 3), (F32, 64, 16, 16),
         (F32, 128, 8, 8)]


def spoil(b, where):
    """NaN in V at (request, key, KV head, column); returns the outputs that have to be NaN, per mask, and the
    attention over the same values with 0 in their places."""
    clean = b.v.view(torch.uint8).clone()
    dirty = b.v.view(torch.uint8)
    for i, (r, j, h, c) in enumerate(where):
        page, slot = int(b.px[b.pp[r] + j // b.page]), j % b.page
        at = (page, h, slot, c) if b.layout == "HND" else (page, slot, h, c)
        dirty[at], clean[at] = (0x7f, 0xff)[i % 2], 0
    dirty = dirty.clone().view(E4M3)
    clean = clean.view(E4M3)
    group = b.q.shape[1] // b.ks.shape[1]

    def want(causal, window):
        bad = torch.zeros(b.q.shape, dtype=torch.bool, device="cuda")
        for r, j, h, c in where:
            a, e = b.qo[r], b.qo[r + 1]
            pos = torch.arange(b.kv[r] - (e - a), b.kv[r], device="cuda")
            sees = torch.ones_like(pos, dtype=torch.bool)
            if causal:
                sees &= j <= pos
            if window >= 0:
                sees &= j >= pos - window
            bad[a:e, h * group:(h + 1) * group, c] |= sees[:, None]
        b.v = clean
        out = b.ref(causal, window)
        b.v = dirty
        return bad, out

    return want


def check(b, want, causal=True, window=-1, **kw):
    bad, clean = want(causal, window)
    o, lse = b.run(causal=causal, window_left=window, **kw)
    assert torch.equal(torch.isnan(o), bad)
    ref.check_attention(torch.where(bad, clean[0].to(o.dtype), o), lse, clean)


def places(b, rng, window=-1, n=12):
    """Keys that some rows of a request see and others do not, and a few that all see."""
    out = []
    for r, kv in enumerate(b.kv):
        new = b.new[r]
        if kv == 0 or new == 0:
            continue
        for _ in range(n):
            lowest = max(0, kv - new - max(window, 0)) if window >= 0 else 0
            j = rng.choice([kv - 1 - rng.randrange(min(new, kv)), rng.randrange(lowest, kv),
                            min(kv - 1, lowest + rng.randrange(max(new, 1)))])
            out.append((r, j, rng.randrange(b.ks.shape[1]), rng.randrange(b.d)))
    return out


@pytest.mark.parametrize("dt,d,page,block", TYPES)
@pytest.mark.parametrize("layout", ["HND", "NHD"])
@pytest.mark.parametrize("hq,hkv,new,kv", [
    (8, 2, [2, 1, 2], [40, 64, 300]),              # few rows
    (2, 2, [8, 3], [100, 9]),                      # a head a KV head
    (8, 2, [5, 30, 1, 12], [200, 30, 77, 64]),     # one query tile
    (8, 2, [64, 200, 130], [500, 200, 1000]),      # two, and several items
    (130, 1, [3], [70]),                           # an item for each head
])
def test_a_later_tokens_nan_spoils_no_earlier_row(dt, d, page, block, layout, hq, hkv, new, kv):
    b = Batch(41, new, kv, hq, hkv, d, page, block, dt, layout)
    check(b, spoil(b, places(b, random.Random(d + page))))


@pytest.mark.parametrize("dt,d,page,block", TYPES)
@pytest.mark.parametrize("new,kv,window", [([2, 2], [300, 40], 50), ([8, 40], [100, 333], 20), ([300, 70], [700, 64], 100),
                                           ([6], [3], 1)])
def test_a_nan_behind_a_window(dt, d, page, block, new, kv, window):
    b = Batch(42, new, kv, 4, 2, d, page, block, dt)
    want = spoil(b, places(b, random.Random(window), window))
    check(b, want, window=window)
    check(b, want, causal=False, window=window)
    check(b, want, causal=False)


@pytest.mark.parametrize("dt,d,page,block", TYPES)
@pytest.mark.parametrize("new,kv", [([2], [20000]), ([6], [9000]), ([300, 2], [4000, 6000])])
@pytest.mark.parametrize("o_dtype", [BF16, F32])
def test_a_nan_in_an_item_that_is_cut(dt, d, page, block, new, kv, o_dtype):
    b = Batch(43, new, kv, 4, 1, d, page, block, dt)
    check(b, spoil(b, places(b, random.Random(kv[0]), n=6)), o_dtype=o_dtype)


@pytest.mark.parametrize("dt,d,page,block", TYPES)
def test_items_after_one_another_in_a_cta(dt, d, page, block):
    # a NaN in every other request of hundreds: what a CTA knows of one item does not reach the next
    rng = random.Random(5)
    new = [rng.choice([1, 2, 2, 7]) for _ in range(700)]
    kv = [n + rng.randrange(200) for n in new]
    b = Batch(44, new, kv, 4, 2, d, page, block, dt)
    check(b, spoil(b, [p for p in places(b, rng, n=1) if p[0] % 2]))
    b = Batch(45, [2] * 700, kv, 4, 2, d, page, block, dt)
    check(b, spoil(b, [p for p in places(b, rng, n=1) if p[0] % 2]))


@pytest.mark.parametrize("dt,d,page,block", TYPES)
@pytest.mark.parametrize("new,kv,window", [([2, 2], [300, 40], -1), ([8, 40], [100, 333], -1), ([8, 40], [100, 333], 20),
                                           ([300, 70], [700, 64], -1)])
def test_a_nan_of_k_spoils_the_rows_that_see_it(dt, d, page, block, new, kv, window):
    # in whole, their lse too, and no others
    b = Batch(46, new, kv, 4, 2, d, page, block, dt)
    rng = random.Random(d)
    want = spoil(b, [])
    bad, clean = want(True, window)
    codes = b.k.view(torch.uint8)
    for r, n in enumerate(kv):
        for j in (n - 1, n - 1 - new[r] // 3):
            h = rng.randrange(2)
            codes[int(b.px[b.pp[r] + j // page]), h, j % page, rng.randrange(d)] = 0xff
            pos = torch.arange(n - new[r], n, device="cuda")
            sees = (j <= pos) & ((j >= pos - window) if window >= 0 else torch.ones_like(pos, dtype=torch.bool))
            bad[b.qo[r]:b.qo[r + 1], 2 * h:2 * h + 2] |= sees[:, None, None]
    o, lse = b.run(window_left=window)
    assert torch.equal(torch.isnan(o), bad) and torch.equal(torch.isnan(lse), bad[..., 0])
    ref.check_attention(torch.where(bad, clean[0].to(o.dtype), o), torch.where(bad[..., 0], clean[1].float(), lse), clean)
