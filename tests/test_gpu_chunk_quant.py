"""pd_attn_chunk_quant against fp64 attention over the values that the 8-bit cache holds: every output within
its own bound (quant_ref.attention), over chunk lengths, cache lengths, groups, pages, blocks, layouts,
windows and types."""
import random

import pytest
import torch

import quant_ref as qref
import step_ref as ref

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import decode_ragged_paged_gb300 as pd

F32, BF16, E4M3 = torch.float32, torch.bfloat16, torch.float8_e4m3fn


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Batch:
    """Queries, an 8-bit cache and its page table; slots that hold no token are NaN, and so are the scales of
    blocks without any."""

    def __init__(self, seed, new, kv, hq, hkv, d, page, block, dt, layout="HND", spare=2, odd=False):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.new, self.kv, self.layout, self.d, self.page, self.block = new, kv, layout, d, page, block
        pages = [ref.ceil_div(n, page) for n in kv]
        self.qo = [sum(new[:i]) for i in range(len(new) + 1)]
        self.pp = [sum(pages[:i]) for i in range(len(new) + 1)]
        num = sum(pages) + spare
        self.px = torch.randperm(num, device="cuda", generator=g)[:sum(pages)].to(torch.int32)
        rnd = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
        self.q = rnd(sum(new), hq, d).to(dt)
        used = torch.zeros(num, page, dtype=torch.bool, device="cuda")
        for r, n in enumerate(kv):
            ids = self.px[self.pp[r]:self.pp[r + 1]].long()
            used[ids] = torch.arange(len(ids) * page, device="cuda").view(-1, page) < n
        held = used.view(num, page // block, block).any(-1)[:, None].expand(-1, hkv, -1)

        def pool():
            x = rnd(num, hkv, page // block, block, d) * torch.exp(0.7 * rnd(num, hkv, page // block, 1, 1))
            s = torch.exp2(torch.ceil(torch.log2(x.abs().amax((3, 4)) / 448)))
            s = s * 1.37 if odd else s
            x = (x / s[..., None, None]).clamp(-448, 448).to(E4M3).view(num, hkv, page, d)
            b = x.view(torch.uint8).clone()
            b.transpose(1, 2)[~used] = 0x7f  # NaN
            b = b if layout == "HND" else b.transpose(1, 2).contiguous()
            return b.view(E4M3), torch.where(held, s, torch.full_like(s, float("nan")))

        (self.k, self.ks), (self.v, self.vs) = pool(), pool()
        self.max_new, self.max_kv = max(new + [0]), max(kv + [0])

    def run(self, **kw):
        q = kw.pop("q", self.q)
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        args = dict(max_qo_len=self.max_new, max_kv_len=self.max_kv, layout=self.layout, dev_status=status)
        args.update(kw)
        o, lse = pd.pd_attn_chunk_quant(q, self.k, self.v, self.ks, self.vs, i32(self.kv), i32(self.pp), self.px,
                                        i32(self.qo), **args)
        torch.cuda.synchronize()
        assert int(status.item()) == 0
        return o, lse

    def ref(self, causal=True, window=-1, scale=None):
        return qref.attention(self.q, self.k, self.v, self.ks, self.vs, self.qo, self.kv, self.pp, self.px, causal=causal,
                              window=window, scale=scale, layout=self.layout)

    def check(self, causal=True, window=-1, **kw):
        o, lse = self.run(causal=causal, window_left=window, **kw)
        ref.check_attention(o, lse, self.ref(causal, window, kw.get("sm_scale")))


# q's type, head dim, page, block
TYPES = [(BF16, 128, 16, 16), (BF16, 64, 32, 8), (BF16, 128, 64, 32), (BF16, 64, 24, 24), (F32, 128, 16, 16),
         (F32, 64, 32, 8)]
MORE = TYPES + [(BF16, 128, 128, 128), (BF16, 128, 256, 64), (BF16, 64, 8, 8), (BF16, 64, 16, 4), (BF16, 128, 6, 3),
                (BF16, 64, 1, 1)]


@pytest.mark.parametrize("dt,d,page,block", MORE)
@pytest.mark.parametrize("layout", ["HND", "NHD"])
@pytest.mark.parametrize("hq,hkv", [(8, 2), (3, 3), (5, 1)])
def test_ragged_chunks(dt, d, page, block, layout, hq, hkv):
    Batch(1, [1, 5, 33, 64, 130, 2, 1], [1, 5, 40, 64, 400, 1000, 65], hq, hkv, d, page, block, dt, layout).check()


@pytest.mark.parametrize("dt,d,page,block", TYPES)
@pytest.mark.parametrize("hq,hkv", [(8, 8), (28, 4), (16, 1), (40, 8), (64, 1), (128, 1), (130, 1)])
def test_one_token(dt, d, page, block, hq, hkv):
    Batch(2, [1] * 6, [1, 17, 64, 127, 128, 700], hq, hkv, d, page, block, dt).check()


@pytest.mark.parametrize("dt,d,page,block", TYPES)
@pytest.mark.parametrize("window", [0, 1, 15, 63, 64, 127, 300, 2 ** 31 - 1])
def test_windows(dt, d, page, block, window):
    b = Batch(3, [1, 40, 200, 129, 3], [300, 40, 333, 700, 64], 8, 2, d, page, block, dt)
    b.check(window=window)
    b.check(causal=False, window=window)


@pytest.mark.parametrize("dt,d,page,block", TYPES)
def test_rows_without_keys(dt, d, page, block):
    b = Batch(4, [3, 0, 7, 200, 140, 0, 1], [0, 50, 2, 60, 140, 0, 0], 8, 2, d, page, block, dt)
    b.check()
    b.check(window=5)
    b.check(causal=False)


@pytest.mark.parametrize("dt,d,page,block", TYPES)
def test_full_attention_scale_and_output_types(dt, d, page, block):
    b = Batch(5, [50, 130], [70, 300], 8, 2, d, page, block, dt)
    b.check(causal=False)
    b.check(sm_scale=0.3)
    o, lse = b.run(o_dtype=F32)
    assert o.dtype == F32
    ref.check_attention(o, lse, b.ref())
    assert b.run(lse=False)[1] is None


@pytest.mark.parametrize("dt,d,page,block", TYPES)
@pytest.mark.parametrize("new,kv", [([1], [20000]), ([4], [9000]), ([3, 1], [5000, 70]), ([40], [12345]),
                                    ([300], [4000])])
def test_long_caches_are_cut_over_the_gpu(dt, d, page, block, new, kv):
    Batch(6, new, kv, 8, 2, d, page, block, dt).check()


@pytest.mark.parametrize("dt,d,page,block", TYPES[:2])
def test_many_requests(dt, d, page, block):
    rng = random.Random(7)
    new = [rng.choice([0, 1, 1, 2, 5]) for _ in range(1300)]
    kv = [max(n, rng.randint(0, 150)) for n in new]
    Batch(7, new, kv, 4, 2, d, page, block, dt).check()


@pytest.mark.parametrize("dt,d,page,block", TYPES)
@pytest.mark.parametrize("seed", range(6))
def test_drawn(dt, d, page, block, seed):
    rng = random.Random(100 + seed)
    B = rng.randint(1, 12)
    new = [int(2 ** rng.uniform(0, 9)) for _ in range(B)]
    kv = [n + int(2 ** rng.uniform(0, 11)) - 1 for n in new]
    hkv = rng.choice([1, 2, 3])
    b = Batch(seed, new, kv, hkv * rng.choice([1, 2, 3, 4, 7, 8]), hkv, d, page, block, dt, rng.choice(["HND", "NHD"]),
              odd=rng.random() < 0.3)
    b.check(window=rng.choice([-1, -1, 20, 200]), causal=rng.random() < 0.8)


@pytest.mark.parametrize("dt,d,page,block", TYPES[:2])
@pytest.mark.parametrize("new,kv,window", [
    ([900, 130, 3], [1200, 130, 500], -1),   # several rounds of whole items and a line
    ([500, 500], [500, 4000], -1),
    ([500, 0, 500], [4000, 0, 501], 100),
    ([700, 300], [600, 300], -1),            # rows without keys among whole items
    ([1] * 40 + [129, 1, 1, 257, 1], [64] * 40 + [200, 300, 64, 257, 1000], -1),  # one tile, and two, in turn
])
def test_whole_items_dealt_by_rounds(dt, d, page, block, new, kv, window):
    Batch(19, new, kv, 128, 8, d, page, block, dt).check(window=window)


@pytest.mark.parametrize("dt,d,page,block", TYPES)
def test_short_caches(dt, d, page, block):
    for B, top in ((1, 64), (3, 65), (4, 256), (9, 512), (16, 513), (19, 1024), (38, 300), (200, 60)):
        rng = random.Random(B)
        new = [rng.choice([0, 1, 1, 2, 9]) if B != 4 else 1 for _ in range(B)]
        kv = [max(n, rng.randint(0, top)) for n in new]
        kv[-1], new[-1] = top, 1
        Batch(24, new, kv, 8, 8 if B != 9 else 2, d, page, block, dt).check(window=rng.choice([-1, 40]))


@pytest.mark.parametrize("page", [8, 24, 40, 48, 72, 96, 192, 200])
@pytest.mark.parametrize("layout", ["HND", "NHD"])
def test_page_sizes(page, layout):
    Batch(22, [1, 70, 200], [777, 70, 1300], 8, 2, 128, page, 8, BF16, layout).check()
    Batch(23, [3, 150], [1500, 460], 8, 2, 64, page, page, BF16, layout).check(window=90)


@pytest.mark.parametrize("dt,d,page,block", TYPES[:2] + TYPES[4:5])
def test_strided_queries_rows_behind_the_last_and_bytes(dt, d, page, block):
    b = Batch(8, [20, 150], [20, 300], 8, 2, d, page, block, dt)
    b.k, b.v = b.k.view(torch.uint8), b.v.view(torch.uint8)
    wide = torch.full((180, 12 * d), float("nan"), device="cuda").to(dt)
    q = wide[:, 2 * d:10 * d].view(180, 8, d)
    q[:170] = b.q
    o = torch.full((180, 8, d), 3.0, device="cuda").to(dt)
    lse = torch.full((180, 8), 3.0, device="cuda")
    o2, l2 = b.run(q=q, o=o, lse=lse)
    ref.check_attention(o2[:170], l2[:170], b.ref())
    assert bool((o[170:] == 3).all()) and bool((lse[170:] == 3).all())


@pytest.mark.parametrize("dt,d,page,block", TYPES)
def test_sizes_far_apart(dt, d, page, block):
    # queries large and tiny, a channel that outweighs the rest, keys' and values' scales far up and down
    b = Batch(9, [70, 1, 30], [200, 90, 300], 8, 2, d, page, block, dt)
    b.q *= 30
    b.check()
    b.q *= 2.0 ** -90
    b.ks *= 2.0 ** 88
    b.vs *= 2.0 ** 40
    b.check()
    b.q[:, :, 3] *= 100
    b.check()
    b.vs *= 2.0 ** -100
    b.q[5], b.q[70] = 0.0, 0.0
    b.check()


@pytest.mark.parametrize("dt,d,page,block", TYPES)
def test_blocks_of_zeros_and_scales_of_zero(dt, d, page, block):
    b = Batch(31, [40, 3], [300, 128], 8, 2, d, page, block, dt)
    b.ks = torch.where(torch.rand_like(b.ks) < 0.3, torch.zeros_like(b.ks), b.ks)
    b.vs = torch.where(torch.rand_like(b.vs) < 0.3, torch.zeros_like(b.vs), b.vs)
    b.ks[torch.isnan(b.vs)] = float("nan")
    b.vs[torch.isnan(b.ks)] = float("nan")
    b.check()
    b.check(window=50)


@pytest.mark.parametrize("dt,d,page,block", TYPES)
@pytest.mark.parametrize("new,kv", [([40, 3], [300, 128]), ([1, 1], [300, 128])])
def test_scales_below_the_smallest(dt, d, page, block, new, kv):
    # of any sign they count as 2^-100: the scores of such a block of K are 0 (but for 2^-80), what is masked stays so
    b = Batch(35, new, kv, 8, 2, d, page, block, dt)
    for t in (b.ks, b.vs):
        t.copy_(torch.where(torch.rand_like(t) < 0.3, torch.full_like(t, -0.5), t))
    b.ks[torch.rand_like(b.ks) < 0.1] = 1e-38
    b.ks[torch.isnan(b.vs)] = float("nan")
    b.vs[torch.isnan(b.ks)] = float("nan")
    b.check()
    b.check(window=50)


@pytest.mark.parametrize("dt,d,page,block", TYPES)
def test_dead_keys_may_hold_anything(dt, d, page, block):
    # before every row's window: values and scales of NaN
    b = Batch(10, [3], [500], 8, 2, d, page, block, dt)
    dead = b.px[:(500 - 3 - 40) // page].long()
    for t in (b.k, b.v):
        t.view(torch.uint8)[dead] = 0x7f
    for t in (b.ks, b.vs):
        t[dead] = float("nan")
    b.check(window=40)
    for t in (b.ks, b.vs):
        t[dead] = float("inf")
    b.check(window=40)


@pytest.mark.parametrize("dt,d,page,block", TYPES[:2] + TYPES[4:5])
def test_nan_reaches_the_rows_that_see_it_and_no_others(dt, d, page, block):
    b = Batch(32, [10, 5], [80, 60], 4, 2, d, page, block, dt)
    good = b.ref()
    where = int(b.px[b.pp[0] + 75 // page]), 75 % page  # seen by the last rows of request 0, KV head 1
    b.v.view(torch.uint8)[where[0], 1, where[1], 3] = 0x7f
    o, lse = b.run()
    bad = torch.isnan(o)
    assert bool(bad[5:10, 2:, 3].all())  # tokens at positions 75 to 79
    assert not bool(bad[10:].any()) and not bool(bad[:, :2].any())
    b.q[2, 0, 1] = float("inf")
    o, lse = b.run()
    assert not bool(torch.isfinite(o[2, 0]).any()) and not bool(torch.isnan(o[3:5, 0]).any())
    keep = torch.ones(15, dtype=torch.bool, device="cuda")
    keep[:10] = False
    ref.check_attention(o[keep], lse[keep], tuple(x[keep] for x in good))


@pytest.mark.parametrize("dt,d,page,block", TYPES)
def test_a_rising_maximum(dt, d, page, block):
    b = Batch(11, [64, 3], [1000, 700], 4, 2, d, page, block, dt)
    for r in range(2):
        ids = b.px[b.pp[r]:b.pp[r + 1]].long()
        n, per = len(ids), page // block
        t = torch.arange(n * per, device="cuda").view(n, 1, per).float() / (n * per)
        b.ks[ids] *= 2.0 ** torch.round(4 * t if r == 0 else 4 - 4 * t)
    b.check()


def test_agrees_with_pd_attn_chunk_over_the_same_values():
    rng = random.Random(1)
    b = Batch(12, [1] * 20 + [9, 200], [rng.randint(1, 3000) for _ in range(20)] + [900, 700], 32, 8, 128, 16, 16, BF16)
    k, v = (torch.nan_to_num(qref.dequant(x, s, "HND")).to(BF16) for x, s in ((b.k, b.ks), (b.v, b.vs)))
    o, lse = b.run()
    o2, lse2 = pd.pd_attn_chunk(b.q, k, v, i32(b.kv), i32(b.pp), b.px, i32(b.qo), max_qo_len=200, max_kv_len=3000)
    top = float(v.float().abs().max())
    assert float((o.float() - o2.float()).abs().max()) <= 2.0 ** -6 * top
    assert float((lse - lse2).abs().max()) <= 2e-3


@pytest.mark.parametrize("dt", [F32, BF16])
def test_bad_batches_are_skipped_and_reported(dt):
    b = Batch(13, [5, 6, 7], [50, 60, 70], 8, 2, 64, 16, 16, dt)
    good = b.ref()

    def call(rows, **kw):
        qo, kv, pp, px = (kw.get(n, x) for n, x in (("qo", b.qo), ("kv", b.kv), ("pp", b.pp), ("px", b.px)))
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        o, lse = pd.pd_attn_chunk_quant(b.q, b.k, b.v, b.ks, b.vs, i32(kv), i32(pp), px, i32(qo),
                                        max_qo_len=kw.get("max_qo", 7), max_kv_len=70, dev_status=status,
                                        o=torch.zeros_like(b.q))
        torch.cuda.synchronize()
        ref.check_attention(o[rows], lse[rows], tuple(x[rows] for x in good))
        return int(status.item())

    assert call(slice(0, 18)) == 0
    assert call(slice(5, 18), kv=[-1, 60, 70]) == 2
    assert call(slice(5, 18), kv=[71, 60, 70]) == 2
    assert call(slice(0, 11), max_qo=6) == 2
    assert call(slice(0, 5), qo=[0, 5, 4, 18]) in (1, 2)
    assert call(slice(0, 11), qo=[0, 5, 11, 19]) == 1
    px = b.px.clone()
    px[0] = 10 ** 6
    assert call(slice(5, 18), px=px) == 3
    px[0] = -1
    assert call(slice(5, 18), px=px) == 3


def test_workspace_reuse_streams_and_a_graph():
    a = Batch(14, [1, 70], [900, 4000], 8, 2, 128, 16, 16, BF16)
    b = Batch(15, [300], [2000], 8, 2, 128, 16, 16, BF16)
    ws = torch.empty(100 << 20, dtype=torch.uint8, device="cuda").fill_(255)
    for x in (a, b, a):
        ref.check_attention(*x.run(workspace=ws), x.ref())
    ref.check_attention(*a.run(workspace=ws[:64]), a.ref())  # too small: the binding takes one that fits
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    ws2 = torch.empty_like(ws)
    args = [(x.q, x.k, x.v, x.ks, x.vs, i32(x.kv), i32(x.pp), x.px, i32(x.qo)) for x in (a, b)]
    torch.cuda.synchronize()
    outs = [[], []]
    for _ in range(5):
        for i, (x, s, w) in enumerate(((a, s1, ws), (b, s2, ws2))):
            outs[i].append(pd.pd_attn_chunk_quant(*args[i], max_qo_len=x.max_new, max_kv_len=x.max_kv, workspace=w,
                                                  stream=s))
    torch.cuda.synchronize()
    for x, res in ((a, outs[0]), (b, outs[1])):
        for o, lse in res:
            ref.check_attention(o, lse, x.ref())
            assert torch.equal(o, res[0][0]) and torch.equal(lse, res[0][1])  # the same bits every time
    kv, qo = args[0][5], args[0][8]
    o, lse = torch.zeros_like(a.q), torch.zeros(a.q.shape[:2], device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(s1):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s1):
            pd.pd_attn_chunk_quant(*args[0], max_qo_len=71, max_kv_len=4000, workspace=ws, o=o, lse=lse)
    for new, n in (([1, 70], [900, 4000]), ([50, 20], [800, 3999]), ([0, 71], [0, 71]), ([71, 0], [71, 4000])):
        kv.copy_(i32(n))
        qo.copy_(i32([0, new[0], sum(new)]))
        m, behind = sum(new), o.clone()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        want = qref.attention(a.q, a.k, a.v, a.ks, a.vs, [0, new[0], m], n, a.pp, a.px)
        ref.check_attention(o[:m], lse[:m], tuple(x[:m] for x in want))
        assert torch.equal(o[m:], behind[m:])


@pytest.mark.parametrize("dt,d,page,block", TYPES[:2] + TYPES[4:5])
def test_outputs_and_workspace_aligned_to_16_bytes_only(dt, d, page, block):
    b = Batch(18, [3, 100], [5000, 300], 8, 2, d, page, block, dt)
    size = b.q.numel()
    buf = torch.zeros(size + 64, dtype=dt, device="cuda")
    off = 16 // buf.element_size()
    o = buf[off:off + size].view(b.q.shape)
    ws = torch.empty((100 << 20) + 16, dtype=torch.uint8, device="cuda")[16:]
    for args in (dict(o=o), dict(workspace=ws), dict(o=o, workspace=ws)):
        ref.check_attention(*b.run(**args), b.ref())
        assert bool((buf[:off] == 0).all()) and bool((buf[off + size:] == 0).all())


def test_cache_past_32_bit_offsets():
    d, hkv, page = 128, 8, 64
    pages = (1 << 32) // (hkv * page * d) + 40
    k, v = (torch.zeros(pages, hkv, page, d, dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.full((pages, hkv, 2), 2.0 ** -7, device="cuda") for _ in range(2))
    g = torch.Generator(device="cuda").manual_seed(16)
    px = torch.tensor([pages - 1, 0, pages - 2, 1, pages - 30], device="cuda", dtype=torch.int32)
    for pool in (k, v):
        pool[px.long()] = (100 * torch.randn(5, hkv, page, d, device="cuda", generator=g)).clamp(-448, 448).to(E4M3).view(
            torch.uint8)
    q = torch.randn(9, 32, d, device="cuda", generator=g).to(BF16)
    at = torch.arange(5, device="cuda", dtype=torch.int32)
    for layout in ("HND", "NHD"):
        kk, vv = (x if layout == "HND" else x.view(pages, page, hkv, d) for x in (k, v))
        o, lse = pd.pd_attn_chunk_quant(q, kk, vv, ks, vs, i32([300]), i32([0, 5]), px, i32([0, 9]), max_qo_len=9,
                                        max_kv_len=300, layout=layout)
        few = [x[px.long()] for x in (kk, vv, ks, vs)]
        ref.check_attention(o, lse, qref.attention(q, *few, [0, 9], [300], [0, 5], at, layout=layout))


@pytest.mark.parametrize("dt,d,page,block", TYPES)
@pytest.mark.parametrize("new,kv", [([1, 7, 130], [2000, 60, 700]), ([900], [4000]), ([1] * 40, [300] * 40)])
def test_a_call_repeats_itself(dt, d, page, block, new, kv):
    b = Batch(28, new, kv, 16, 4, d, page, block, dt)
    first = b.run()
    for _ in range(4):
        again = b.run()
        assert torch.equal(again[0], first[0]) and torch.equal(again[1], first[1])


def test_bounds_are_read_back_on_the_stream():
    b = Batch(33, [1, 30], [100, 60], 8, 2, 128, 16, 16, BF16)
    ref.check_attention(*b.run(max_qo_len=None, max_kv_len=None), b.ref())


def test_refusals():
    b = Batch(17, [4], [40], 8, 2, 64, 16, 16, BF16)
    pools, lists = (b.k, b.v, b.ks, b.vs), (i32(b.kv), i32(b.pp), b.px, i32(b.qo))
    kw = dict(max_qo_len=4, max_kv_len=40)
    bad = [
        lambda: pd.pd_attn_chunk_quant(b.q.half(), *pools, *lists, **kw),
        lambda: pd.pd_attn_chunk_quant(b.q[:, :7], *pools, *lists, **kw),
        lambda: pd.pd_attn_chunk_quant(b.q.transpose(0, 1), *pools, *lists, **kw),
        lambda: pd.pd_attn_chunk_quant(b.q, b.k.float(), b.v.float(), *pools[2:], *lists, **kw),
        lambda: pd.pd_attn_chunk_quant(b.q, b.k, b.v.view(torch.uint8), *pools[2:], *lists, **kw),
        lambda: pd.pd_attn_chunk_quant(b.q, b.k, b.v, b.ks[:-1], b.vs, *lists, **kw),
        lambda: pd.pd_attn_chunk_quant(b.q, b.k, b.v, b.ks, b.vs.repeat(1, 1, 2), *lists, **kw),
        lambda: pd.pd_attn_chunk_quant(b.q, b.k, b.v, b.ks.repeat(1, 1, 3), b.vs.repeat(1, 1, 3), *lists, **kw),
        lambda: pd.pd_attn_chunk_quant(b.q, b.k, b.v, b.ks.double(), b.vs.double(), *lists, **kw),
        lambda: pd.pd_attn_chunk_quant(b.q, *pools, *lists, o=b.q[:2], **kw),
        lambda: pd.pd_attn_chunk_quant(b.q, *pools, *lists[:3], i32([0]), **kw),
        lambda: pd.pd_attn_chunk(b.q, b.k, b.v, *lists, **kw),
    ]
    for call in bad:
        with pytest.raises(pd.PdError):
            call()
