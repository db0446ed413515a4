"""pd_attn_chunk against fp64 attention: every output within its own bound (step_ref.attention), over
chunk lengths, cache lengths, groups, pages, layouts, windows and types."""
import ctypes
import random

import pytest
import torch

import step_ref as ref

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import decode_ragged_paged_gb300 as pd

F32, BF16 = torch.float32, torch.bfloat16


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Batch:
    """Queries, pools and page table; slots that hold no token are filled with `fill`."""

    def __init__(self, seed, new, kv, hq, hkv, d, page, dt, layout="HND", fill=float("nan"), spare=2):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.new, self.kv, self.layout, self.d = new, kv, layout, d
        pages = [ref.ceil_div(n, page) for n in kv]
        self.qo = [sum(new[:i]) for i in range(len(new) + 1)]
        self.pp = [sum(pages[:i]) for i in range(len(new) + 1)]
        num = sum(pages) + spare
        self.px = torch.randperm(num, device="cuda", generator=g)[:sum(pages)].to(torch.int32)
        rnd = lambda *s: torch.randn(*s, device="cuda", generator=g).to(dt)  # noqa: E731
        self.q = rnd(sum(new), hq, d)
        shape = (num, hkv, page, d) if layout == "HND" else (num, page, hkv, d)
        self.k, self.v = rnd(*shape), rnd(*shape)
        used = torch.zeros(num, page, dtype=torch.bool, device="cuda")
        for r, n in enumerate(kv):
            ids = self.px[self.pp[r]:self.pp[r + 1]].long()
            used[ids] = torch.arange(len(ids) * page, device="cuda").view(-1, page) < n
        for pool in (self.k, self.v):
            (pool.transpose(1, 2) if layout == "HND" else pool)[~used] = fill
        self.max_new, self.max_kv = max(new + [0]), max(kv + [0])

    def run(self, **kw):
        q = kw.pop("q", self.q)
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        args = dict(max_qo_len=self.max_new, max_kv_len=self.max_kv, layout=self.layout, dev_status=status)
        args.update(kw)
        o, lse = pd.pd_attn_chunk(q, self.k, self.v, i32(self.kv), i32(self.pp), self.px, i32(self.qo), **args)
        torch.cuda.synchronize()
        assert int(status.item()) == 0
        return o, lse

    def ref(self, causal=True, window=-1, scale=None):
        return ref.attention(self.q, self.k, self.v, self.qo, self.kv, self.pp, self.px, causal=causal, window=window,
                             scale=scale, layout=self.layout)

    def check(self, causal=True, window=-1, **kw):
        o, lse = self.run(causal=causal, window_left=window, **kw)
        ref.check_attention(o, lse, self.ref(causal, window, kw.get("sm_scale")))


TYPES = [(F32, 64, 16), (F32, 128, 24), (BF16, 128, 16), (BF16, 64, 32), (BF16, 128, 24), (BF16, 64, 1),
         (BF16, 128, 128), (BF16, 128, 256), (BF16, 64, 8)]


@pytest.mark.parametrize("dt,d,page", TYPES)
@pytest.mark.parametrize("layout", ["HND", "NHD"])
@pytest.mark.parametrize("hq,hkv", [(8, 2), (3, 3), (5, 1)])
def test_ragged_chunks(dt, d, page, layout, hq, hkv):
    b = Batch(1, [1, 5, 33, 64, 130, 2, 1], [1, 5, 40, 64, 400, 1000, 65], hq, hkv, d, page, dt, layout)
    b.check()


@pytest.mark.parametrize("dt,d,page", TYPES[:5])
@pytest.mark.parametrize("hq,hkv", [(8, 8), (28, 4), (16, 1), (40, 8), (64, 1), (128, 1), (130, 1)])
def test_one_token(dt, d, page, hq, hkv):
    Batch(2, [1] * 6, [1, 17, 64, 127, 128, 700], hq, hkv, d, page, dt).check()


@pytest.mark.parametrize("dt,d,page", TYPES[:4])
@pytest.mark.parametrize("window", [0, 1, 15, 63, 64, 127, 128, 300, 2 ** 31 - 1])
def test_windows(dt, d, page, window):
    b = Batch(3, [1, 40, 200, 129, 3], [300, 40, 333, 700, 64], 8, 2, d, page, dt)
    b.check(window=window)
    b.check(causal=False, window=window)


@pytest.mark.parametrize("dt,d,page", TYPES[:4])
def test_rows_without_keys(dt, d, page):
    # empty caches, no new tokens, and more new tokens than keys: the first rows see nothing
    b = Batch(4, [3, 0, 7, 200, 140, 0, 1], [0, 50, 2, 60, 140, 0, 0], 8, 2, d, page, dt)
    b.check()
    b.check(window=5)
    b.check(causal=False)


@pytest.mark.parametrize("dt,d,page", TYPES[:4])
def test_full_attention_scale_and_output_types(dt, d, page):
    b = Batch(5, [50, 130], [70, 300], 8, 2, d, page, dt)
    b.check(causal=False)
    b.check(sm_scale=0.3)
    o, lse = b.run(o_dtype=F32)
    assert o.dtype == F32
    ref.check_attention(o, lse, b.ref())
    o2, none = b.run(lse=False)
    assert none is None


@pytest.mark.parametrize("dt,d,page", TYPES[:4])
@pytest.mark.parametrize("new,kv", [([1], [20000]), ([4], [9000]), ([3, 1], [5000, 70]), ([40], [12345]),
                                    ([300], [4000])])
def test_long_caches_are_cut_over_the_gpu(dt, d, page, new, kv):
    Batch(6, new, kv, 8, 2, d, page, dt).check()


@pytest.mark.parametrize("dt,d,page", [TYPES[0], TYPES[2], TYPES[3]])
def test_many_requests(dt, d, page):
    rng = random.Random(7)
    new = [rng.choice([0, 1, 1, 2, 5]) for _ in range(1300)]
    kv = [max(n, rng.randint(0, 150)) for n in new]
    Batch(7, new, kv, 4, 2, d, page, dt).check()


@pytest.mark.parametrize("dt,d,page", TYPES[:4])
@pytest.mark.parametrize("seed", range(6))
def test_drawn(dt, d, page, seed):
    rng = random.Random(100 + seed)
    B = rng.randint(1, 12)
    new = [int(2 ** rng.uniform(0, 9)) for _ in range(B)]
    kv = [n + int(2 ** rng.uniform(0, 11)) - 1 for n in new]
    hkv = rng.choice([1, 2, 3])
    b = Batch(seed, new, kv, hkv * rng.choice([1, 2, 3, 4, 7, 8]), hkv, d, page, dt, rng.choice(["HND", "NHD"]))
    b.check(window=rng.choice([-1, -1, 20, 200]), causal=rng.random() < 0.8)


@pytest.mark.parametrize("dt,d,page", [TYPES[0], TYPES[2], TYPES[3]])
@pytest.mark.parametrize("new,kv,window", [
    ([900, 130, 3], [1200, 130, 500], -1),   # several rounds of whole items and a line
    ([500, 500], [500, 4000], -1),           # short items first: some parts of the line get no share
    ([500, 0, 500], [4000, 0, 501], 100),
    ([700, 300], [600, 300], -1),            # rows without keys among whole items
])
def test_whole_items_dealt_by_rounds(dt, d, page, new, kv, window):
    Batch(19, new, kv, 128, 8, d, page, dt).check(window=window)


@pytest.mark.parametrize("dt,d,page", [TYPES[0], TYPES[2], TYPES[3]])
def test_many_requests_of_several_blocks(dt, d, page):
    # more requests, and then more blocks, than a warp plans by itself
    rng = random.Random(20)
    new = [rng.choice([33, 20, 70, 0, 1]) for _ in range(140)]
    Batch(20, new, [n + rng.randint(0, 80) for n in new], 64, 4, d, page, dt).check()
    Batch(21, [1300, 5], [1300, 2000], 128, 1, d, page, dt).check(window=64)


@pytest.mark.parametrize("dt,d,page", TYPES[:4])
def test_short_caches(dt, d, page):
    # items that are not cut, up to the lengths and batches from which they are, and beyond
    for B, top in ((1, 64), (3, 65), (4, 256), (9, 512), (16, 513), (19, 1024), (20, 1025), (38, 300), (200, 60)):
        rng = random.Random(B)
        new = [rng.choice([0, 1, 1, 2, 9]) if B != 4 else 1 for _ in range(B)]
        kv = [max(n, rng.randint(0, top)) for n in new]
        kv[-1], new[-1] = top, 1
        Batch(24, new, kv, 8, 8 if B != 9 else 2, d, page, dt).check(window=rng.choice([-1, 40]))


@pytest.mark.parametrize("page", [8, 12, 20, 24, 40, 48, 72, 96, 192, 200])
@pytest.mark.parametrize("layout", ["HND", "NHD"])
def test_page_sizes(page, layout):
    # pages that end inside a tile, and tiles that end inside a page, at any offset
    Batch(22, [1, 70, 200], [777, 70, 1300], 8, 2, 128 if page % 16 else 64, page, BF16, layout).check()
    Batch(23, [3, 150], [1500, 460], 8, 2, 64, page, BF16, layout).check(window=90)


@pytest.mark.parametrize("dt,d,page", TYPES[:4])
def test_strided_queries_and_rows_behind_the_last(dt, d, page):
    b = Batch(8, [20, 150], [20, 300], 8, 2, d, page, dt)
    wide = torch.full((180, 12 * d), float("nan"), device="cuda").to(dt)
    q = wide[:, 2 * d:10 * d].view(180, 8, d)
    q[:170] = b.q
    o = torch.full((180, 8, d), 3.0, device="cuda").to(dt)
    lse = torch.full((180, 8), 3.0, device="cuda")
    o2, l2 = b.run(q=q, o=o, lse=lse)
    ref.check_attention(o2[:170], l2[:170], b.ref())
    assert bool((o[170:] == 3).all()) and bool((lse[170:] == 3).all())


@pytest.mark.parametrize("dt,d,page", TYPES[:4])
def test_large_scores_and_infinite_masked_places(dt, d, page):
    b = Batch(9, [70, 1], [200, 90], 8, 2, d, page, dt, fill=float("inf"))
    b.q *= 30
    b.check()
    b = Batch(9, [70, 1], [200, 90], 8, 2, d, page, dt, fill=-float("inf"))
    b.check()
    # keys that have left every row's window may hold anything
    b = Batch(10, [3], [500], 8, 2, d, page, dt)
    dead = b.px[:(500 - 3 - 40) // page].long()
    b.k[dead], b.v[dead] = float("nan"), float("nan")
    b.check(window=40)


@pytest.mark.parametrize("dt,d,page", TYPES[:4])
def test_a_rising_maximum(dt, d, page):
    # scores that grow along the keys, past any bound kept from earlier tiles, and that fall again
    b = Batch(11, [64, 3], [1000, 700], 4, 2, d, page, dt)
    rows = b.k.transpose(1, 2) if b.layout == "HND" else b.k
    for r in range(2):
        ids = b.px[b.pp[r]:b.pp[r + 1]].long()
        n = b.kv[r]
        t = torch.arange(len(ids) * page, device="cuda").view(-1, page)
        up = (t.float() / n * 12).clamp(max=12) if r == 0 else ((n - t).float() / n * 12).clamp(min=0)
        rows[ids] = (rows[ids].float() * up[:, :, None, None]).to(dt)
    b.check()


def test_decode_agrees_with_pd_attn_decode():
    rng = random.Random(1)
    b = Batch(12, [1] * 20, [rng.randint(1, 3000) for _ in range(20)], 32, 8, 128, 16, BF16)
    o, lse = b.run()
    o2, lse2 = pd.pd_attn_decode(b.q, b.k, b.v, i32(b.kv), i32(b.pp), b.px, max_kv_len=b.max_kv)
    assert float((o.float() - o2.float()).abs().max()) <= 1e-2 and float((lse - lse2).abs().max()) <= 1e-3


@pytest.mark.parametrize("dt", [F32, BF16])
def test_bad_batches_are_skipped_and_reported(dt):
    b = Batch(13, [5, 6, 7], [50, 60, 70], 8, 2, 64, 16, dt, fill=0.0)
    good = b.ref()

    def call(rows, **kw):
        """Runs with the changes and checks the other requests' rows; returns the status."""
        qo, kv, pp, px = (kw.get(n, x) for n, x in (("qo", b.qo), ("kv", b.kv), ("pp", b.pp), ("px", b.px)))
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        o, lse = pd.pd_attn_chunk(b.q, b.k, b.v, i32(kv), i32(pp), px, i32(qo), max_qo_len=kw.get("max_qo", 7),
                                  max_kv_len=70, dev_status=status, o=torch.zeros_like(b.q))
        torch.cuda.synchronize()
        ref.check_attention(o[rows], lse[rows], tuple(x[rows] for x in good))
        return int(status.item())

    assert call(slice(0, 18)) == 0
    assert call(slice(5, 18), kv=[-1, 60, 70]) == 2
    assert call(slice(5, 18), kv=[71, 60, 70]) == 2
    assert call(slice(0, 11), max_qo=6) == 2
    assert call(slice(0, 5), qo=[0, 5, 4, 18]) in (1, 2)
    assert call(slice(0, 11), qo=[0, 5, 11, 19]) == 1
    assert call(slice(5, 18), pp=[1, 4, 8, 13]) in (0, 3)     # request 0 on another's pages or short of them
    px = b.px.clone()
    px[0] = 10 ** 6
    assert call(slice(5, 18), px=px) == 3
    px[0] = -1
    assert call(slice(5, 18), px=px) == 3


def test_workspace_reuse_streams_and_a_graph():
    a = Batch(14, [1, 70], [900, 4000], 8, 2, 128, 16, BF16)
    b = Batch(15, [300], [2000], 8, 2, 128, 16, BF16)
    ws = torch.empty(100 << 20, dtype=torch.uint8, device="cuda").fill_(255)
    for x in (a, b, a):
        ref.check_attention(*x.run(workspace=ws), x.ref())
    o, lse = a.run(workspace=ws[:64])       # too small: the binding takes one that fits
    ref.check_attention(o, lse, a.ref())
    # two streams at once, a workspace each
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    ws2 = torch.empty_like(ws)
    args = [(x.q, x.k, x.v, i32(x.kv), i32(x.pp), x.px, i32(x.qo)) for x in (a, b)]
    torch.cuda.synchronize()
    outs = [[], []]
    for _ in range(5):
        for i, (x, s, w) in enumerate(((a, s1, ws), (b, s2, ws2))):
            outs[i].append(pd.pd_attn_chunk(*args[i], max_qo_len=x.max_new, max_kv_len=x.max_kv, workspace=w, stream=s))
    torch.cuda.synchronize()
    for x, res in ((a, outs[0]), (b, outs[1])):
        r = x.ref()
        for o, lse in res:
            ref.check_attention(o, lse, r)
            assert torch.equal(o, res[0][0]) and torch.equal(lse, res[0][1])  # the same bits every time
    # captured, replayed with other lengths within the bounds
    kv, qo = args[0][3], args[0][6]
    o, lse = torch.zeros_like(a.q), torch.zeros(a.q.shape[:2], device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(s1):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s1):
            pd.pd_attn_chunk(*args[0], max_qo_len=71, max_kv_len=4000, workspace=ws, o=o, lse=lse)
    for new, n in (([1, 70], [900, 4000]), ([50, 20], [800, 3999]), ([0, 71], [0, 71]), ([71, 0], [71, 4000])):
        kv.copy_(i32(n))
        qo.copy_(i32([0, new[0], sum(new)]))
        m, behind = sum(new), o.clone()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        want = ref.attention(a.q, a.k, a.v, [0, new[0], m], n, a.pp, a.px)
        ref.check_attention(o[:m], lse[:m], tuple(x[:m] for x in want))
        assert torch.equal(o[m:], behind[m:])  # rows behind the last request's are left alone


@pytest.mark.parametrize("dt,d,page", TYPES[:4])
def test_outputs_and_workspace_aligned_to_16_bytes_only(dt, d, page):
    b = Batch(18, [3, 100], [5000, 300], 8, 2, d, page, dt)
    size = b.q.numel()
    buf = torch.zeros(size + 64, dtype=dt, device="cuda")
    off = 16 // buf.element_size()
    o = buf[off:off + size].view(b.q.shape)
    ws = torch.empty((100 << 20) + 16, dtype=torch.uint8, device="cuda")[16:]
    for args in (dict(o=o), dict(workspace=ws), dict(o=o, workspace=ws)):
        got, lse = b.run(**args)
        ref.check_attention(got, lse, b.ref())
        assert bool((buf[:off] == 0).all()) and bool((buf[off + size:] == 0).all())


def test_cache_past_32_bit_offsets():
    d, hkv, page = 128, 8, 64
    pages = (1 << 32) // (hkv * page * d) + 40
    k, v = (torch.zeros(pages, hkv, page, d, dtype=BF16, device="cuda") for _ in range(2))
    g = torch.Generator(device="cuda").manual_seed(16)
    px = torch.tensor([pages - 1, 0, pages - 2, 1, pages - 30], device="cuda", dtype=torch.int32)
    for pool in (k, v):
        pool[px.long()] = torch.randn(5, hkv, page, d, device="cuda", generator=g).to(BF16)
    q = torch.randn(9, 32, d, device="cuda", generator=g).to(BF16)
    for layout in ("HND", "NHD"):
        kk, vv = (x if layout == "HND" else x.view(pages, page, hkv, d) for x in (k, v))
        o, lse = pd.pd_attn_chunk(q, kk, vv, i32([300]), i32([0, 5]), px, i32([0, 9]), max_qo_len=9, max_kv_len=300,
                                  layout=layout)
        ref.check_attention(o, lse, ref.attention(q, kk, vv, [0, 9], [300], [0, 5], px, layout=layout))


def test_more_work_than_32_bits_of_units():
    """16384 single tokens over 2^20 keys each, 8 heads: 2^31 units and 262144 more. All requests share
    one list of pages. Keys count by their position (V is a ramp), so that any that are left out show.
    Bounds: a row's sum takes 2^14 additions of a tile's weights in fp32, its output 2^16 of 16 keys
    each in the tensor cores (a truncating adder, 2^-23 each)."""
    requests, hq, d, page, n = 16384, 8, 64, 4096, 1 << 20
    g = torch.Generator(device="cuda").manual_seed(29)
    k = torch.randn(n // page, hq, page, d, device="cuda", generator=g).to(BF16)
    ramp = torch.arange(n, device="cuda", dtype=torch.float32).view(-1, 1, page, 1) / n
    v = (ramp * (1 + torch.arange(d, device="cuda") / d)).expand(-1, hq, -1, -1).to(BF16).contiguous()
    q = torch.randn(requests, hq, d, device="cuda", generator=g).to(BF16)
    px = torch.arange(n // page, device="cuda", dtype=torch.int32).repeat(requests)
    pp = torch.arange(requests + 1, device="cuda", dtype=torch.int32) * (n // page)
    qo, kv = torch.arange(requests + 1, device="cuda", dtype=torch.int32), i32([n] * requests)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    o = torch.full_like(q, float("nan"))
    lse = torch.full((requests, hq), float("nan"), device="cuda")
    pd.pd_attn_chunk(q, k, v, kv, pp, px, qo, max_qo_len=1, max_kv_len=n, o=o, lse=lse, dev_status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    assert bool(torch.isfinite(o.float()).all()) and bool(torch.isfinite(lse).all())
    scale = d ** -0.5
    at = torch.cat([torch.tensor([0, 1, requests - 1]), torch.randint(requests, (5,))]).cuda()
    for h in (0, 3, hq - 1):
        kh, vh, qh = k[:, h].reshape(n, d).double(), v[:, h].reshape(n, d).double(), q[at, h].double()
        s = qh @ kh.T * scale
        es = 4 * d * 2.0 ** -24 * scale * (qh.abs() @ kh.abs().T).amax(-1)
        want = torch.logsumexp(s, -1)
        out = torch.softmax(s, -1) @ vh  # (and of |V|, as no value is negative)
        rel = 2 * es + 2.0 ** -20 + 2.0 ** -10
        assert bool(((lse[at, h].double() - want).abs() <= rel + 2.0 ** -21 * (1 + want.abs())).all())
        lim = ((rel + 2.0 ** -8 + 2.0 ** -7)[:, None] + 2.0 ** -8) * out
        assert bool(((o[at, h].double() - out).abs() <= lim).all())


def test_requests_on_the_same_rows_are_refused():
    """512 requests that all claim the same 2^23 rows (the indptr falls back to 0 in between), of a
    block each, and one of 5 rows: 2^32 + 5 blocks. The plan refuses the batch before any row is
    read, so q need not have them."""
    rows, B = 1 << 23, 1025
    q = torch.zeros(8, 64, 64, device="cuda")
    k = torch.zeros(1, 1, 16, 64, device="cuda")
    o = torch.full_like(q, 3.0)
    qo = i32([0, rows] * 512 + [0, 5])
    kv, pp = i32([1] * B), torch.arange(B + 1, device="cuda", dtype=torch.int32)
    px = torch.zeros(B, device="cuda", dtype=torch.int32)
    lib = pd.load_library()
    desc = pd.make_attn_desc(q, k)
    batch = pd.make_batch(kv, pp, px, 1, qo_indptr=qo, total_qo=rows, max_qo_len=rows, max_kv_len=1)
    size = lib.pd_attn_chunk_workspace_size(ctypes.byref(desc), ctypes.byref(batch))
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    status = i32([0])
    assert lib.pd_attn_chunk(ctypes.byref(desc), ctypes.byref(batch), -1, 0, q.data_ptr(), k.data_ptr(), k.data_ptr(),
                             o.data_ptr(), None, ws.data_ptr(), size, status.data_ptr(), None) == 0
    torch.cuda.synchronize()
    assert int(status.item()) == 1 and bool((o == 3).all())


def few_keys(b, causal, window):
    """Which rows see fewer than 128 keys."""
    n = torch.cat([torch.full((x,), y) for x, y in zip(b.new, b.kv)])
    t = torch.cat([torch.arange(y - x, y) for x, y in zip(b.new, b.kv)])
    lo = (t - window).clamp(min=0) if window >= 0 else torch.zeros_like(t)
    return (((t + 1 if causal else n) - lo) < 128).cuda()


@pytest.mark.parametrize("d,page,layout", [(64, 16, "HND"), (128, 24, "NHD"), (128, 16, "HND")])
@pytest.mark.parametrize("new,kv,causal,window", [
    ([128], [128], True, -1),                            # a prompt's first chunk
    ([1, 1, 1, 2, 5, 1], [1, 2, 60, 64, 127, 126], True, -1),
    ([7, 200, 300], [3, 140, 300], True, -1),            # rows without keys; a second block that sees more
    ([300, 1], [1000, 3000], True, 20),                  # a narrow window over a long cache
    ([40, 90], [100, 90], False, -1),
    ([200], [260], False, 30),                           # its last rows see the fewest
    ([1] * 300, [1 + i % 126 for i in range(300)], True, -1),
])
def test_rows_that_see_few_keys_have_exact_weights(d, page, layout, new, kv, causal, window):
    """Weights of rows with fewer than 128 keys enter the product with V as two bf16 terms: the second
    is the first's remainder, at most 2^-8 of the weight, and off by at most 2^-8 of that: 2^-16 in all.
    (step_ref.attention of fp32 queries allows for everything but that.)"""
    b = Batch(25, new, kv, 8, 2, d, page, BF16, layout)
    o, lse = b.run(causal=causal, window_left=window, o_dtype=F32, sm_scale=0.05)
    kw = dict(causal=causal, window=window, scale=0.05, layout=layout)
    lists = (b.qo, b.kv, b.pp, b.px)
    ro, rl, ob, lb = ref.attention(b.q.float(), b.k, b.v, *lists, **kw)
    sizes = ref.attention(b.q.float(), b.k, b.v.abs(), *lists, **kw)[0]
    few = few_keys(b, causal, window)
    assert bool(few.any())
    ref.check_attention(o, lse, (ro, rl, ob + torch.where(few, 2.0 ** -16, 2.0 ** -8)[:, None, None] * sizes, lb))


@pytest.mark.parametrize("d", [64, 128])
def test_two_keys_stay_within_the_library_bound(d):
    # outputs of 2 to 4, whose own rounding takes 2^-7 of the 1e-2, from values that lie far apart
    b = Batch(26, [1] * 200, [2] * 200, 32, 8, d, 16, BF16)
    g = torch.Generator(device="cuda").manual_seed(27)
    b.v[:, :, 0] = 3.5 + 0.5 * torch.rand(b.v[:, :, 0].shape, device="cuda", generator=g).to(BF16)
    b.v[:, :, 1] = torch.rand(b.v[:, :, 1].shape, device="cuda", generator=g).to(BF16)
    o, lse = b.run()
    assert float((o.double() - b.ref()[0]).abs().max()) <= 1e-2


@pytest.mark.parametrize("dt,d,page", TYPES[:4])
@pytest.mark.parametrize("new,kv", [([1, 7, 130], [2000, 60, 700]), ([900], [4000]), ([1] * 40, [300] * 40)])
def test_a_call_repeats_itself(dt, d, page, new, kv):
    b = Batch(28, new, kv, 16, 4, d, page, dt)
    first = b.run()
    for _ in range(4):
        again = b.run()
        assert torch.equal(again[0], first[0]) and torch.equal(again[1], first[1])


def test_refusals():
    b = Batch(17, [4], [40], 8, 2, 64, 16, F32)
    args = (b.k, b.v, i32(b.kv), i32(b.pp), b.px, i32(b.qo))
    kw = dict(max_qo_len=4, max_kv_len=40)
    bad = [
        lambda: pd.pd_attn_chunk(b.q.bfloat16(), *args, **kw),
        lambda: pd.pd_attn_chunk(b.q[:, :7], *args, **kw),
        lambda: pd.pd_attn_chunk(b.q.transpose(0, 1), *args, **kw),
        lambda: pd.pd_attn_chunk(b.q, *args, o=b.q[:2], **kw),
        lambda: pd.pd_attn_chunk(b.q, *args, lse=torch.zeros(2, device="cuda"), **kw),
        lambda: pd.pd_attn_chunk(b.q, b.k[:, :1], *args[1:], **kw),
        lambda: pd.pd_attn_chunk(b.q, *args[:2], i32(b.kv).long(), *args[3:], **kw),
        lambda: pd.pd_attn_chunk(b.q, *args[:5], i32([0]), **kw),
    ]
    for call in bad:
        with pytest.raises(pd.PdError):
            call()
