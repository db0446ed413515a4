"""pd_kv_append_quant against the definition in 64 bits: every 8-bit value and every scale equal."""
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


class Cache:
    """Pools with something in every slot, page lists of `kv` tokens a request, new rows."""

    def __init__(self, seed, new, kv, heads, d, page, block, dt, layout="HND", spare=2):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.new, self.kv, self.layout, self.page, self.block = new, kv, layout, page, block
        pages = [ref.ceil_div(n, page) for n in kv]
        self.qo = [sum(new[:i]) for i in range(len(new) + 1)]
        self.pp = [sum(pages[:i]) for i in range(len(new) + 1)]
        num = sum(pages) + spare
        self.px = torch.randperm(num, device="cuda", generator=g)[:sum(pages)].to(torch.int32)
        shape = (num, heads, page, d) if layout == "HND" else (num, page, heads, d)
        rnd = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
        self.k, self.v = ((rnd(*shape) * 60).clamp(-448, 448).to(E4M3) for _ in range(2))
        self.ks, self.vs = (torch.exp2(torch.randint(-12, -4, (num, heads, page // block), device="cuda", generator=g)
                                       .float()) for _ in range(2))
        size = torch.exp(1.5 * rnd(sum(new), heads, 1))
        self.kn, self.vn = ((rnd(sum(new), heads, d) * size).to(dt) for _ in range(2))

    def want(self):
        lists = (self.qo, self.kv, self.pp, self.px.tolist(), self.page, self.block, self.layout)
        return (*qref.append(self.kn, self.k, self.ks, *lists), *qref.append(self.vn, self.v, self.vs, *lists))

    def run(self, **kw):
        status = i32([0])
        args = dict(max_kv_len=max(self.kv), layout=self.layout, dev_status=status)
        args.update(kw)
        pd.pd_kv_append_quant(args.pop("kn", self.kn), args.pop("vn", self.vn), self.k, self.v, self.ks, self.vs,
                              i32(self.qo), i32(self.kv), i32(self.pp), self.px, **args)
        torch.cuda.synchronize()
        assert int(status.item()) == 0

    def check(self, want):
        k, ks, v, vs = want
        for got, ex in ((self.k, k), (self.v, v)):
            assert torch.equal(torch.nan_to_num(got.double(), nan=1e6), torch.nan_to_num(ex, nan=1e6))
        assert torch.equal(self.ks.double(), ks) and torch.equal(self.vs.double(), vs)


@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("layout", ["HND", "NHD"])
@pytest.mark.parametrize("heads,d,page,block", [(2, 128, 16, 16), (3, 64, 32, 16), (1, 128, 64, 64), (5, 64, 24, 8),
                                                (2, 64, 6, 3), (2, 40, 20, 4), (1, 64, 1, 1), (1, 256, 256, 256),
                                                (1, 128, 512, 512)])
def test_ragged_batches(dt, layout, heads, d, page, block):
    new = [1, 0, 17, 64, 100, 3, 1, 33, 0]
    kv = [1, 40, 30, 64, 333, 700, 65, 47, 0]
    c = Cache(1, new, kv, heads, d, page, block, dt, layout)
    want = c.want()
    c.run()
    c.check(want)
    c.run()  # again: the same cache
    c.check(want)


@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("seed", range(4))
def test_drawn(dt, seed):
    rng = random.Random(seed)
    new = [rng.choice([0, 1, 1, 2, rng.randint(1, 120)]) for _ in range(rng.randint(1, 70))]
    new[0] = max(new[0], 1)
    kv = [n + rng.choice([0, rng.randint(0, 90)]) for n in new]
    page = rng.choice([16, 32, 64])
    c = Cache(seed, new, kv, rng.choice([1, 4, 8]), rng.choice([64, 128]), page, rng.choice([8, 16, page]), dt,
              rng.choice(["HND", "NHD"]))
    want = c.want()
    c.run()
    c.check(want)


@pytest.mark.parametrize("dt", [BF16, F32])
def test_token_by_token_as_a_decode_appends(dt):
    # 40 tokens one after another into blocks of 16; the scales only grow, and earlier values follow
    c = Cache(3, [1, 1, 1], [5, 16, 33], 4, 128, 32, 16, dt)
    c.pp, c.px = [0, 4, 8, 12], torch.randperm(14, device="cuda")[:12].to(torch.int32)
    c.k, c.v, c.ks, c.vs = (torch.cat([t.view(torch.uint8) if t.dtype == E4M3 else t] * 4)[:14].contiguous()
                            for t in (c.k, c.v, c.ks, c.vs))
    c.k, c.v = c.k.view(E4M3), c.v.view(E4M3)
    g = torch.Generator(device="cuda").manual_seed(4)
    for i in range(40):
        for t in (c.kn, c.vn):
            t.copy_(torch.randn(t.shape, device="cuda", generator=g) * 2.0 ** (i % 7))
        want = c.want()
        c.run()
        c.check(want)
        c.kv = [n + 1 for n in c.kv]


@pytest.mark.parametrize("dt", [BF16, F32])
def test_special_values(dt):
    c = Cache(5, [20, 3, 16, 2], [20, 20, 16, 18], 2, 64, 16, 16, dt)
    c.kn[0, 0, 5], c.kn[1, 0, 6], c.kn[2, 1, 7] = float("nan"), float("inf"), -float("inf")
    c.kn[23:39] = 0.0                      # a block of zeros
    c.vn[:16] = 0.0
    c.vn[16:20] *= 1e-37                   # below the smallest scale
    c.vn[20:23] = 3e38                     # and far up
    c.vn[23:39] = float("nan")             # nothing finite
    c.kn[39:] = torch.tensor([448.0, -448.0], device="cuda").to(dt).repeat(32)  # exactly the largest value
    c.vn[39, :, 0] = 449.0 if dt == F32 else 450.0
    want = c.want()
    c.run()
    c.check(want)


def test_the_callers_own_scales_need_not_be_powers_of_two():
    c = Cache(6, [3, 5], [20, 30], 2, 64, 16, 16, F32)
    c.ks *= 1.3
    c.vs *= 300.0  # large: kept, and the new values are divided by it
    want = c.want()
    c.run()
    k, ks, v, vs = want
    # x / s goes through one fp32 division before it is rounded: next to a tie it may take the other side,
    # one step in 2^16 or so of the values; scales are equal
    assert torch.equal(c.ks.double(), ks) and torch.equal(c.vs.double(), vs)
    for got, ex in ((c.k, k), (c.v, v)):
        off = (got.double() - ex).abs()
        assert bool((off <= 2.0 ** -3 * ex.abs().clamp(min=2.0 ** -6)).all()) and int((off > 0).sum()) <= 2


@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("layout", ["HND", "NHD"])
def test_slices_rows_behind_the_last_and_bytes(dt, layout):
    c = Cache(7, [20, 7], [45, 7], 4, 64, 16, 8, dt, layout)
    wide = torch.full((40, 16 * 64), float("nan"), device="cuda").to(dt)
    kn, vn = (wide[:, a * 64:(a + 4) * 64].view(40, 4, 64) for a in (2, 8))
    kn[:27], vn[:27] = c.kn, c.vn
    want = c.want()
    c.k, c.v = c.k.view(torch.uint8), c.v.view(torch.uint8)  # pools as bytes
    c.run(kn=kn, vn=vn)
    c.k, c.v = c.k.view(E4M3), c.v.view(E4M3)
    c.check(want)


def test_bad_requests_are_skipped_and_reported():
    def call(rows, **kw):
        """Runs with the changes; the requests `rows` are as they should be, the pages of the others untouched
        (with `px`: the page that it lost)."""
        c = Cache(8, [5, 6, 7], [50, 60, 70], 2, 64, 16, 16, BF16)
        before = [t.clone() for t in (c.k.view(torch.uint8), c.ks)]
        want = c.want()
        qo, kv, pp, px = (kw.get(n, x) for n, x in (("qo", c.qo), ("kv", c.kv), ("pp", c.pp), ("px", c.px)))
        status = i32([0])
        pd.pd_kv_append_quant(c.kn, c.vn, c.k, c.v, c.ks, c.vs, i32(qo), i32(kv), i32(pp), px, max_kv_len=70,
                              dev_status=status)
        torch.cuda.synchronize()
        for r in range(3):
            ids = c.px[c.pp[r]:c.pp[r + 1]].long()
            if r in rows:
                assert torch.equal(c.k[ids].double(), want[0][ids]) and torch.equal(c.ks[ids].double(), want[1][ids])
            else:
                ids = ids[-1:] if "px" in kw else ids
                assert torch.equal(c.k.view(torch.uint8)[ids], before[0][ids]) and torch.equal(c.ks[ids], before[1][ids])
        return int(status.item())

    c = Cache(8, [5, 6, 7], [50, 60, 70], 2, 64, 16, 16, BF16)
    assert call([0, 1, 2]) == 0
    assert call([1, 2], kv=[4, 60, 70]) == 2          # fewer tokens than new ones
    assert call([0, 1], kv=[50, 60, 71]) == 2
    assert call([1, 2], kv=[-1, 60, 70]) == 2
    assert call([0, 1], qo=[0, 5, 11, 19]) == 1       # rows past k_new
    px = c.px.clone()
    px[3] = 10 ** 6
    assert call([1, 2], px=px) == 3
    px[3] = -1
    assert call([1, 2], px=px) == 3


def test_streams_and_a_graph():
    a, b = Cache(9, [1] * 9, [1 + 7 * i for i in range(9)], 8, 128, 16, 16, BF16), Cache(10, [90], [200], 8, 128, 64,
                                                                                         32, BF16)
    wa, wb = a.want(), b.want()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    args = [(c.kn, c.vn, c.k, c.v, c.ks, c.vs, i32(c.qo), i32(c.kv), i32(c.pp), c.px) for c in (a, b)]
    torch.cuda.synchronize()
    for _ in range(3):
        pd.pd_kv_append_quant(*args[0], max_kv_len=70, stream=s1)
        pd.pd_kv_append_quant(*args[1], max_kv_len=200, stream=s2.cuda_stream)
    torch.cuda.synchronize()
    a.check(wa)
    b.check(wb)
    # captured, replayed with other lengths and values
    with torch.cuda.stream(s1):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s1):
            pd.pd_kv_append_quant(*args[0], max_kv_len=70)
    for i in range(3):
        a.kv = [max(1, n - 3) for n in a.kv]
        args[0][7].copy_(i32(a.kv))
        a.kn *= 1.7
        want = a.want()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        a.check(want)


def test_lengths_are_read_back_without_a_bound():
    c = Cache(11, [3], [40], 2, 64, 16, 16, BF16)
    want = c.want()
    c.run(max_kv_len=None)
    c.check(want)


def test_pool_past_32_bit_offsets():
    heads, d, page = 8, 128, 64
    pages = (1 << 32) // (heads * page * d) + 40
    k, v = (torch.zeros(pages, heads, page, d, dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.zeros(pages, heads, 4, device="cuda") for _ in range(2))
    px = i32([pages - 1, 0, pages - 2])
    g = torch.Generator(device="cuda").manual_seed(12)
    kn, vn = (torch.randn(150, heads, d, device="cuda", generator=g).to(BF16) for _ in range(2))
    for layout in ("HND", "NHD"):
        kk, vv = (x if layout == "HND" else x.view(pages, page, heads, d) for x in (k, v))
        pd.pd_kv_append_quant(kn, vn, kk, vv, ks, vs, i32([0, 150]), i32([170]), i32([0, 3]), px, max_kv_len=170,
                              layout=layout)
        got = ref.gather(qref.dequant(kk[px.long()], ks[px.long()], layout), torch.arange(3, device="cuda"), 170, layout)
        # off by half a step of e4m3, of a value or of its block's smallest step: 2^-10 of a scale <= 2^-6
        assert bool(((got[20:] - kn.double()).abs() <= 2.0 ** -4 * kn.double().abs() + 2.0 ** -16).all())


def test_refusals():
    c = Cache(13, [4], [40], 2, 64, 16, 16, F32)
    lists = (i32(c.qo), i32(c.kv), i32(c.pp), c.px)
    bad = [
        (c.kn.half(), c.vn, c.k, c.v, c.ks, c.vs, *lists),
        (c.kn, c.vn.bfloat16(), c.k, c.v, c.ks, c.vs, *lists),
        (c.kn[:, :1], c.vn[:, :1], c.k, c.v, c.ks, c.vs, *lists),
        (c.kn, c.vn, c.k.float(), c.v.float(), c.ks, c.vs, *lists),
        (c.kn, c.vn, c.k, c.v, c.ks.double(), c.vs, *lists),
        (c.kn, c.vn, c.k, c.v, c.ks[:, :1], c.vs, *lists),
        (c.kn, c.vn, c.k, c.v, c.ks.repeat(1, 1, 3), c.vs, *lists),
        (c.kn, c.vn, c.k, c.v, c.ks.repeat(1, 1, 2), c.vs, *lists),
        (c.kn, c.vn, c.k, c.v, c.ks, c.vs, i32([0]), *lists[1:]),
        (c.kn.expand(4, 2, 64)[:1].expand(4, 2, 64), c.vn, c.k, c.v, c.ks, c.vs, *lists),
        (c.kn.cpu(), c.vn, c.k, c.v, c.ks, c.vs, *lists),
    ]
    for args in bad:
        with pytest.raises(pd.PdError):
            pd.pd_kv_append_quant(*args, max_kv_len=40)
