"""pd_qk_norm_rope and pd_qk_norm_rope_append against fp64: every value within its own bound
(step_ref.norm_rope_bound), copies bit for bit, everything else left as it was."""
import pytest
import torch

import step_ref as ref

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import decode_ragged_paged_gb300 as pd

F32, BF16 = torch.float32, torch.bfloat16


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def freqs(rope, base=10000.0):
    half = rope // 2
    return (base ** (-torch.arange(half, device="cuda", dtype=torch.float64) / half)).float() if rope else None


def check(got, x, w, inv_freq, pos, eps, interleaved):
    want, size = ref.norm_rope(x, w, inv_freq, pos, eps=eps, interleaved=interleaved)
    err = (got.double() - want).abs()
    lim = ref.norm_rope_bound(want, size, got.dtype)
    assert bool((err <= lim).all()), f"worst error / bound {float((err / lim.clamp(min=1e-300)).max())}"


CASES = [
    # tokens, hq, hkv, dim, rope, interleaved, dtype
    (1, 8, 2, 128, 128, False, BF16),
    (1, 1, 1, 64, 64, True, F32),
    (5, 32, 8, 128, 128, False, BF16),
    (130, 32, 8, 128, 128, True, BF16),
    (333, 40, 40, 128, 128, False, BF16),
    (77, 28, 4, 128, 64, False, BF16),       # half of each head rotated
    (77, 28, 4, 128, 32, True, BF16),
    (64, 5, 1, 64, 16, False, F32),
    (64, 7, 7, 80, 40, False, BF16),         # runs of 4: 10 lanes of 16 a head
    (33, 3, 2, 96, 96, True, F32),
    (33, 3, 3, 100, 20, False, BF16),        # runs of 2
    (33, 4, 2, 192, 64, False, BF16),
    (33, 4, 2, 256, 256, True, BF16),
    (33, 4, 2, 256, 128, False, F32),
    (9, 2, 1, 512, 512, False, BF16),
    (9, 2, 1, 4, 4, True, BF16),
    (21, 6, 3, 128, 0, False, BF16),         # norms alone
    (3000, 16, 4, 128, 128, False, BF16),
]


@pytest.mark.parametrize("t,hq,hkv,d,rope,interleaved,dt", CASES)
def test_rows(t, hq, hkv, d, rope, interleaved, dt):
    g = gen(t + d)
    q, k = (torch.randn(t, h, d, device="cuda", generator=g).to(dt) for h in (hq, hkv))
    qw, kw = ((1 + 0.3 * torch.randn(d, device="cuda", generator=g)).to(dt) for _ in range(2))
    pos = torch.randint(0, 1 << 20, (t,), device="cuda", generator=g, dtype=torch.int32)
    f = freqs(rope)
    qo, ko = pd.pd_qk_norm_rope(q, k, qw, kw, f, pos if rope else None, eps=1e-5, interleaved=interleaved)
    check(qo, q, qw, f, pos, 1e-5, interleaved)
    check(ko, k, kw, f, pos, 1e-5, interleaved)
    # without weights: rotation alone
    qo, ko = pd.pd_qk_norm_rope(q, k, None, kw, f, pos if rope else None, eps=1e-5, interleaved=interleaved)
    check(qo, q, None, f, pos, 1e-5, interleaved)
    check(ko, k, kw, f, pos, 1e-5, interleaved)


@pytest.mark.parametrize("layout,page", [("HND", 16), ("NHD", 16), ("HND", 1), ("NHD", 24), ("HND", 7)])
@pytest.mark.parametrize("t,hq,hkv,d,rope,interleaved,dt", CASES[2:10])
def test_append(layout, page, t, hq, hkv, d, rope, interleaved, dt):
    g = gen(3 * t + d)
    row = torch.randn(t, (hq + 2 * hkv) * d, device="cuda", generator=g).to(dt)  # a fused projection's rows
    q, k, v = (x.view(t, -1, d) for x in row.split([hq * d, hkv * d, hkv * d], 1))
    before = row.clone()
    qw, kw = ((1 + 0.3 * torch.randn(d, device="cuda", generator=g)).to(dt) for _ in range(2))
    pos = torch.randint(0, 40000, (t,), device="cuda", generator=g, dtype=torch.int32)
    f = freqs(rope)
    pages = t // page + 3
    shape = (pages, hkv, page, d) if layout == "HND" else (pages, page, hkv, d)
    kp, vp = (torch.randn(shape, device="cuda", generator=g).to(dt) for _ in range(2))
    kp0, vp0 = kp.clone(), vp.clone()
    slot = torch.randperm(pages * page, device="cuda", generator=g)[:t].contiguous()
    pad = torch.rand(t, device="cuda", generator=g) < 0.2
    slot[pad] = -1
    q_out = torch.full((t, hq, d), 7.0, device="cuda").to(dt)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = pd.pd_qk_norm_rope_append(q, k, v, qw, kw, f, pos, slot, kp, vp, eps=1e-6, interleaved=interleaved,
                                    q_out=q_out, dev_status=status, layout=layout)
    assert out is q_out and int(status.item()) == 0 and torch.equal(row, before)
    real = ~pad
    check(q_out[real], q[real], qw, f, pos[real], 1e-6, interleaved)
    assert bool((q_out[pad] == 7.0).all())

    def rows_of(pool):  # [pages * page][hkv][d], a copy
        return (pool.transpose(1, 2) if layout == "HND" else pool).reshape(-1, hkv, d)

    s = slot[real]
    check(rows_of(kp)[s], k[real], kw, f, pos[real], 1e-6, interleaved)
    assert torch.equal(rows_of(vp)[s], v[real])
    others = torch.ones(pages * page, dtype=torch.bool, device="cuda")
    others[s] = False
    assert torch.equal(rows_of(kp)[others], rows_of(kp0)[others])
    assert torch.equal(rows_of(vp)[others], rows_of(vp0)[others])


def test_in_place_and_odd_alignment():
    g = gen(5)
    for dt, d, off in ((BF16, 128, 4), (BF16, 64, 2), (F32, 64, 2), (BF16, 128, 8)):
        buf = torch.randn(50 * (6 * d + 2 * off) + off, device="cuda", generator=g).to(dt)
        x = buf[off:off + 50 * (6 * d + 2 * off)].view(50, 6 * d + 2 * off)  # rows and base off 16 bytes
        q, k = x[:, :4 * d].view(50, 4, d), x[:, 4 * d:6 * d].view(50, 2, d)
        q0, k0, rest = q.clone(), k.clone(), x[:, 6 * d:].clone()
        pos = torch.arange(50, device="cuda", dtype=torch.int32)
        w = torch.ones(d + 8, device="cuda").to(dt)[8:]
        qo, ko = pd.pd_qk_norm_rope(q, k, w, w, freqs(d), pos, q_out=q, k_out=k)
        assert qo.data_ptr() == q.data_ptr()
        check(q, q0, w, freqs(d), pos, 1e-6, False)
        check(k, k0, w, freqs(d), pos, 1e-6, False)
        assert torch.equal(x[:, 6 * d:], rest)


def test_far_and_negative_positions():
    q = torch.randn(6, 2, 64, device="cuda", generator=gen(6))
    pos = torch.tensor([0, 1, 2 ** 24 + 1, 2 ** 27 + 3, -5, -2 ** 27], device="cuda", dtype=torch.int32)
    for f in (freqs(64), freqs(64, 500000.0), -freqs(64), 100 * freqs(64)):
        for inter in (False, True):
            qo, _ = pd.pd_qk_norm_rope(q, q[:, :1], None, None, f, pos, interleaved=inter)
            want, size = ref.norm_rope(q, None, f, pos, eps=0, interleaved=inter)
            # an angle is off by position * 2^-52 of its frequency beside the bound's own 2^-24s
            angle = (pos.double().abs()[:, None, None] * f.abs().double().max()) * 2.0 ** -51
            assert bool(((qo.double() - want).abs() <= ref.norm_rope_bound(want, size, F32) + angle * size).all())


def test_values_at_the_ends_of_the_range():
    x = torch.zeros(4, 1, 64, device="cuda")
    x[1] = 1e-30
    x[2, 0, 3] = float("nan")
    x[3] = 1e18
    pos = torch.arange(4, device="cuda", dtype=torch.int32)
    w = torch.ones(64, device="cuda")
    qo, ko = pd.pd_qk_norm_rope(x, x, w, None, freqs(64), pos)
    assert bool((qo[0] == 0).all()) and bool(qo[2].isnan().all())
    want, size = ref.norm_rope(x[[1, 3]], w, freqs(64), pos[[1, 3]], eps=1e-6, interleaved=False)
    assert bool(((qo[[1, 3]].double() - want).abs() <= ref.norm_rope_bound(want, size, F32)).all())
    clean = [e for e in range(64) if e not in (3, 35)]
    assert bool(ko[2, 0, clean].eq(0).all())  # without a norm a value touches its own pair only


def test_slots_past_the_pools_are_reported():
    q = torch.randn(3, 4, 64, device="cuda")
    kp = torch.zeros(2, 4, 16, 64, device="cuda")
    vp = torch.zeros_like(kp)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    slot = torch.tensor([31, 32, 2 ** 40], device="cuda")
    pos = torch.arange(3, device="cuda", dtype=torch.int32)
    out = pd.pd_qk_norm_rope_append(q, q, q, None, None, freqs(64), pos, slot, kp, vp, dev_status=status)
    assert int(status.item()) == 3
    check(out, q, None, freqs(64), pos, 0.0, False)
    assert torch.equal(vp[1, :, 15], q[0]) and int((vp != 0).sum()) == q[0].numel()


def test_pools_past_32_bit_offsets():
    d, hkv, page = 128, 8, 64
    pages = (1 << 32) // (hkv * page * d) + 2   # past 2^32 elements
    kp, vp = (torch.empty(pages, hkv, page, d, dtype=BF16, device="cuda") for _ in range(2))
    q = torch.randn(4, 8, d, device="cuda", generator=gen(8)).to(BF16)
    slot = torch.tensor([0, pages * page - 1, (pages - 1) * page, page - 1], device="cuda")
    for layout in ("HND", "NHD"):
        kq, vq = (kp, vp) if layout == "HND" else (kp.view(pages, page, hkv, d), vp.view(pages, page, hkv, d))
        pd.pd_qk_norm_rope_append(q, q, q, None, None, None, None, slot, kq, vq, layout=layout)
        for i, s in enumerate(slot.tolist()):
            row = (kq[s // page, :, s % page], vq[s // page, :, s % page]) if layout == "HND" else (
                kq[s // page, s % page], vq[s // page, s % page])
            assert torch.equal(row[0], q[i]) and torch.equal(row[1], q[i])


def test_a_stream_of_its_own_and_a_graph():
    g = gen(9)
    q = torch.randn(200, 8, 128, device="cuda", generator=g).to(BF16)
    k = torch.randn(200, 2, 128, device="cuda", generator=g).to(BF16)
    w = torch.ones(128, device="cuda").to(BF16)
    f = freqs(128)
    pos = torch.arange(200, device="cuda", dtype=torch.int32)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    qo, ko = pd.pd_qk_norm_rope(q, k, w, w, f, pos, stream=s)
    s.synchronize()
    check(qo, q, w, f, pos, 1e-6, False)
    with torch.cuda.stream(s):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            pd.pd_qk_norm_rope(q, k, w, w, f, pos, q_out=qo, k_out=ko)
    pos += 1000
    q.mul_(2)
    torch.cuda.synchronize()
    graph.replay()
    torch.cuda.synchronize()
    check(qo, q, w, f, pos, 1e-6, False)


def test_refusals():
    q = torch.randn(4, 8, 64, device="cuda")
    pos = torch.arange(4, device="cuda", dtype=torch.int32)
    pool, slot = torch.zeros(2, 8, 16, 64, device="cuda"), torch.arange(4, device="cuda")
    bad = [
        lambda: pd.pd_qk_norm_rope(q, q[:3], None, None, freqs(64), pos),
        lambda: pd.pd_qk_norm_rope(q, q.bfloat16(), None, None, freqs(64), pos),
        lambda: pd.pd_qk_norm_rope(q, q, torch.ones(32, device="cuda"), None, freqs(64), pos),
        lambda: pd.pd_qk_norm_rope(q, q, None, None, freqs(64), pos[:3]),
        lambda: pd.pd_qk_norm_rope(q, q, None, None, freqs(64), pos.long()),
        lambda: pd.pd_qk_norm_rope(q, q, None, None, freqs(128), pos),
        lambda: pd.pd_qk_norm_rope(q.transpose(0, 1), q, None, None, freqs(64), pos),
        lambda: pd.pd_qk_norm_rope(q, q, None, None, freqs(64), pos, q_out=q[:, :4]),
        lambda: pd.pd_qk_norm_rope_append(q, q, q, None, None, freqs(64), pos, slot.int(), pool, pool),
        lambda: pd.pd_qk_norm_rope_append(q, q, q, None, None, freqs(64), pos, slot, pool[:, :4], pool),
        lambda: pd.pd_qk_norm_rope_append(q, q, q, None, None, freqs(64), pos, slot, pool, pool, layout="NHD"),
        lambda: pd.pd_qk_norm_rope_append(q, q, q[:, :2], None, None, freqs(64), pos, slot, pool, pool),
    ]
    for call in bad:
        with pytest.raises(pd.PdError):
            call()


def test_tokens_that_are_one_row_are_refused():
    # a broadcast row's stride of 0 would be read as rows one after another
    one, q = torch.randn(1, 8, 64, device="cuda").expand(4, 8, 64), torch.randn(4, 8, 64, device="cuda")
    pos = torch.arange(4, device="cuda", dtype=torch.int32)
    pool, slot = torch.zeros(2, 8, 16, 64, device="cuda"), torch.arange(4, device="cuda")
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    for call in (lambda: pd.pd_qk_norm_rope(one, q, None, None, freqs(64), pos),
                 lambda: pd.pd_qk_norm_rope(q, one, None, None, freqs(64), pos),
                 lambda: pd.pd_qk_norm_rope(q, q, None, None, freqs(64), pos, q_out=one),
                 lambda: pd.pd_qk_norm_rope_append(q, q, one, None, None, freqs(64), pos, slot, pool, pool),
                 lambda: pd.pd_attn_chunk(one, pool, pool, i32([4]), i32([0, 1]), i32([0]), i32([0, 4]), max_qo_len=4,
                                          max_kv_len=4)):
        with pytest.raises(pd.PdError):
            call()
    got, _ = pd.pd_qk_norm_rope(one[:1], q[:1], None, None, None, None)
    assert torch.equal(got, one[:1])
