"""pd_qk_norm_rope_axes and its append against the formula in 64 bits, within the bound of the form with one
position a token (step_ref.norm_rope_bound: the arithmetic is the same)."""
import pytest
import torch

import step_ref as ref

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import decode_ragged_paged_gb300 as pd

F32, BF16 = torch.float32, torch.bfloat16


def axes_ref(x, w, inv_freq, axes, positions, *, eps, interleaved):
    """step_ref.norm_rope, a frequency at a time: each turns by its own axis's positions."""
    y, size = ref.norm_rope(x, w, None, None, eps=eps, interleaved=interleaved)
    half = inv_freq.numel()
    out = y.clone()
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, half + i)
        t = (positions[axes[i]].double() * inv_freq[i].double())[:, None]
        out[..., a] = y[..., a] * t.cos() - y[..., b] * t.sin()
        out[..., b] = y[..., a] * t.sin() + y[..., b] * t.cos()
        size[..., a] = size[..., b] = torch.hypot(y[..., a], y[..., b])
    return out, size


def make(seed, T, hq, hkv, d, rope, A, dt, far=200000):
    g = torch.Generator(device="cuda").manual_seed(seed)
    q, k, v = (torch.randn(T, h, d, device="cuda", generator=g).to(dt) for h in (hq, hkv, hkv))
    w = [(1 + 0.2 * torch.randn(d, device="cuda", generator=g)).to(dt) for _ in range(2)]
    inv_freq = (10000.0 ** (-torch.arange(rope // 2, device="cuda", dtype=torch.float64) / (rope // 2))).float()
    pos = torch.randint(0, far, (A, T), generator=g, device="cuda", dtype=torch.int32)
    return q, k, v, *w, inv_freq, pos


def check(got, x, w, inv_freq, axes, pos, dt, interleaved):
    want, size = axes_ref(x, w, inv_freq, axes, pos, eps=1e-6, interleaved=interleaved)
    assert bool(((got.double() - want).abs() <= ref.norm_rope_bound(want, size, dt)).all())


def runs(half, sizes):
    out = sum(([a] * n for a, n in enumerate(sizes)), [])
    return (out + [len(sizes) - 1] * half)[:half]


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("hq,hkv,d,rope", [(8, 2, 128, 128), (3, 1, 64, 64), (28, 4, 128, 64), (2, 2, 256, 256),
                                           (1, 1, 20, 12), (5, 5, 512, 512)])
@pytest.mark.parametrize("T,A,pattern", [(1, 3, "runs"), (33, 3, "turns"), (700, 2, "runs"), (97, 4, "turns"),
                                         (40, 1, "runs")])
def test_rotation(dt, interleaved, hq, hkv, d, rope, T, A, pattern):
    if dt == F32 and d == 512:
        d, rope = 256, 256  # (a head is 64 of its widest vectors at most)
    q, k, _, qw, kw, f, pos = make(T, T, hq, hkv, d, rope, A, dt)
    half = rope // 2
    axes = [i % A for i in range(half)] if pattern == "turns" else runs(half, [half // 4, half // 3, half, 1][:A])
    qo, ko = pd.pd_qk_norm_rope_axes(q, k, qw, kw, f, axes, pos, interleaved=interleaved)
    check(qo, q, qw, f, axes, pos, dt, interleaved)
    check(ko, k, kw, f, axes, pos, dt, interleaved)
    qi, ki = q.clone(), k.clone()  # in place, and without weights
    pd.pd_qk_norm_rope_axes(qi, ki, None, kw, f, bytes(axes), pos, interleaved=interleaved, q_out=qi, k_out=ki)
    check(qi, q, None, f, axes, pos, dt, interleaved)
    assert torch.equal(ki, ko)


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("layout", ["HND", "NHD"])
def test_append(dt, layout):
    T, hq, hkv, d, page = 130, 8, 2, 128, 16
    q, k, v, qw, kw, f, pos = make(2, T, hq, hkv, d, d, 3, dt)
    axes = bytes([0] * 16 + [1] * 24 + [2] * 24)
    shape = (20, hkv, page, d) if layout == "HND" else (20, page, hkv, d)
    kp, vp = (torch.full(shape, 7.0, device="cuda").to(dt) for _ in range(2))
    slots = torch.randperm(20 * page, device="cuda")[:T]
    slots[5], slots[T - 1] = -1, -1  # padding rows
    q_out = torch.full_like(q, 7.0)
    pd.pd_qk_norm_rope_axes_append(q, k, v, qw, kw, f, axes, pos, slots, kp, vp, q_out=q_out, layout=layout)
    real = slots >= 0
    check(q_out[real], q[real], qw, f, axes, pos[:, real], dt, False)
    assert bool((q_out[~real] == 7).all())
    rows = lambda p: (p.transpose(1, 2) if layout == "HND" else p).reshape(-1, hkv, d)  # noqa: E731
    check(rows(kp)[slots[real]], k[real], kw, f, axes, pos[:, real], dt, False)
    assert torch.equal(rows(vp)[slots[real]], v[real])
    free = torch.ones(20 * page, dtype=torch.bool, device="cuda")
    free[slots[real]] = False
    assert bool((rows(kp)[free] == 7).all()) and bool((rows(vp)[free] == 7).all())


def test_one_axis_and_equal_axes_are_the_form_with_one_position():
    q, k, v, qw, kw, f, pos = make(3, 200, 32, 8, 128, 128, 3, BF16)
    want = pd.pd_qk_norm_rope(q, k, qw, kw, f, pos[0])
    same = pos[:1].expand(3, -1)  # a stride of 0 between the axes
    for axes, p in ((bytes(64), pos[:1]), ([i % 3 for i in range(64)], same), (bytes(64), pos)):
        got = pd.pd_qk_norm_rope_axes(q, k, qw, kw, f, axes, p)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_strided_rows_and_positions():
    T, d = 50, 64
    q, k, v, qw, kw, f, pos = make(4, T, 6, 2, d, d, 3, BF16)
    wide = torch.zeros(T, 10 * d, device="cuda").to(BF16)
    qs, ks = wide[:, :6 * d].view(T, 6, d), wide[:, 6 * d:8 * d].view(T, 2, d)
    qs.copy_(q), ks.copy_(k)
    more = torch.full((3, T + 13), -5, dtype=torch.int32, device="cuda")
    more[:, :T] = pos
    axes = [i % 3 for i in range(d // 2)]
    want = pd.pd_qk_norm_rope_axes(q, k, qw, kw, f, axes, pos)
    got = pd.pd_qk_norm_rope_axes(qs, ks, qw, kw, f, axes, more[:, :T])
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_negative_and_far_positions():
    q, k, v, qw, kw, f, pos = make(5, 64, 4, 4, 128, 128, 3, F32)
    pos[0, :8], pos[1, :8], pos[2, :8] = -3, 2 ** 31 - 1, -2 ** 31
    axes = runs(64, [20, 20, 24])
    got, _ = pd.pd_qk_norm_rope_axes(q, k, qw, kw, f, axes, pos)
    want, size = axes_ref(q, qw, f, axes, pos, eps=1e-6, interleaved=False)
    # an angle is off by at most 2^31 * (2^-52 + 2 pi 2^-64) and fp64's own cosine by about as much: 2^-20 of the size
    assert bool(((got.double() - want).abs() <= ref.norm_rope_bound(want, size, F32) + 2.0 ** -20 * size).all())


def test_graph_and_stream():
    q, k, v, qw, kw, f, pos = make(6, 90, 8, 2, 128, 128, 3, BF16)
    axes = bytes([0] * 16 + [1] * 24 + [2] * 24)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = pd.pd_qk_norm_rope_axes(q, k, qw, kw, f, axes, pos, stream=s)
    torch.cuda.synchronize()
    check(got[0], q, qw, f, axes, pos, BF16, False)
    qo, ko = torch.zeros_like(q), torch.zeros_like(k)
    with torch.cuda.stream(s):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            pd.pd_qk_norm_rope_axes(q, k, qw, kw, f, axes, pos, q_out=qo, k_out=ko)
    pos += 17
    torch.cuda.synchronize()
    graph.replay()
    torch.cuda.synchronize()
    check(qo, q, qw, f, axes, pos, BF16, False)


def test_refusals():
    q, k, v, qw, kw, f, pos = make(7, 10, 4, 2, 64, 64, 3, BF16)
    good = [0] * 32
    bad = [
        lambda: pd.pd_qk_norm_rope_axes(q, k, qw, kw, f, [0] * 31, pos),
        lambda: pd.pd_qk_norm_rope_axes(q, k, qw, kw, f, [3] * 32, pos),
        lambda: pd.pd_qk_norm_rope_axes(q, k, qw, kw, f, [-1] * 32, pos),
        lambda: pd.pd_qk_norm_rope_axes(q, k, qw, kw, f, 32, pos),
        lambda: pd.pd_qk_norm_rope_axes(q, k, qw, kw, None, good, pos),
        lambda: pd.pd_qk_norm_rope_axes(q, k, qw, kw, f, good, pos[0]),
        lambda: pd.pd_qk_norm_rope_axes(q, k, qw, kw, f, good, pos[:, :9]),
        lambda: pd.pd_qk_norm_rope_axes(q, k, qw, kw, f, good, pos.long()),
        lambda: pd.pd_qk_norm_rope_axes(q, k, qw, kw, f, good, pos.T.contiguous().T),
        lambda: pd.pd_qk_norm_rope_axes(q, k, qw, kw, f, good, pos.repeat(2, 1)),
        lambda: pd.pd_qk_norm_rope_axes(q, k, qw, kw, f, good, None),
    ]
    for call in bad:
        with pytest.raises(pd.PdError):
            call()
