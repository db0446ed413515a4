"""A serving step over a cache held in 8 bits, as it is used: tables from lengths, norm and rotation with a
time, a height and a width, append to the 8-bit pages, attention of the new tokens; over several steps of a ragged
batch, and captured. Each call against its 64-bit form over what the calls before it left."""
import ctypes
import random
import subprocess
import threading

import pytest
import torch

import quant_ref as qref
import step_ref as ref
from test_gpu_axes import axes_ref

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import decode_ragged_paged_gb300 as pd

F32, BF16, E4M3 = torch.float32, torch.bfloat16, torch.float8_e4m3fn


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("dt,hq,hkv,d,page,block,layout,window,captured,most", [
    (F32, 8, 2, 64, 16, 4, "HND", -1, False, 100),
    (BF16, 32, 8, 128, 16, 16, "HND", -1, False, 100),
    (BF16, 4, 4, 128, 64, 32, "NHD", 50, False, 100),
    (BF16, 28, 4, 128, 16, 8, "HND", -1, True, 100),
    (BF16, 8, 2, 64, 24, 24, "NHD", -1, True, 100),
    (BF16, 8, 4, 128, 32, 16, "HND", -1, True, 3),    # a token or a few drafted ones a request
    (BF16, 8, 1, 64, 16, 16, "NHD", 40, True, 1),
])
def test_steps(dt, hq, hkv, d, page, block, layout, window, captured, most):
    g = torch.Generator(device="cuda").manual_seed(1)
    rng = random.Random(2)
    B, steps, cap = 9, 6, 260
    plan = [[min(most, rng.choice([0, 1, 1, 3, 40])) for _ in range(B)] for _ in range(steps)]
    plan[0] = [min(most, n) for n in (1, 100, 17, 16, 0, 33, 2, 5, 64)]
    num_pages = sum(ref.ceil_div(sum(p[r] for p in plan), page) for r in range(B)) + 5
    shape = (num_pages, hkv, page, d) if layout == "HND" else (num_pages, page, hkv, d)
    kp, vp = (torch.full(shape, 0x7f, dtype=torch.uint8, device="cuda").view(E4M3) for _ in range(2))  # NaN
    ks, vs = (torch.full((num_pages, hkv, page // block), float("nan"), device="cuda") for _ in range(2))
    free = torch.randperm(num_pages, device="cuda", generator=g).to(torch.int32)
    count, table = i32([num_pages]), torch.full((B, 40), -1, dtype=torch.int32, device="cuda")
    cached, new = torch.zeros(B, dtype=torch.int32, device="cuda"), i32(plan[0])
    half = d // 2
    inv_freq = (10000.0 ** (-torch.arange(half, device="cuda", dtype=torch.float64) / half)).float()
    axes = [0] * (half // 4) + [1 + i % 2 for i in range(half - half // 4)]
    qw, kw = ((1 + 0.2 * torch.randn(d, device="cuda", generator=g)).to(dt) for _ in range(2))
    qkv = torch.zeros(cap, (hq + 2 * hkv) * d, device="cuda").to(dt)
    q, k, v = (x.view(cap, -1, d) for x in qkv.split([hq * d, hkv * d, hkv * d], 1))
    grid = torch.randint(0, 64, (2, cap), generator=g, device="cuda", dtype=torch.int32)  # height and width
    pos = torch.zeros(3, cap, dtype=torch.int32, device="cuda")
    status = i32([0])
    q_out, o = (torch.zeros(cap, hq, d, device="cuda").to(dt) for _ in range(2))
    k_out, lse = torch.zeros(cap, hkv, d, device="cuda").to(dt), torch.zeros(cap, hq, device="cuda")
    ws = torch.empty(128 << 20, dtype=torch.uint8, device="cuda")
    out = pd.BatchTables(*(torch.zeros(n, dtype=t, device="cuda") for n, t in (
        (B + 1, torch.int32), (B, torch.int32), (B + 1, torch.int32), (num_pages, torch.int32), (cap, torch.int32),
        (cap, torch.int64))))

    def step():
        t = pd.pd_batch_tables(new, cached, table, page_size=page, num_pages=num_pages, total_qo=cap,
                               max_page_indices=num_pages, free_pages=free, free_count=count, free_count_out=count,
                               out=out, dev_status=status)
        pos[0].copy_(t.positions)
        pos[1:].copy_(grid)
        pd.pd_qk_norm_rope_axes(q, k, qw, kw, inv_freq, axes, pos, q_out=q_out, k_out=k_out)
        pd.pd_kv_append_quant(k_out, v, kp, vp, ks, vs, t.qo_indptr, t.kv_len, t.page_indptr, t.page_indices,
                              max_kv_len=400, dev_status=status, layout=layout)
        pd.pd_attn_chunk_quant(q_out, kp, vp, ks, vs, t.kv_len, t.page_indptr, t.page_indices, t.qo_indptr,
                               window_left=window, max_qo_len=most, max_kv_len=400, o=o, lse=lse, workspace=ws,
                               dev_status=status, layout=layout)

    graph, have = None, [0] * B
    for i, ns in enumerate(plan):
        new.copy_(i32(ns))
        qkv.copy_(torch.randn(qkv.shape, device="cuda", generator=g) * torch.exp(0.5 * torch.randn(
            cap, 1, device="cuda", generator=g)))
        before = [x.clone() for x in (kp, ks, vp, vs)]
        o.fill_(7), lse.fill_(7)
        torch.cuda.synchronize()
        if not captured or i == 0:
            step()
        else:
            if graph is None:
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph):
                    step()
            graph.replay()
        torch.cuda.synchronize()
        assert int(status.item()) == 0
        at = sum(ns)
        have = [h + n for h, n in zip(have, ns)]
        qo = [sum(ns[:r]) for r in range(B + 1)]
        for got, x, w in ((q_out, q, qw), (k_out, k, kw)):
            want, size = axes_ref(x[:at], w, inv_freq, axes, pos[:, :at], eps=1e-6, interleaved=False)
            assert bool(((got[:at].double() - want).abs() <= ref.norm_rope_bound(want, size, dt)).all())
        pp, px = out.page_indptr.tolist(), out.page_indices
        assert out.kv_len.tolist() == have
        # the cache: of the rows that the calls before handed on, exactly
        for x, (pool, scale), (was, was_scale) in ((k_out, (kp, ks), before[:2]), (v, (vp, vs), before[2:])):
            want, want_scale = qref.append(x, was, was_scale, qo, have, pp, px.tolist(), page, block, layout)
            assert torch.equal(torch.nan_to_num(pool.double(), nan=1e6), torch.nan_to_num(want, nan=1e6))
            assert torch.equal(torch.nan_to_num(scale.double(), nan=-1), torch.nan_to_num(want_scale, nan=-1))
        ref.check_attention(o[:at], lse[:at], qref.attention(q_out[:at], kp, vp, ks, vs, qo, have, pp, px, window=window,
                                                             layout=layout))
        assert bool((o[at:] == 7).all()) and bool((lse[at:] == 7).all())  # rows behind the last
        cached.copy_(out.kv_len)


@pytest.mark.parametrize("handle", [False, True])
def test_results_of_a_call_on_another_stream_are_its_own(handle):
    """Memory that the current stream has let go of, but will still write, is not taken for them."""
    q, k = (torch.randn(300, 8, 128, device="cuda").bfloat16() for _ in range(2))
    pool = torch.randn(20, 8, 16, 128, device="cuda").to(E4M3)
    scale = torch.ones(20, 8, 1, device="cuda")
    pp, px, qo, kv = i32([0, 19]), torch.arange(20, device="cuda", dtype=torch.int32), i32([0, 300]), i32([300])
    pos, freq = torch.arange(600, device="cuda", dtype=torch.int32).view(2, 300), torch.ones(64, device="cuda")
    stream = torch.cuda.Stream()
    calls = [
        lambda **kw: pd.pd_qk_norm_rope_axes(q, k, None, None, freq, [0, 1] * 32, pos, **kw),
        lambda **kw: pd.pd_attn_chunk_quant(q, pool, pool, scale, scale, kv, pp, px, qo, max_qo_len=300, max_kv_len=300,
                                            **kw),
    ]
    for call in calls:
        want = call()
        torch.cuda.synchronize()
        spent = [torch.empty_like(t) for t in want] + [torch.empty(1 << 20, dtype=torch.uint8, device="cuda")]
        torch.cuda._sleep(20_000_000)
        for t in spent:
            t.fill_(7)
        del t, spent
        got = call(stream=stream.cuda_stream if handle else stream)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("handle", [False, True])
def test_lengths_are_read_on_the_stream_of_the_call(handle):
    """Without bounds a call reads the lengths back, and waits for what writes them on its own stream: here they
    become 60 new tokens of 300 behind a delay, and are one of one before."""
    q, k, v = (torch.randn(60, 8, 128, device="cuda").bfloat16() for _ in range(3))
    pool, scale = torch.randn(20, 8, 16, 128, device="cuda").to(E4M3), torch.ones(20, 8, 1, device="cuda")
    pp, px = i32([0, 19]), torch.arange(20, device="cuda", dtype=torch.int32)
    kv, qo, late_kv, late_qo = i32([1]), i32([0, 1]), i32([300]), i32([0, 60])
    stream = torch.cuda.Stream()

    def append(**kw):
        pools = [pool.clone(), pool.clone(), scale.clone(), scale.clone()]
        pd.pd_kv_append_quant(k, v, *pools, qo, kv, pp, px, **kw)
        return [x.view(torch.uint8) for x in pools]

    calls = [
        (lambda **kw: pd.pd_attn_chunk_quant(q, pool, pool, scale, scale, kv, pp, px, qo, **kw), True),
        (append, False),
    ]
    for call, new in calls:
        status = i32([0])
        kv.copy_(late_kv), qo.copy_(late_qo)
        want = call(max_kv_len=300, **(dict(max_qo_len=60) if new else {}))
        torch.cuda.synchronize()
        want = [t.clone() for t in want]
        kv.fill_(1), qo.copy_(i32([0, 1]))
        torch.cuda.synchronize()
        with torch.cuda.stream(stream):
            torch.cuda._sleep(40_000_000)
            kv.copy_(late_kv), qo.copy_(late_qo)
        got = call(stream=stream.cuda_stream if handle else stream, dev_status=status)
        torch.cuda.synchronize()
        assert int(status.item()) == 0
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_other_threads_run_during_a_call(tmp_path):
    """A call that takes long on the host (here: entry points that sleep, in the library's place) does not keep
    the interpreter's lock."""
    src = tmp_path / "slow.c"
    src.write_text("#include <unistd.h>\nint slow(void) { usleep(300000); return 0; }\n")
    subprocess.run(["gcc", "-shared", "-fPIC", "-o", tmp_path / "slow.so", src], check=True)
    slow = ctypes.cast(ctypes.CDLL(str(tmp_path / "slow.so")).slow, ctypes.c_void_p).value
    x, pool = torch.zeros(4, 8, 64, device="cuda"), torch.zeros(4, 8, 16, 64, device="cuda")
    codes, scale = pool.to(E4M3), torch.ones(4, 8, 1, device="cuda")
    n, ids, px, f = i32([4]), i32([0, 4]), i32([0, 1, 2, 3]), torch.ones(32, device="cuda")
    slot, ws = torch.zeros(4, dtype=torch.int64, device="cuda"), torch.zeros(64, dtype=torch.uint8, device="cuda")
    o, lse = torch.empty_like(x), torch.empty(4, 8, device="cuda")
    calls = [
        lambda: pd.pd_qk_norm_rope_axes(x, x, None, None, f, bytes(32), px.view(1, 4), q_out=x, k_out=x),
        lambda: pd.pd_qk_norm_rope_axes_append(x, x, x, None, None, f, bytes(32), px.view(1, 4), slot, pool, pool,
                                               q_out=x),
        lambda: pd.pd_kv_append_quant(x, x, codes, codes, scale, scale, ids, n, ids, px, max_kv_len=4),
        lambda: pd.pd_attn_chunk_quant(x, codes, codes, scale, scale, n, ids, px, ids, max_qo_len=4, max_kv_len=4, o=o,
                                       lse=lse, workspace=ws),
    ]
    ticks, stop = [0], threading.Event()

    def count():
        while not stop.wait(0.002):
            ticks[0] += 1

    thread = threading.Thread(target=count)
    thread.start()
    bind = pd._load_bind()
    try:
        bind.init_more(*[slow] * 5)
        during = []
        for call in calls:
            before = ticks[0]
            call()
            during.append(ticks[0] - before)
    finally:
        pd._bind = None
        pd._load_bind()  # the library's own again
        stop.set()
        thread.join()
    assert min(during) >= 20, during  # of about 150; two at most with the lock held


@pytest.mark.parametrize("hq,hkv,d,page,block,layout", [(8, 2, 128, 16, 16, "HND"), (16, 2, 64, 32, 8, "NHD"),
                                                        (4, 4, 128, 24, 8, "NHD"), (7, 1, 128, 64, 64, "HND")])
@pytest.mark.parametrize("new,kv", [
    ([1, 2, 1, 2], [900, 37, 2, 4100]),         # 8 query rows a KV head, or fewer
    ([2, 1, 0, 2], [193, 192, 50, 191]),        # ends around a turn of all warps' keys
    ([1] * 5, [15, 16, 17, 1, 5000]),
    ([8], [3000]), ([4, 3], [2000, 1000]),
])
@pytest.mark.parametrize("window", [-1, 100])
def test_few_rows(hq, hkv, d, page, block, layout, new, kv, window):
    from test_gpu_chunk_quant import Batch
    Batch(3, new, kv, hq, hkv, d, page, block, BF16, layout).check(window=window)


@pytest.mark.parametrize("n,hq,hkv,d,most", [(140, 4, 1, 128, 1000), (300, 8, 1, 128, 1024), (304, 2, 1, 128, 200),
                                             (456, 4, 1, 64, 1024), (457, 4, 1, 64, 700), (150, 6, 3, 64, 900)])
def test_few_rows_of_as_many_requests_as_ctas(n, hq, hkv, d, most):
    """An item a CTA, or just more than that; more requests than a CTA makes the line of by itself."""
    from test_gpu_chunk_quant import Batch
    rng = random.Random(n)
    kv = [rng.choice([1, 31, 32, 33, 128, rng.randint(1, most)]) for _ in range(n - 1)] + [most]
    Batch(4, [1] * n, kv, hq, hkv, d, 16, 16, BF16).check()
