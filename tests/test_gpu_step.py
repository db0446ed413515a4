"""A serving step as it is used: tables from lengths, norm + rotation + append into the pages, attention
of the new tokens, over several steps of a ragged batch; against fp64 attention over a dense cache."""
import ctypes
import random
import subprocess
import threading

import pytest
import torch

import step_ref as ref

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import decode_ragged_paged_gb300 as pd


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("dt,hq,hkv,d,page,layout,window,captured", [
    (torch.float32, 8, 2, 64, 16, "HND", -1, False),
    (torch.bfloat16, 32, 8, 128, 16, "HND", -1, False),
    (torch.bfloat16, 4, 4, 128, 64, "NHD", 50, False),
    (torch.bfloat16, 28, 4, 128, 16, "HND", -1, True),
    (torch.bfloat16, 8, 2, 64, 24, "NHD", -1, True),
])
def test_steps(dt, hq, hkv, d, page, layout, window, captured):
    g = torch.Generator(device="cuda").manual_seed(1)
    rng = random.Random(2)
    B, steps, cap = 9, 5, 260
    plan = [[rng.choice([0, 1, 1, 3, 40]) for _ in range(B)] for _ in range(steps)]
    plan[0] = [1, 100, 17, 16, 0, 33, 2, 5, 64]
    num_pages = sum(ref.ceil_div(sum(p[r] for p in plan), page) for r in range(B)) + 5
    shape = (num_pages, hkv, page, d) if layout == "HND" else (num_pages, page, hkv, d)
    kp, vp = (torch.full(shape, float("nan"), device="cuda").to(dt) for _ in range(2))
    free = torch.randperm(num_pages, device="cuda", generator=g).to(torch.int32)
    count, table = i32([num_pages]), torch.full((B + 3, 40), -1, dtype=torch.int32, device="cuda")
    rows = torch.randperm(B + 3, device="cuda", generator=g)[:B].to(torch.int32)
    cached, new = torch.zeros(B, dtype=torch.int32, device="cuda"), i32(plan[0])
    inv_freq = (10000.0 ** (-torch.arange(d // 2, device="cuda", dtype=torch.float64) / (d // 2))).float()
    qw, kw = ((1 + 0.2 * torch.randn(d, device="cuda", generator=g)).to(dt) for _ in range(2))
    qkv = torch.zeros(cap, (hq + 2 * hkv) * d, device="cuda").to(dt)
    q, k, v = (x.view(cap, -1, d) for x in qkv.split([hq * d, hkv * d, hkv * d], 1))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    q_out, o = (torch.zeros(cap, hq, d, device="cuda").to(dt) for _ in range(2))
    lse = torch.zeros(cap, hq, device="cuda")
    ws = torch.empty(96 << 20, dtype=torch.uint8, device="cuda")
    out = pd.BatchTables(*(torch.zeros(n, dtype=t, device="cuda") for n, t in (
        (B + 1, torch.int32), (B, torch.int32), (B + 1, torch.int32), (num_pages, torch.int32), (cap, torch.int32),
        (cap, torch.int64))))

    def step():
        t = pd.pd_batch_tables(new, cached, table, page_size=page, num_pages=num_pages, total_qo=cap,
                               max_page_indices=num_pages, rows=rows, free_pages=free, free_count=count,
                               free_count_out=count, out=out, dev_status=status)
        pd.pd_qk_norm_rope_append(q, k, v, qw, kw, inv_freq, t.positions, t.slot_map, kp, vp, q_out=q_out,
                                  dev_status=status, layout=layout)
        pd.pd_attn_chunk(q_out, kp, vp, t.kv_len, t.page_indptr, t.page_indices, t.qo_indptr, window_left=window,
                         max_qo_len=100, max_kv_len=400, o=o, lse=lse, workspace=ws, dev_status=status, layout=layout)

    graph = None
    past_k, past_v = [[] for _ in range(B)], [[] for _ in range(B)]
    have = [0] * B
    for i, ns in enumerate(plan):
        new.copy_(i32(ns))
        qkv.copy_(torch.randn(qkv.shape, device="cuda", generator=g))
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
        at = 0
        for r, n in enumerate(ns):
            pos = torch.arange(have[r], have[r] + n, device="cuda")
            kn, size = ref.norm_rope(k[at:at + n], kw, inv_freq, pos, eps=1e-6, interleaved=False)
            qn, qsize = ref.norm_rope(q[at:at + n], qw, inv_freq, pos, eps=1e-6, interleaved=False)
            assert bool(((q_out[at:at + n].double() - qn).abs() <= ref.norm_rope_bound(qn, qsize, dt)).all())
            past_k[r].append((kn, size))
            past_v[r].append(v[at:at + n].clone())
            have[r] += n
            ids = out.page_indices[int(out.page_indptr[r]):int(out.page_indptr[r + 1])]
            got_k, got_v = (ref.gather(x, ids, have[r], layout) for x in (kp, vp))
            if have[r]:
                want, size = (torch.cat([p[e] for p in past_k[r]]) for e in (0, 1))
                assert bool(((got_k - want).abs() <= ref.norm_rope_bound(want, size, dt)).all())
                assert torch.equal(got_v, torch.cat(past_v[r]).double())
            at += n
        assert out.kv_len.tolist() == have and int(count.item()) == num_pages - sum(
            ref.ceil_div(h, page) for h in have)
        # attention over what the cache holds, through the plain form's own dense gather
        qo = [sum(ns[:r]) for r in range(B + 1)]
        want = ref.attention(q_out[:at], kp, vp, qo, have, out.page_indptr.tolist(), out.page_indices, window=window,
                             layout=layout)
        ref.check_attention(o[:at], lse[:at], want)
        cached.copy_(out.kv_len)


@pytest.mark.parametrize("handle", [False, True])
def test_results_of_a_call_on_another_stream_are_its_own(handle):
    """Memory that the current stream has let go of, but will still write, is not taken for them."""
    q, k = (torch.randn(300, 8, 128, device="cuda").bfloat16() for _ in range(2))
    pool = torch.randn(20, 8, 16, 128, device="cuda").bfloat16()
    pp, px, qo, kv = i32([0, 19]), torch.arange(20, device="cuda", dtype=torch.int32), i32([0, 300]), i32([300])
    new, have, table = i32([300]), i32([0]), px.view(1, 20).clone()
    stream = torch.cuda.Stream()
    calls = [
        lambda **kw: pd.pd_qk_norm_rope(q, k, None, None, None, None, **kw),
        lambda **kw: pd.pd_attn_chunk(q, pool, pool, kv, pp, px, qo, max_qo_len=300, max_kv_len=300, **kw),
        lambda **kw: pd.pd_slot_map(qo, kv, pp, px, page_size=16, num_pages=20, total_qo=300, max_kv_len=300, **kw),
        lambda **kw: pd.pd_batch_tables(new, have, table, page_size=16, num_pages=20, total_qo=300,
                                        max_page_indices=19, **kw),
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
    """Without bounds a call reads the lengths back, and waits for what writes them on its own stream:
    here they become 60 new tokens of 300 behind a delay, and are one of one before."""
    q, k, v = (torch.randn(60, 8, 128, device="cuda").bfloat16() for _ in range(3))
    pool = torch.randn(20, 8, 16, 128, device="cuda").bfloat16()
    pp, px = i32([0, 19]), torch.arange(20, device="cuda", dtype=torch.int32)
    kv, qo, late_kv, late_qo = i32([1]), i32([0, 1]), i32([300]), i32([0, 60])
    mla_q, mla_pool = torch.randn(1, 4, 576, device="cuda").bfloat16(), torch.randn(20, 16, 576, device="cuda").bfloat16()
    stream = torch.cuda.Stream()

    def append(**kw):
        pools = [pool.clone(), pool.clone()]
        pd.pd_kv_append(k, v, *pools, qo, kv, pp, px, **kw)
        return pools

    calls = [
        (lambda **kw: pd.pd_attn_chunk(q, pool, pool, kv, pp, px, qo, **kw), True),
        (lambda **kw: pd.pd_slot_map(qo, kv, pp, px, page_size=16, num_pages=20, total_qo=60, **kw), False),
        (lambda **kw: pd.pd_attn_prefill(q, pool, pool, kv, pp, px, qo, **kw), True),
        (lambda **kw: pd.pd_attn_mixed(q, pool, pool, kv, pp, px, qo, **kw), True),
        (lambda **kw: pd.pd_attn_decode(q[:1], pool, pool, kv, pp, px, **kw), False),
        (lambda **kw: pd.pd_mla_decode(mla_q, mla_pool, kv, pp, px, **kw), False),
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


def test_a_batch_of_refused_requests_is_skipped_without_bounds():
    """Lengths of -1 (pd_batch_tables: no request could be served) are no bound of -1: the calls skip
    and report them as they do beside others."""
    status = i32([0])
    table = torch.zeros(2, 4, dtype=torch.int32, device="cuda")
    t = pd.pd_batch_tables(i32([3, 2]), i32([0, 0]), table, page_size=16, num_pages=8, total_qo=5, max_page_indices=8,
                           free_pages=i32([5, 6]), free_count=i32([0]), free_count_out=i32([0]), dev_status=status)
    torch.cuda.synchronize()
    assert t.kv_len.tolist() == [-1, -1] and int(status.item()) == 7
    q, pool = torch.randn(5, 4, 64, device="cuda"), torch.randn(8, 2, 16, 64, device="cuda")
    o, lse = torch.full_like(q, 3.0), torch.full((5, 4), 3.0, device="cuda")
    status.zero_()
    pd.pd_attn_chunk(q, pool, pool, t.kv_len, t.page_indptr, t.page_indices, t.qo_indptr, o=o, lse=lse,
                     dev_status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 2 and bool((o == 3).all()) and bool((lse == 3).all())
    status.zero_()
    pos, slot = pd.pd_slot_map(t.qo_indptr, t.kv_len, t.page_indptr, t.page_indices, page_size=16, num_pages=8,
                               total_qo=5, dev_status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 2 and pos.tolist() == [0] * 5 and slot.tolist() == [-1] * 5
    dec = torch.full((2, 4, 64), 3.0, device="cuda")
    status.zero_()
    pd.pd_attn_decode(q[:2], pool, pool, t.kv_len, t.page_indptr, t.page_indices, o=dec, dev_status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 2 and bool((dec == 3).all())


def _runtime():
    lib = ctypes.CDLL("libcudart.so.13")  # the one that is loaded
    lib.cudaStreamCreate.argtypes = [ctypes.POINTER(ctypes.c_void_p)]
    lib.cudaStreamBeginCapture.argtypes = [ctypes.c_void_p, ctypes.c_int]
    lib.cudaStreamEndCapture.argtypes = [ctypes.c_void_p, ctypes.POINTER(ctypes.c_void_p)]
    lib.cudaStreamDestroy.argtypes = [ctypes.c_void_p]
    return lib


def test_an_error_of_another_call_is_not_the_step_calls():
    """The thread's last error of something else (here: a device that is not there) is not returned by
    calls that were launched."""
    q, pool = torch.randn(5, 4, 64, device="cuda"), torch.randn(8, 2, 16, 64, device="cuda")
    o, lse = torch.empty_like(q), torch.empty(5, 4, device="cuda")
    ws = torch.empty(32 << 20, dtype=torch.uint8, device="cuda")
    kv, pp, px, qo = i32([60]), i32([0, 4]), i32([0, 1, 2, 3]), i32([0, 5])
    pos, slot = torch.empty(5, dtype=torch.int32, device="cuda"), torch.empty(5, dtype=torch.int64, device="cuda")
    want = pd.pd_attn_chunk(q, pool, pool, kv, pp, px, qo, max_qo_len=5, max_kv_len=60)[0].clone()
    torch.cuda.synchronize()
    rt = _runtime()
    try:
        assert rt.cudaSetDevice(99) != 0 and rt.cudaPeekAtLastError() != 0
        pd.pd_attn_chunk(q, pool, pool, kv, pp, px, qo, max_qo_len=5, max_kv_len=60, o=o, lse=lse, workspace=ws)
        pd.pd_slot_map(qo, kv, pp, px, page_size=16, num_pages=8, total_qo=5, max_kv_len=60, positions=pos,
                       slot_map=slot)
    finally:
        rt.cudaGetLastError()
    torch.cuda.synchronize()
    assert torch.equal(o, want)


def test_a_refused_launch_leaves_no_error_behind():
    """A launch on the default stream while another stream is captured is refused by the runtime: the
    call says so, and the thread's next call starts clean."""
    lib, rt = pd.load_library(), _runtime()
    kv, pp, px, qo = i32([60]), i32([0, 4]), i32([0, 1, 2, 3]), i32([0, 5])
    pos, slot = torch.empty(5, dtype=torch.int32, device="cuda"), torch.empty(5, dtype=torch.int64, device="cuda")
    batch = pd.make_batch(kv, pp, px, 8, qo_indptr=qo, total_qo=5, max_kv_len=60)
    call = lambda: lib.pd_slot_map(ctypes.byref(batch), 16, pos.data_ptr(), slot.data_ptr(), None, None)  # noqa: E731
    assert call() == pd.PD_OK
    torch.cuda.synchronize()
    stream, graph = ctypes.c_void_p(), ctypes.c_void_p()
    assert rt.cudaStreamCreate(ctypes.byref(stream)) == 0
    try:
        assert rt.cudaStreamBeginCapture(stream, 0) == 0
        rc, left = call(), rt.cudaPeekAtLastError()
        rt.cudaStreamEndCapture(stream, ctypes.byref(graph))
    finally:
        rt.cudaGetLastError()
        rt.cudaStreamDestroy(stream)
    assert rc == pd.PD_ERR_CUDA and left == 0
    assert call() == pd.PD_OK
    torch.cuda.synchronize()


def test_other_threads_run_during_a_call(tmp_path):
    """A call that takes long on the host (here: entry points that sleep, in the library's place) does
    not keep the interpreter's lock."""
    src = tmp_path / "slow.c"
    src.write_text("#include <unistd.h>\nint slow(void) { usleep(300000); return 0; }\n")
    subprocess.run(["gcc", "-shared", "-fPIC", "-o", tmp_path / "slow.so", src], check=True)
    slow = ctypes.cast(ctypes.CDLL(str(tmp_path / "slow.so")).slow, ctypes.c_void_p).value
    x, pool = torch.zeros(4, 8, 64, device="cuda"), torch.zeros(4, 8, 16, 64, device="cuda")
    n, ids, pos = i32([4]), i32([0, 4]), i32([0, 1, 2, 3])
    slot, ws = torch.zeros(4, dtype=torch.int64, device="cuda"), torch.zeros(64, dtype=torch.uint8, device="cuda")
    o, lse = torch.empty_like(x), torch.empty(4, 8, device="cuda")
    out = pd.BatchTables(ids.clone(), n.clone(), ids.clone(), pos.clone(), pos.clone(), slot)
    calls = [
        lambda: pd.pd_batch_tables(n, n, pos.view(1, 4), page_size=16, num_pages=4, total_qo=4, max_page_indices=4, out=out),
        lambda: pd.pd_qk_norm_rope(x, x, None, None, None, None, q_out=x, k_out=x),
        lambda: pd.pd_qk_norm_rope_append(x, x, x, None, None, None, None, slot, pool, pool, q_out=x),
        lambda: pd.pd_attn_chunk(x, pool, pool, n, ids, pos, ids, max_qo_len=4, max_kv_len=4, o=o, lse=lse, workspace=ws),
    ]
    ticks, stop = [0], threading.Event()

    def count():
        while not stop.wait(0.002):
            ticks[0] += 1

    thread = threading.Thread(target=count)
    thread.start()
    bind = pd._load_bind()
    try:
        bind.init(pd.PdError, *[slow] * 5)
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


def test_flags_without_a_truth_value_are_refused():
    x, pool = torch.zeros(4, 8, 64, device="cuda"), torch.zeros(4, 8, 16, 64, device="cuda")
    flag = torch.tensor([True, False])
    with pytest.raises(RuntimeError, match="ambiguous"):
        pd.pd_attn_chunk(x, pool, pool, i32([4]), i32([0, 1]), i32([0]), i32([0, 4]), causal=flag)
    with pytest.raises(RuntimeError, match="ambiguous"):
        pd.pd_qk_norm_rope(x, x, None, None, None, None, interleaved=flag)


@pytest.mark.parametrize("handle", [False, True])
def test_results_of_an_attention_call_on_another_stream_are_its_own(handle):
    """As above, for the calls beside the step's: results and workspace are allocated on the call's stream."""
    q, pool = torch.randn(300, 8, 128, device="cuda").bfloat16(), torch.randn(20, 8, 16, 128, device="cuda").bfloat16()
    pp, px, qo, kv = i32([0, 19]), torch.arange(20, device="cuda", dtype=torch.int32), i32([0, 300]), i32([300])
    B = 40
    many = dict(kv_len=i32([300] * B), page_indptr=torch.arange(B + 1, device="cuda", dtype=torch.int32) * 19,
                page_indices=px[:19].repeat(B))
    mla_q, mla_pool = torch.randn(B, 4, 576, device="cuda").bfloat16(), torch.randn(20, 16, 576, device="cuda").bfloat16()
    two = dict(kv_len=i32([299, 300]), page_indptr=i32([0, 19, 38]), page_indices=px[:19].repeat(2), max_kv_len=300,
               qo_indptr=i32([0, 299, 300]))
    stream = torch.cuda.Stream()
    calls = [
        lambda **kw: pd.pd_attn_prefill(q, pool, pool, kv, pp, px, qo, max_qo_len=300, max_kv_len=300, **kw),
        lambda **kw: pd.pd_attn_mixed(q, pool, pool, kv, pp, px, qo, max_qo_len=300, max_kv_len=300, **kw),
        lambda **kw: pd.pd_attn_mixed_split(q, pool, pool, num_prefill=1, max_qo_len=299, **two, **kw),
        lambda **kw: pd.pd_attn_decode(q[:B], pool, pool, max_kv_len=300, **many, **kw),
        lambda **kw: pd.pd_mla_decode(mla_q, mla_pool, max_kv_len=300, **many, **kw),
    ]
    for call in calls:
        want = call()
        torch.cuda.synchronize()
        # what the call takes from a pool of memory is in use there until the delay is over
        spent = [torch.empty_like(t) for t in want] + [torch.empty(1 << 20, dtype=torch.uint8, device="cuda")]
        torch.cuda.synchronize()
        torch.cuda._sleep(20_000_000)
        for t in spent:
            t.fill_(7)
        del t, spent
        got = call(stream=stream.cuda_stream if handle else stream)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
