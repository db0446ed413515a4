"""pd_batch_tables and pd_slot_map against plain integers: every result equal, entry for entry."""
import ctypes
import random
import threading

import pytest
import torch

import step_ref as ref

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import decode_ragged_paged_gb300 as pd

NAMES = ("qo_indptr", "kv_len", "page_indptr", "page_indices", "positions", "slot_map")


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Case:
    """Lengths, a block table holding the cached pages, and a free list, from a seed."""

    def __init__(self, seed, cached, new, page, *, rows=True, spare_free=9, pops=True):
        rng = random.Random(seed)
        self.cached, self.new, self.page, self.pops = cached, new, page, pops
        B = len(new)
        tot = [ref.ceil_div(max(c, 0) + max(n, 0), page) for c, n in zip(cached, new)]
        old = [ref.ceil_div(max(c, 0), page) if pops else t for c, t in zip(cached, tot)]
        self.cols, self.nrows = max(tot + [1]) + 2, B + 5 if rows else max(B, 1)
        self.num_pages = sum(tot) + spare_free
        ids = list(range(self.num_pages))
        rng.shuffle(ids)
        self.rows = rng.sample(range(self.nrows), B) if rows else None
        self.table = [[-7] * self.cols for _ in range(self.nrows)]
        for r in range(B):
            for j in range(old[r]):
                self.table[self.rows[r] if rows else r][j] = ids.pop()
        self.free = ids
        self.count = len(ids)
        self.total_qo, self.nnz = sum(max(n, 0) for n in new), sum(tot)

    def run(self, *, in_place=False, total_qo=None, nnz=None, out=None, stream=None):
        total_qo = self.total_qo if total_qo is None else total_qo
        nnz = self.nnz if nnz is None else nnz
        table = i32(self.table)
        free = i32(self.free) if self.pops else None
        count = i32([self.count]) if self.pops else None
        left = (count if in_place else i32([-1])) if self.pops else None
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        t = pd.pd_batch_tables(i32(self.new), i32(self.cached), table, page_size=self.page, num_pages=self.num_pages,
                               total_qo=total_qo, max_page_indices=nnz,
                               rows=i32(self.rows) if self.rows is not None else None, free_pages=free,
                               free_count=count, free_count_out=left, out=out, dev_status=status, stream=stream)
        torch.cuda.synchronize()
        want_table = [list(r) for r in self.table]
        want = ref.tables(self.rows, self.cached, self.new, want_table, self.free, self.count, page=self.page,
                          num_pages=self.num_pages, total_qo=total_qo, max_page_indices=nnz, pops=self.pops)
        for name in NAMES:
            got = getattr(t, name).tolist()
            assert got[:len(want[name])] == want[name], name
        assert table.tolist() == want_table
        if self.pops:
            assert left.item() == want["left"]
        return int(status.item()), t


@pytest.mark.parametrize("page", [1, 8, 16, 24, 128])
@pytest.mark.parametrize("in_place", [False, True])
def test_lengths_at_page_edges(page, in_place):
    edge = sorted({0, 1, page - 1, page, page + 1, 3 * page, 3 * page + 1})
    cached = [c for c in edge for _ in range(4)]
    new = [n for _ in edge for n in (0, 1, page, 2 * page + 1)]
    status, _ = Case(1, cached, new, page).run(in_place=in_place)
    assert status == 0


@pytest.mark.parametrize("batch", [1, 2, 31, 1000, 1025, 5000, 8192])
def test_batch_sizes(batch):
    rng = random.Random(batch)
    cached = [rng.randint(0, 300) for _ in range(batch)]
    new = [rng.choice([0, 1, 1, 1, 2, 40]) for _ in range(batch)]
    assert Case(2, cached, new, 16).run(in_place=batch % 2 == 0)[0] == 0
    assert Case(3, cached, new, 16, rows=False).run()[0] == 0


def test_long_requests_and_many_entries():
    assert Case(4, [100000, 0, 7], [1, 70000, 30000], 16).run()[0] == 0


@pytest.mark.parametrize("shape", ["even", "ragged", "one"])
def test_page_lists_of_many_entries_a_thread(shape):
    # long enough that requests are looked up ahead, with empty ones between them
    rng = random.Random(6)
    if shape == "one":
        cached, new = [0, 660000, 0, 3, 0], [0, 5, 2, 0, 0]
    else:
        cached = [2300 if shape == "even" else rng.choice([0, 0, 1, 500, 9000]) for _ in range(400)]
        new = [rng.choice([0, 1, 3]) for _ in cached]
    c = Case(7, cached, new, 1, rows=shape != "one")
    assert c.nnz > 4 * 1024 * torch.cuda.get_device_properties(0).multi_processor_count
    assert c.run()[0] == 0


def test_without_a_free_list():
    assert Case(5, [0, 15, 16, 100], [1, 1, 1, 33], 16, pops=False).run()[0] == 0
    assert Case(5, [0, 15, 16, 100], [1, 1, 1, 33], 16, pops=False, rows=False).run()[0] == 0


def test_padded_rows_and_untouched_tails():
    c = Case(6, [3, 40, 0], [1, 1, 5], 16)
    out = tuple(torch.full((n,), -99, dtype=t, device="cuda") for n, t in
                ((4, torch.int32), (3, torch.int32), (4, torch.int32), (c.nnz + 6, torch.int32), (20, torch.int32),
                 (23, torch.int64)))
    status, t = c.run(total_qo=20, nnz=c.nnz + 6, out=out)
    assert status == 0
    assert t.slot_map[7:20].tolist() == [-1] * 13 and t.positions[7:].tolist() == [0] * 13
    assert t.page_indices[c.nnz:].tolist() == [-99] * 6 and t.slot_map[20:].tolist() == [-99] * 3


def test_empty_batch():
    c = Case(7, [], [], 16, rows=False)
    status, t = c.run(total_qo=5)
    assert status == 0 and t.qo_indptr.tolist() == [0] and t.slot_map.tolist() == [-1] * 5


@pytest.mark.parametrize("in_place", [False, True])
def test_free_list_runs_out(in_place):
    c = Case(8, [0, 31, 32, 5, 16], [33, 1, 1, 1, 16], 16)
    for count in (0, 2, 3, 4, 5, 10 ** 6, -3):
        c.count = count
        status, t = c.run(in_place=in_place)
        kv = t.kv_len.tolist()
        assert kv[1] == 32 and kv[3] == 6  # no new page needed: served
        assert (status == 7) == (count < 5)


def test_bad_requests_are_refused_and_the_rest_served():
    c = Case(9, [0, 20, 5, 7, 3, 1], [4, 1, 2, 3, 1, 1], 16)
    c.cached[1] = -1
    c.new[2] = -3
    c.rows[4] = c.rows[0]       # listed by an earlier request
    c.rows[3] = c.nrows         # past the table
    status, t = c.run()
    assert status in (2, 8)
    assert t.kv_len.tolist() == [4, -1, -1, -1, -1, 2]
    c = Case(9, [0, 2, 40], [4, 100, 1], 16)
    c.cached[1] = 2 ** 31 - 5   # past 32 bits, and more pages than columns
    status, t = c.run()
    assert status == 2 and t.kv_len.tolist() == [4, -1, 41]


def test_a_row_listed_many_times_goes_to_the_first():
    c = Case(10, [5] * 300, [20] * 300, 16)
    c.rows = [c.rows[i % 7] for i in range(300)]
    status, t = c.run()
    assert status == 8 and (t.kv_len[:7] == 25).all() and (t.kv_len[7:] == -1).all()


def test_capacities():
    c = Case(11, [0, 17, 33], [10, 5, 7], 16)
    for total, nnz in ((22, c.nnz), (21, c.nnz), (14, c.nnz), (9, c.nnz), (0, c.nnz), (22, c.nnz - 1), (22, 1), (22, 0)):
        status, _ = c.run(total_qo=total, nnz=nnz)
        assert (status == 1) == (total < 22 or nnz < c.nnz)


def test_bad_page_ids_are_entered_and_reported():
    c = Case(12, [20, 3], [14, 1], 16)
    c.table[c.rows[0]][0] = c.num_pages       # under cached tokens only
    status, t = c.run()
    assert status == 3
    c = Case(12, [20, 3], [14, 1], 16)
    c.free[-1] = -5
    status, t = c.run()
    assert status == 3 and t.slot_map.tolist()[12:14] == [-1, -1]


def test_repeated_and_captured_with_other_lengths():
    B, page = 40, 16
    rng = random.Random(13)
    cached0 = [rng.randint(0, 100) for _ in range(B)]
    c = Case(13, cached0, [3] * B, page, spare_free=400)
    table, free = i32(c.table), i32(c.free)
    new, cached, count = i32(c.new), i32(c.cached), i32([c.count])
    want_table = [list(r) for r in c.table]
    kw = dict(page_size=page, num_pages=c.num_pages, total_qo=200, max_page_indices=600, rows=i32(c.rows),
              free_pages=free, free_count=count, free_count_out=count)
    host_count, host_cached = c.count, list(cached0)
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        t = pd.pd_batch_tables(new, cached, table, **kw)   # a first step, then captured ones
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            pd.pd_batch_tables(new, cached, table, out=t, **kw)
    stream.synchronize()
    for step in range(6):
        want = ref.tables(c.rows, host_cached, c.new, want_table, c.free, host_count, page=page,
                          num_pages=c.num_pages, total_qo=200, max_page_indices=600)
        for name in NAMES:
            got = getattr(t, name).tolist()
            assert got[:len(want[name])] == want[name], (step, name)
        assert table.tolist() == want_table and count.item() == want["left"]
        host_count, host_cached = want["left"], want["kv_len"]
        c.new = [rng.randint(0, 5) for _ in range(B)]
        cached.copy_(t.kv_len)
        new.copy_(i32(c.new))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()


@pytest.mark.parametrize("page", [1, 16, 24])
def test_slot_map(page):
    c = Case(14, [0, 15, 100, 7, 0], [1, 40, 0, 3, 20], page)
    _, t = c.run(total_qo=c.total_qo + 9)
    pos, slot = pd.pd_slot_map(t.qo_indptr, t.kv_len, t.page_indptr, t.page_indices, page_size=page,
                               num_pages=c.num_pages, total_qo=c.total_qo + 9)
    assert torch.equal(pos, t.positions) and torch.equal(slot, t.slot_map)


def test_slot_map_reports_bad_batches():
    def call(qo, kv, pp, px, total=4):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        _, slot = pd.pd_slot_map(i32(qo), i32(kv), i32(pp), i32(px), page_size=16, num_pages=4, total_qo=total,
                                 max_kv_len=64, dev_status=status)
        return int(status.item()), slot.tolist()
    assert call([0, 2, 4], [20, 3], [0, 2, 3], [1, 2, 0]) == (0, [34, 35, 1, 2])
    assert call([0, 2, 4], [20, 1], [0, 2, 3], [1, 2, 0]) == (2, [34, 35, -1, -1])     # fewer keys than rows
    assert call([0, 2, 4], [-1, 3], [0, 2, 3], [1, 2, 0]) == (2, [-1, -1, 1, 2])
    assert call([0, 2, 4], [65, 3], [0, 5, 6], [1] * 6)[0] == 2                        # past max_kv_len
    assert call([0, 2, 4], [20, 3], [0, 1, 2], [1, 0]) == (3, [-1, -1, 1, 2])          # a page short
    assert call([0, 2, 4], [20, 3], [0, 2, 3], [1, 4, 0]) == (3, [-1, -1, 1, 2])       # id out of range
    assert call([0, 2, 4], [20, 3], [3, 2, 3], [1, 2, 0])[0] == 1


def test_threads_with_large_batches_of_different_sizes():
    """Calls of 8192 and of 2500 requests with a row list from two threads, on a stream each: neither
    call's shared memory is taken from the other's."""
    lib = pd.load_library()
    failed, ran, start = [], [0, 0], threading.Barrier(2)

    def worker(which, B):
        g = torch.Generator().manual_seed(which)
        rows = torch.randperm(B, generator=g).int()
        cached, new = (torch.randint(0, 40, (B,), generator=g, dtype=torch.int32) for _ in range(2))
        page, cols = 16, 8
        total, nnz = int(new.sum()), int(((cached + new + page - 1) // page).sum())
        table = torch.randint(0, 100, (B, cols), generator=g, dtype=torch.int32)
        dev = [t.cuda() for t in (rows, cached, new, table)]
        out = [torch.zeros(n, dtype=t, device="cuda") for n, t in ((B + 1, torch.int32), (B, torch.int32),
               (B + 1, torch.int32), (nnz, torch.int32), (total, torch.int32), (total, torch.int64))]
        stream = torch.cuda.Stream()
        desc = pd.TablesDesc(B, page, 100, B, cols, total, nnz, 0)
        ptrs = [t.data_ptr() for t in dev] + [None] * 3 + [t.data_ptr() for t in out]
        torch.cuda.synchronize()
        start.wait()
        for i in range(3000):
            rc = lib.pd_batch_tables(ctypes.byref(desc), *ptrs, None, stream.cuda_stream)
            if rc != 0:
                failed.append((B, i, rc))
                break
            ran[which] += 1
        stream.synchronize()
        want = ref.tables(rows.tolist(), cached.tolist(), new.tolist(), table.tolist(), [], 0, page=page, num_pages=100,
                          total_qo=total, max_page_indices=nnz, pops=False)
        for name, t in zip(NAMES, out):
            if t.tolist() != want[name]:
                failed.append((B, name))

    threads = [threading.Thread(target=worker, args=x) for x in ((0, 8192), (1, 2500))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed and ran == [3000, 3000]
