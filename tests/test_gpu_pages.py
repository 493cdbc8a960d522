"""copy_pages, free_pages, fork_pages and compact_pages on the GPU against the same steps one at a time."""
import numpy as np
import pytest
import torch

import kv_cache_quantize_b200 as kvq
from _attention import compact_plain, fork_plain, free_plain

pytestmark = pytest.mark.gpu


def caches_of(pages, seed, shapes=(((16, 2, 64), torch.int8), ((16, 2, 64), torch.int8), ((16, 1, 3), torch.float32))):
    """Device caches of several types inside guarded storages, and numpy copies of their bytes."""
    r = np.random.default_rng(seed)
    dev, host = [], []
    for shape, dtype in shapes:
        b = int(np.prod(shape)) * torch.empty(0, dtype=dtype).element_size()
        raw = r.integers(0, 256, (pages, b), dtype=np.uint8)
        host.append(raw.copy())
        t = torch.from_numpy(raw).cuda()
        dev.append(t.view(dtype).view(pages, *shape))
    return dev, host


def same(dev, host):
    for d, h in zip(dev, host):
        got = d.reshape(d.shape[0], -1).contiguous().view(torch.uint8).cpu().numpy()
        assert np.array_equal(got, h)


def i32(x):
    return torch.tensor(np.asarray(x, dtype=np.int32), device="cuda")


@pytest.mark.parametrize("shape,dtype", [((16, 4, 128), torch.int8), ((1,), torch.int8), ((3, 1, 5), torch.uint8),
                                         ((7, 2, 18), torch.bfloat16), ((16, 1, 323), torch.uint8),
                                         ((64, 4, 128), torch.bfloat16), ((5, 1), torch.float32), ((4, 4), torch.int8),
                                         ((8200,), torch.uint8), ((3, 8192), torch.int8)], ids=str)
@pytest.mark.parametrize("n", [1, 37])
@pytest.mark.parametrize("index", [torch.int32, torch.int64])
def test_copy(shape, dtype, n, index):
    dev, host = caches_of(90, 1, ((shape, dtype), (shape, dtype)))
    order = np.random.default_rng(2).permutation(90)
    src, dst = order[:n], order[n:2 * n]
    kvq.get_error()
    kvq.copy_pages(dev, torch.tensor(src, device="cuda", dtype=index), torch.tensor(dst, device="cuda", dtype=index),
                   check=True)
    for h in host:
        h[dst] = h[src]
    same(dev, host)


def test_copy_skips_and_reports():
    dev, host = caches_of(20, 3)
    kvq.get_error()
    kvq.copy_pages(dev, i32([-1, 3, 5, 20, 6, -2]), i32([1, -1, 7, 8, 99, 9]))
    assert kvq.get_error() == kvq.FAULT_SLOT_RANGE
    for h in host:
        h[7] = h[5]
    same(dev, host)
    kvq.copy_pages(dev, i32([-1, 4, 4]), i32([2, -1, 4]), check=True)
    same(dev, host)
    kvq.copy_pages(dev, i32([]), i32([]), check=True)


def test_copy_strided_pages_and_odd_addresses():
    """Padding between pages, a slice of a wider store, and bases that are not 16-byte aligned keep their other bytes."""
    for pad, off in ((16, 0), (16, 16), (5, 1), (4, 4), (8, 2)):
        raw = torch.randint(0, 256, (40 * (96 + pad) + 64,), dtype=torch.uint8, device="cuda")
        view = raw[off:].as_strided((40, 96), (96 + pad, 1))
        want = raw.clone()
        want[off:].as_strided((40, 96), (96 + pad, 1))[i32([1, 2, 39]).long()] = view[i32([30, 0, 17]).long()]
        kvq.copy_pages([view], i32([30, 0, 17]), i32([1, 2, 39]), check=True)
        assert torch.equal(raw, want)


def test_copy_many_caches_and_a_large_cache():
    dev, host = caches_of(12, 4, tuple(((3 + i, 16), torch.int8) for i in range(64)))
    kvq.copy_pages(dev, i32([0, 5]), i32([11, 7]), check=True)
    for h in host:
        h[[11, 7]] = h[[0, 5]]
    same(dev, host)
    big = torch.empty((70000, 65536), dtype=torch.uint8, device="cuda")     # page offsets beyond 32 bits
    big[69999] = 7
    big[1] = 9
    kvq.copy_pages([big], i32([69999, 1]), i32([2, 69998]), check=True)
    assert bool((big[2] == 7).all()) and bool((big[69998] == 9).all())


def state(seed, rows, cols, pages, block, live, share=True):
    """A table whose first `live` rows hold sequences, some of them sharing their first pages."""
    r = np.random.default_rng(seed)
    table = np.full((rows, cols), -1, np.int32)
    lens, ref = np.zeros(rows, np.int32), np.zeros(pages, np.int32)
    free = list(r.permutation(pages))
    for i in range(live):
        n = int(r.integers(0, cols * block + 1))
        held = -(-n // block)
        if held > len(free):
            continue
        lens[i] = n
        for e in range(held):
            if share and i > 0 and e < lens[i - 1] // block and table[i - 1, e] >= 0 and r.integers(0, 2) and \
                    (e == 0 or table[i, e - 1] == table[i - 1, e - 1]):
                table[i, e] = table[i - 1, e]
            else:
                table[i, e] = free.pop()
            ref[table[i, e]] += 1
    return table, lens, ref


@pytest.mark.parametrize("index", [torch.int32, torch.int64])
@pytest.mark.parametrize("rows,cols,pages,block,live", [(1, 1, 1, 1, 1), (9, 5, 60, 16, 7), (200, 33, 9000, 3, 180)])
def test_free(rows, cols, pages, block, live, index):
    table, lens, ref = state(5, rows, cols, pages, block, live)
    dt, dl, dr = i32(table), i32(lens), i32(ref)
    names = np.random.default_rng(6).permutation(rows)[: max(1, rows // 2)]
    kvq.get_error()
    kvq.free_pages(dt, dl, dr, torch.tensor(names, device="cuda", dtype=index), block, check=True)
    assert not free_plain(table, lens, ref, names, block)
    for d, h in ((dt, table), (dl, lens), (dr, ref)):
        assert np.array_equal(d.cpu().numpy(), h)


def test_free_twice_and_bad_rows():
    table, lens, ref = state(7, 6, 4, 30, 8, 5)
    lens[0] = max(int(lens[0]), 1)
    dt, dl, dr = i32(table), i32(lens), i32(ref)
    kvq.get_error()
    kvq.free_pages(dt, dl, dr, i32([2, 2, -1, 2, 5]), 8, check=True)
    free_plain(table, lens, ref, [2, 5], 8)
    assert np.array_equal(dt.cpu().numpy(), table) and np.array_equal(dr.cpu().numpy(), ref)
    kvq.free_pages(dt, dl, dr, i32([6, -2, 3]), 8)
    assert kvq.get_error() == kvq.FAULT_SLOT_RANGE
    free_plain(table, lens, ref, [3], 8)
    assert np.array_equal(dt.cpu().numpy(), table) and np.array_equal(dr.cpu().numpy(), ref)
    # a length that the row cannot hold, a page that is not there, a page that is free already
    bad = np.full((3, 4), -1, np.int32)
    bad[0], bad[1], bad[2, 0] = [0, 1, 2, 3], [4, 99, 5, -1], 6
    ln, rc = np.array([99, 24, 8], np.int32), np.ones(10, np.int32)
    rc[6] = 0
    dt, dl, dr = i32(bad), i32(ln), i32(rc)
    kvq.free_pages(dt, dl, dr, i32([0, 1, 2]), 8)
    assert kvq.get_error() == kvq.FAULT_SLOT_RANGE
    assert free_plain(bad, ln, rc, [0, 1, 2], 8)
    assert np.array_equal(dt.cpu().numpy(), bad) and np.array_equal(dr.cpu().numpy(), rc)
    assert np.array_equal(dl.cpu().numpy(), ln)


def run_fork(table, lens, ref, parents, children, block, seed=8, index=torch.int32, want_bits=0, shapes=None):
    dev, host = caches_of(len(ref), seed, shapes) if shapes else caches_of(len(ref), seed)
    dt, dl, dr = i32(table), i32(lens), i32(ref)
    kvq.get_error()
    fresh = kvq.fork_pages(dev, dt, dl, dr, torch.tensor(parents, device="cuda", dtype=index),
                           torch.tensor(children, device="cuda", dtype=index), block)
    bits = kvq.get_error()
    want, wb = fork_plain(host, table, lens, ref, parents, children, block)
    assert fresh.tolist() == want and bits == wb == want_bits
    for d, h in ((dt, table), (dl, lens), (dr, ref)):
        assert np.array_equal(d.cpu().numpy(), h)
    same(dev, host)


@pytest.mark.parametrize("index", [torch.int32, torch.int64])
@pytest.mark.parametrize("rows,cols,pages,block,live,n", [(3, 1, 5, 1, 1, 2), (40, 6, 150, 16, 10, 30), (40, 6, 150, 7, 10, 30),
                                                          (3000, 4, 20000, 16, 100, 2900)])
def test_fork(rows, cols, pages, block, live, n, index):
    table, lens, ref = state(9, rows, cols, pages, block, live)
    r = np.random.default_rng(10)
    parents = [int(x) for x in r.integers(0, live, n)]
    children = [int(x) for x in live + r.permutation(rows - live)[:n]]
    run_fork(table, lens, ref, parents, children, block, index=index)


def test_fork_without_room_and_without_caches():
    table, lens, ref = state(11, 20, 3, 14, 4, 2, share=False)
    lens[:2] = [9, 10]
    table[:2] = [[0, 3, 5], [13, 1, 2]]
    ref[:] = 0
    ref[[0, 3, 5, 13, 1, 2]] = 1
    run_fork(table, lens, ref, [0, 1] * 5, list(range(2, 12)), 4, want_bits=kvq.FAULT_NO_PAGE)
    # whole pages only: nothing to copy, no page needed
    table[:] = -1
    lens[:], ref[:] = 0, 1
    table[0, :2], lens[0] = [4, 9], 8
    run_fork(table, lens, ref, [0, 0, 1], [5, 6, 7], 4)
    dt, dl, dr = i32(table), i32(lens), i32(ref)
    fresh = kvq.fork_pages([], dt, dl, dr, i32([0]), i32([9]), 4, check=True)
    assert fresh.tolist() == [-1] and dl.tolist()[9] == 8 and dt[9].tolist() == dt[0].tolist()


def test_fork_refusals_leave_rows_empty():
    base = state(12, 12, 4, 60, 8, 4, share=False)
    base[1][:4] = [20, 9, 32, 5]
    base[0][:4], base[2][:] = -1, 0
    at = 0
    for i in range(4):
        for e in range(-(-int(base[1][i]) // 8)):
            base[0][i, e] = at
            base[2][at] = 1
            at += 1
    f = kvq.FAULT_SLOT_RANGE
    for parents, children, bits in (([0, 1], [5, 5], f), ([0, 0], [1, 5], f), ([12, 0], [6, 7], f), ([0, -1], [-2, 8], f),
                                    ([0, -1], [4, -1], 0), ([0, 4], [4, 5], f), ([0, 4, 0], [4, 0, 4], f), ([2, 2], [2, 6], f),
                                    ([7, 8], [8, 9], f), ([7], [8], 0)):
        table, lens, ref = (x.copy() for x in base)
        run_fork(table, lens, ref, parents, children, 8, want_bits=bits)
    table, lens, ref = (x.copy() for x in base)
    lens[3] = 33                                             # longer than its row
    run_fork(table, lens, ref, [3, 0], [5, 6], 8, want_bits=f)


@pytest.mark.parametrize("rows,cols,pages,block,live", [(1, 1, 1, 1, 1), (9, 5, 60, 16, 7), (150, 20, 5000, 3, 140),
                                                        (4, 2, 3000, 16, 4)])
@pytest.mark.parametrize("in_place", [False, True])
def test_compact(rows, cols, pages, block, live, in_place):
    table, lens, ref = state(13, rows, cols, pages, block, live)
    dev, host = caches_of(pages, 14)
    dt, dr = i32(table), i32(ref)
    kvq.get_error()
    if in_place:
        nt, nr, pm = kvq.compact_pages(dev, dt, dr, new_table=dt, new_ref_count=dr, check=True)
        assert nt is dt and nr is dr
    else:
        nt, nr, pm = kvq.compact_pages(dev, dt, dr, check=True)
        assert np.array_equal(dt.cpu().numpy(), table) and np.array_equal(dr.cpu().numpy(), ref)
    wt, wr, wm = compact_plain(host, table, ref)
    assert np.array_equal(nt.cpu().numpy(), wt) and np.array_equal(nr.cpu().numpy(), wr) and pm.tolist() == wm
    same(dev, host)


def test_compact_full_empty_and_bad_entries():
    for fill in (0, 1):
        dev, host = caches_of(50, 15)
        nt, nr, pm = kvq.compact_pages(dev, i32([[-1, -1]]), i32([fill] * 50), check=True)
        assert pm.tolist() == ([-1] * 50 if fill == 0 else list(range(50))) and nr.tolist() == [fill] * 50
        same(dev, host)
    dev, host = caches_of(10, 16)
    ref = np.array([0, 1, 0, 1, 0, 0, 0, 2, 0, 0], np.int32)
    nt, nr, pm = kvq.compact_pages(dev, i32([[1, 7, 10, -5], [3, 7, 2, -1]]), i32(ref))
    assert kvq.get_error() == kvq.FAULT_SLOT_RANGE
    assert nt.tolist() == [[1, 2, -1, -1], [0, 2, -1, -1]] and nr.tolist() == [1, 1, 2] + [0] * 7
    compact_plain(host, np.array([[1]]), ref)
    same(dev, host)


def test_page_operations_captured_and_replayed():
    """free, fork and compact in one graph: a beam step, replayed on states reset to the start."""
    table, lens, ref = state(17, 30, 5, 200, 16, 10)
    dev, host = caches_of(200, 18)
    first = [d.clone() for d in dev]
    dt, dl, dr = i32(table), i32(lens), i32(ref)
    keep = [dt.clone(), dl.clone(), dr.clone()]
    parents, children = i32([0, 3, 3, 9]), i32([12, 5, 20, 29])
    drop = i32([5])

    def step():
        kvq.free_pages(dt, dl, dr, drop, 16)
        fresh = kvq.fork_pages(dev, dt, dl, dr, parents, children, 16)
        return (fresh, *kvq.compact_pages(dev, dt, dr))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        fresh, nt, nr, pm = step()
    for _ in range(2):
        for d, f in zip((*dev, dt, dl, dr), (*first, *keep)):
            d.copy_(f)
        kvq.get_error()
        g.replay()
        torch.cuda.synchronize()
        assert kvq.get_error() == 0
        t, l, r, h = table.copy(), lens.copy(), ref.copy(), [x.copy() for x in host]
        free_plain(t, l, r, [5], 16)
        wf, bits = fork_plain(h, t, l, r, [0, 3, 3, 9], [12, 5, 20, 29], 16)
        assert bits == 0 and fresh.tolist() == wf
        assert np.array_equal(dt.cpu().numpy(), t) and np.array_equal(dr.cpu().numpy(), r)
        wt, wr, wm = compact_plain(h, t, r)
        assert np.array_equal(nt.cpu().numpy(), wt) and np.array_equal(nr.cpu().numpy(), wr) and pm.tolist() == wm
        same(dev, h)
    del g
