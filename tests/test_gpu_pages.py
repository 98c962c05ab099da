"""spec_cache_compact and spec_page_fork against plain loops, bit for bit."""
import numpy as np
import pytest
import torch

from tree_util import compact_ref, fork_ref, random_tables

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module")
def sv():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import rejection_sampling_verify_07_amd as sv

    sv.load_library()
    return sv


def ints(a):
    return torch.from_numpy(np.ascontiguousarray(a, np.int32)).to(DEV)


def make_pool(rng, slabs, pages, heads, size, row, dtype):
    """The same random values as a numpy array [slabs, pages, heads, size, row] and a GPU tensor of it."""
    a = rng.integers(-100, 100, (slabs, pages, heads, size, row)).astype(dtype)
    return a, torch.from_numpy(a.copy()).to(DEV)


def form(t, heads):
    """The call's form of a [slabs, pages, heads, size, row] tensor."""
    return t if heads != 1 else t[:, :, 0]


def random_paths(rng, drafts, accepted):
    path = np.full(int(sum(drafts)) + len(drafts), -1, np.int64)
    at = 0
    for k, n in zip(drafts, accepted):
        path[at] = 0
        path[at + 1:at + 1 + n] = 1 + np.sort(rng.permutation(k)[:n])
        at += k + 1
    return path


COMPACT = [
    # slabs, heads, row, dtype, page, drafts, lengths over the newest rows
    (1, 1, 8, np.int16, 16, [5], [40]),
    (2, 1, 8, np.int16, 16, [5, 0, 9], [0, 3, 30]),
    (3, 2, 5, np.int8, 5, [1, 12, 7, 30], [3, 100, 0, 51]),
    (12, 8, 64, np.int16, 16, [12] * 3, [200, 17, 1]),
    (2, 1, 512, np.int32, 1, [20, 4], [9, 2]),
    (5, 3, 9, np.int16, 7, [3, 0, 128, 64], [5, 0, 77, 1]),
    (64, 1, 1024, np.int16, 32, [24, 8], [100, 31]),
]


@pytest.mark.parametrize("slabs,heads,row,dtype,size,drafts,context", COMPACT)
@pytest.mark.parametrize("paged", [True, False])
def test_compact(sv, slabs, heads, row, dtype, size, drafts, context, paged):
    rng = np.random.default_rng(slabs * 100 + row)
    b = len(drafts)
    lengths = np.array(context) + np.array(drafts) + 1
    if not paged:
        size = int(lengths.max()) + 2
    most = -(-int(lengths.max()) // size)
    pages = b * most + 3 if paged else b + 1
    table = rng.permutation(pages)[:b * most].reshape(b, most) if paged else None
    for accepted in ([k for k in drafts], [0] * b, [int(rng.integers(0, k + 1)) for k in drafts],
                     [min(k, 3) for k in drafts]):
        pool, gpu = make_pool(rng, slabs, pages, heads, size, row, dtype)
        path = random_paths(rng, drafts, accepted)
        cu = np.concatenate([[0], np.cumsum(drafts)])
        ragged = len(set(drafts)) > 1
        want, new = compact_ref(pool, table, lengths, path, np.array(accepted), cu, max(drafts))
        got = sv.compact_cache(form(gpu, heads), ints(path), ints(accepted), ints(lengths),
                               None if table is None else ints(table), ints(cu) if ragged else None)
        assert np.array_equal(got.cpu().numpy(), new)
        assert np.array_equal(gpu.cpu().numpy(), want)


def test_compact_unusual_inputs(sv):
    """Bad paths, counts, pages and lengths: what the call leaves out, and nothing else moves."""
    rng = np.random.default_rng(5)
    size, most, pages = 4, 6, 40
    drafts = [6] * 9
    table = rng.permutation(pages)[:9 * 4].reshape(9, 4)
    table = np.concatenate([table, np.full((9, 2), -1)], axis=1)
    lengths = np.array([14, 14, 14, 14, 14, 14, 3, 99, -5])
    path = np.array([[0, 2, 4, 6, -1, -1, -1],   # sound
                     [0, 2, 2, 5, -1, -1, -1],   # does not rise
                     [0, 3, 9, 4, -1, -1, -1],   # past K
                     [0, -1, 2, 3, -1, -1, -1],  # not there
                     [0, 2, 4, 6, -1, -1, -1],   # count -1
                     [0, 2, 4, 6, -1, -1, -1],   # count past K
                     [0, 2, 4, 6, -1, -1, -1],   # positions below 0
                     [0, 2, 4, 6, -1, -1, -1],   # length past the table, in pages that are none
                     [0, 2, 4, 6, -1, -1, -1]])
    nacc = np.array([3, 3, 3, 3, -1, 7, 3, 3, 3])
    table[0, 2] = pages + 7
    pool, gpu = make_pool(rng, 2, pages, 1, size, 8, np.int16)
    want, new = compact_ref(pool, table, lengths, path.reshape(-1), nacc, None, 6)
    got = sv.compact_cache(form(gpu, 1), ints(path.reshape(-1)), ints(nacc), ints(lengths), ints(table))
    assert np.array_equal(got.cpu().numpy(), new) and np.array_equal(gpu.cpu().numpy(), want)
    assert not np.array_equal(want, pool)
    # path[0] other than 0; cu_draft entries out of range
    bad = path[:3].copy()
    bad[1, 0] = 1
    cu = np.array([0, 6, 14, 18])
    want, new = compact_ref(pool, table[:3], lengths[:3], bad.reshape(-1), nacc[:3], cu, 6)
    gpu.copy_(torch.from_numpy(pool))
    got = sv.compact_cache(form(gpu, 1), ints(bad.reshape(-1)), ints(nacc[:3]), ints(lengths[:3]), ints(table[:3]),
                           ints(cu), max_draft=6)
    assert np.array_equal(got.cpu().numpy(), new) and np.array_equal(gpu.cpu().numpy(), want)


def test_compact_strided_pool_and_table(sv):
    """Slabs, pages and positions that are parts of larger tensors, a table with wider rows, every piece size."""
    rng = np.random.default_rng(6)
    for dtype, row, off in ((np.int8, 7, 1), (np.int8, 6, 2), (np.int16, 4, 2), (np.int32, 8, 1), (np.int32, 3, 1)):
        wide = rng.integers(-100, 100, (3, 14, 9, 2, row + 2 * off)).astype(dtype)  # [slabs, pages, size, heads, row]
        gpu = torch.from_numpy(wide.copy()).to(DEV)
        part = gpu[:, 1:13, :8, :, off:off + row].transpose(2, 3)
        pool = wide[:, 1:13, :8, :, off:off + row].transpose(0, 1, 3, 2, 4)
        table = rng.permutation(12).reshape(4, 3)
        held = torch.full((4, 5), 77, dtype=torch.int32, device=DEV)
        held[:, :3] = ints(table)
        drafts, lengths = [5] * 4, np.array([24, 17, 8, 6])
        path = random_paths(rng, drafts, [3, 5, 1, 2])
        want, new = compact_ref(pool, table, lengths, path, np.array([3, 5, 1, 2]), None, 5)
        got = sv.compact_cache(part, ints(path), ints([3, 5, 1, 2]), ints(lengths), held[:, :3])
        wide[:, 1:13, :8, :, off:off + row] = want.transpose(0, 1, 3, 2, 4)
        assert np.array_equal(got.cpu().numpy(), new)
        assert np.array_equal(gpu.cpu().numpy(), wide)  # the surroundings too


FORK = [
    # slabs, heads, row, dtype, page, sequences, places, longest
    (1, 1, 8, np.int16, 16, 1, 1, 40),
    (2, 1, 8, np.int16, 16, 4, 4, 37),
    (3, 2, 5, np.int8, 5, 6, 11, 33),
    (12, 8, 64, np.int16, 16, 8, 8, 100),
    (2, 1, 6, np.int32, 1, 5, 3, 9),
    (4, 1, 256, np.int16, 32, 64, 64, 300),
    (1, 1, 4, np.int8, 3, 1100, 1500, 20),
]


def run_fork(sv, gpu, heads, table, lengths, parents, refs, **kw):
    new = kw.pop("new_lengths", None)
    got = sv.fork_pages(form(gpu, heads), ints(table), ints(lengths), None if parents is None else ints(parents),
                        ints(refs), None if new is None else ints(new), **kw)
    return {k: v.cpu().numpy() for k, v in got.items()}


def check_fork(got, gpu, want):
    assert np.array_equal(got["page_table"], want[1])
    assert np.array_equal(got["refs"], want[2])
    assert got["free"][0] == want[3]
    assert np.array_equal(gpu.cpu().numpy(), want[0])


@pytest.mark.parametrize("slabs,heads,row,dtype,size,old,places,longest", FORK)
@pytest.mark.parametrize("short", [False, True])
def test_fork(sv, slabs, heads, row, dtype, size, old, places, longest, short):
    rng = np.random.default_rng(old * 10 + size)
    lengths = rng.integers(0, longest + 1, old)
    lengths[0] = longest
    most = -(-longest // size) + 1
    table, refs = random_tables(rng, old, most, old * most + 1, lengths, size)
    pages = old * most + (2 if short else 2 * places)  # short: not enough for everybody
    refs = np.concatenate([refs, np.zeros(pages - len(refs), np.int64)])
    refs[table[0, 0]] += 1  # a holder outside the call
    parents = rng.integers(-1, old + 1, places)
    more = lengths[np.clip(parents, 0, old - 1)] + rng.integers(-3, size + 2, places)
    pool, gpu = make_pool(rng, slabs, pages, heads, size, row, dtype)
    for new in (None, more, np.full(places, INT := most * size + 5)):
        want = fork_ref(pool, table, lengths, parents, refs, new)
        gpu.copy_(torch.from_numpy(pool))
        check_fork(run_fork(sv, gpu, heads, table, lengths, parents, refs, new_lengths=new), gpu, want)
    assert INT > longest


def test_fork_many_pages(sv):
    """More pages and table entries than one workgroup counts."""
    rng = np.random.default_rng(8)
    old, size, most, pages = 300, 4, 130, 70001
    lengths = rng.integers(0, most * size + 1, old)
    table, refs = random_tables(rng, old, most, pages, lengths, size, share=0.9)
    refs[rng.permutation(pages)[:20000]] += 1
    parents = rng.integers(0, old, 350)
    pool, gpu = make_pool(rng, 1, pages, 1, size, 2, np.int8)
    want = fork_ref(pool, table, lengths, parents, refs, np.full(350, most * size))
    check_fork(run_fork(sv, gpu, 1, table, lengths, parents, refs, new_lengths=np.full(350, most * size)), gpu, want)


def test_fork_forms(sv):
    """Beams' parents, no parents, counts in place, tables that are no pages, lengths out of range."""
    rng = np.random.default_rng(9)
    size, most = 4, 5
    lengths = np.array([9, 9, 9, 20, 20, 17, -3, 99])
    table, refs = random_tables(rng, 8, most, 60, np.clip(lengths, 0, most * size), size)
    pool, gpu = make_pool(rng, 3, 60, 2, size, 4, np.int16)
    local = np.array([1, 1, 0, 3, 2, 2, -1, 4])
    want = fork_ref(pool, table, lengths, local, refs, lengths + 1, beams=4)
    check_fork(run_fork(sv, gpu, 2, table, lengths, local, refs, new_lengths=lengths + 1, beams=4), gpu, want)
    gpu.copy_(torch.from_numpy(pool))
    want = fork_ref(pool, table, lengths, None, refs, lengths + 2)
    check_fork(run_fork(sv, gpu, 2, table, lengths, None, refs, new_lengths=lengths + 2), gpu, want)
    # counts in place, in a table with entries that are no pages
    table[0, 1], table[3, 4], table[5, 4], table[1, 2] = -1, 60, -7, 2 ** 31 - 1
    parents = np.array([0, 0, 3, 3, 5, 1, 1, 7])
    gpu.copy_(torch.from_numpy(pool))
    want = fork_ref(pool, table, lengths, parents, refs, None)
    held = ints(refs)
    out = {"page_table": torch.full((8, 9), 5, dtype=torch.int32, device=DEV)[:, 2:7], "refs": held,
           "free": torch.empty(1, dtype=torch.int32, device=DEV)}
    got = sv.fork_pages(gpu, ints(table), ints(lengths), ints(parents), held, out=out)
    check_fork({k: v.cpu().numpy() for k, v in got.items()}, gpu, want)
    assert got["refs"] is held


def test_pages_captured(sv):
    """Both calls in a captured graph, replayed with other inputs in the same tensors and eager work between."""
    rng = np.random.default_rng(10)
    size, most, b, k = 4, 8, 6, 7
    lengths = rng.integers(k + 1, most * size - 4, b)
    table, refs = random_tables(rng, b, most, 100, lengths, size, share=0.0)
    pool, gpu = make_pool(rng, 2, 100, 1, size, 16, np.int16)
    t = dict(table=ints(table), lengths=ints(lengths), refs=ints(refs), parents=ints(np.arange(b)),
             path=ints(random_paths(rng, [k] * b, [2] * b)), nacc=ints([2] * b))
    shorter = torch.empty(b, dtype=torch.int32, device=DEV)
    compact = sv.CompactCachePlan(gpu[:, :, 0], t["path"], t["nacc"], t["lengths"], t["table"], out=shorter)
    fork = sv.ForkPagesPlan(gpu[:, :, 0], t["table"], shorter, t["parents"], t["refs"])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        compact()
        fork()
    for turn in range(4):
        acc = [int(x) for x in rng.integers(0, k + 1, b)]
        path, parents = random_paths(rng, [k] * b, acc), rng.integers(0, b, b)
        for name, a in (("path", path), ("nacc", acc), ("parents", parents)):
            t[name].copy_(ints(a))
        gpu.copy_(torch.from_numpy(pool))
        moved, new = compact_ref(pool, table, lengths, path, np.array(acc), None, k)
        want = fork_ref(moved, table, new, parents, refs)
        graph.replay()
        torch.cuda.synchronize()
        assert np.array_equal(shorter.cpu().numpy(), new)
        check_fork({n: v.cpu().numpy() for n, v in fork.out.items()}, gpu, want)
