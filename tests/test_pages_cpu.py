"""Argument checks of the calls on paged caches: no GPU is needed, nothing here
reaches a launch."""
import ctypes as C

import numpy as np
import pytest
import torch

from tree_util import compact_ref, fork_ref

FAKE = 1 << 40  # never dereferenced


def at(i):
    return (1 << 44) + (i << 32)


@pytest.fixture(scope="module")
def P():
    import os

    from rejection_sampling_verify_07_amd import binding, pages

    if not os.path.exists(binding.LIB_PATH):
        from rejection_sampling_verify_07_amd import build

        build.build()
    binding.load_library()
    return pages


@pytest.fixture(scope="module")
def lib(P):
    return P.load_library()


def _pool(P, **kw):
    d = dict(slabs=2, pages=40, page_size=16, heads=3, row_bytes=32, slab_stride=40 * 1536, page_stride=1536,
             head_stride=512, position_stride=32)
    d.update({k: v for k, v in kw.items() if k in d})
    return P.PoolT(**d), {k: v for k, v in kw.items() if k not in d}


POOLS = [
    (dict(), 0), (dict(slabs=0), 1), (dict(pages=0), 1), (dict(page_size=0), 1), (dict(heads=0), 1),
    (dict(row_bytes=0), 1), (dict(slab_stride=-1), 1), (dict(page_stride=1535), 1), (dict(head_stride=511), 1),
    (dict(position_stride=31), 1), (dict(position_stride=0), 1), (dict(slab_stride=1 << 62, slabs=3), 1),
    (dict(slabs=1, heads=1, pages=4, row_bytes=1 << 36, position_stride=1 << 36, page_stride=1 << 40), 2)]


def _compact(P, lib, data=FAKE, lengths=at(1), path=at(2), nacc=at(3), out=at(4), **kw):
    pool, kw = _pool(P, **kw)
    d = dict(pool=pool, batch=4, max_draft=5, total_draft=20, max_pages=8, table_stride=8, page_table=at(5))
    d.update(kw)
    return lib.spec_cache_compact(C.byref(P.CompactShapeT(**d)), data, lengths, path, nacc, out, None)


def _fork(P, lib, data=FAKE, table=at(1), lengths=at(2), parents=at(3), new=at(4), refs=at(5), o=(at(6), at(7), at(8)),
          ws=None, have=0, **kw):
    pool, kw = _pool(P, **kw)
    d = dict(pool=pool, old=4, batch=6, beams=0, max_pages=8, table_stride=8, out_table_stride=8)
    d.update(kw)
    n = C.c_size_t(have)
    st = lib.spec_page_fork(C.byref(P.ForkShapeT(**d)), data, table, lengths, parents, new, refs, *o, ws, C.byref(n), None)
    return st, n.value


@pytest.mark.parametrize("kw,code", POOLS)
def test_pools(P, lib, kw, code):
    if code:  # (a sound one would be launched)
        assert _compact(P, lib, **kw) == code
    st, need = _fork(P, lib, **kw)
    assert st == code and (code or (need > 0 and need % 256 == 0))


@pytest.mark.parametrize("kw,code", [
    (dict(batch=0), 1), (dict(max_draft=-1), 1), (dict(total_draft=-1), 1), (dict(max_pages=0), 1),
    (dict(total_draft=19), 1), (dict(total_draft=21, cu_draft=at(9)), 1), (dict(table_stride=7), 1),
    (dict(page_table=None), 1), (dict(page_table=None, max_pages=1, pages=3), 1),
    (dict(max_draft=129, total_draft=516), 2), (dict(max_pages=(1 << 26) + 1, table_stride=1 << 27), 2),
    (dict(data=None), 1), (dict(path=None), 1), (dict(nacc=None), 1), (dict(out=None), 1),
    (dict(lengths=at(1) + 2), 1), (dict(path=at(2) + 1), 1), (dict(nacc=at(3) + 2), 1), (dict(out=at(4) + 1), 1),
    (dict(page_table=at(5) + 2), 1), (dict(cu_draft=at(9) + 2), 1),
    (dict(out=at(1)), 1), (dict(out=at(1) + 12), 1), (dict(out=at(2) + 92), 1), (dict(out=at(5) + 124), 1),
    (dict(lengths=FAKE + 64), 1), (dict(out=FAKE + 1024), 1), (dict(path=FAKE - 92), 1)])
def test_compact_refusals(P, lib, kw, code):
    assert _compact(P, lib, **kw) == code


def test_compact_null_shape(P, lib):
    assert lib.spec_cache_compact(None, FAKE, None, at(2), at(3), at(4), None) == 1
    assert lib.spec_cache_compact_profiled(None, None, FAKE, None, at(2), at(3), at(4), None) == 1


@pytest.mark.parametrize("kw,code", [
    (dict(), 0), (dict(old=0), 1), (dict(batch=0), 1), (dict(beams=-1), 1), (dict(beams=4), 1), (dict(beams=2), 0),
    (dict(max_pages=0), 1), (dict(table_stride=7), 1), (dict(out_table_stride=7), 1),
    (dict(old=1, table_stride=0), 0), (dict(max_pages=(1 << 26) + 1, table_stride=1 << 27, out_table_stride=1 << 27), 2),
    (dict(old=1 << 29), 2), (dict(batch=1 << 29), 2), (dict(table_stride=1 << 62), 2),
    (dict(row_bytes=1 << 24, position_stride=1 << 24, head_stride=1 << 28, page_stride=3 << 28, slab_stride=120 << 28), 0),
    (dict(row_bytes=1 << 29, position_stride=1 << 29, head_stride=1 << 33, page_stride=3 << 33, slab_stride=120 << 33), 2)])
def test_fork_shapes(P, lib, kw, code):
    assert _fork(P, lib, **kw)[0] == code


def test_fork_pointers(P, lib):
    need = _fork(P, lib)[1]
    ok = dict(ws=at(0), have=need)
    for bad in (dict(data=None), dict(table=None), dict(lengths=None), dict(refs=None), dict(o=(None, at(7), at(8))),
                dict(o=(at(6), None, at(8))), dict(o=(at(6), at(7), None)), dict(table=at(1) + 2), dict(parents=at(3) + 1),
                dict(new=at(4) + 2), dict(refs=at(5) + 2), dict(o=(at(6) + 2, at(7), at(8))),
                dict(o=(at(1), at(7), at(8))),             # the new tables over the old
                dict(o=(at(3) + 20, at(7), at(8))),        # over the parents' last
                dict(o=(at(6), at(2), at(8))), dict(o=(at(6), at(5) + 4, at(8))),  # counts beside themselves
                dict(o=(at(6), at(7), at(7) + 4)), dict(o=(at(6), at(6) + 4, at(8))), dict(o=(FAKE, at(7), at(8))),
                dict(table=FAKE + 64), dict(ws=at(0) + 128)):
        assert _fork(P, lib, **{**ok, **bad})[0] == 1, bad
    assert _fork(P, lib, ws=at(0), have=need - 1)[0] == 3
    n = C.c_size_t(0)
    assert lib.spec_page_fork(None, *[None] * 10, C.byref(n), None) == 1


def test_binding_refusals(P):
    x = torch.zeros(2, 6, 4, 8)
    i = torch.zeros(6, dtype=torch.int32)
    with pytest.raises(ValueError, match="GPU"):
        P.compact_cache(x, i, i[:1])
    with pytest.raises(ValueError, match="pool must be"):
        P.compact_cache(x[0, 0], i, i[:1])
    with pytest.raises(ValueError, match="GPU"):
        P.fork_pages(x, i[None], i[:1], None, i)


def test_oracle_of_forks():
    """The plain form itself, on a case that can be followed by hand: three places continue one sequence of two whole
    pages and a started one, a fourth another; the first of the three keeps the started page."""
    pool = np.arange(12 * 2).reshape(1, 12, 1, 2, 1)
    table = np.array([[5, 3, 7, -1], [2, -1, -1, -1]])
    refs = np.zeros(12, int)
    refs[[5, 3, 7, 2]] = 1
    refs[0] = 4
    out, new, counts, left = fork_ref(pool, table, np.array([5, 2]), np.array([0, 1, 0, 0]), refs, np.array([5, 3, 5, 7]))
    assert new.tolist() == [[5, 3, 7, -1], [2, 1, -1, -1], [5, 3, 4, -1], [5, 3, 6, 8]]
    assert counts.tolist() == [4, 1, 1, 3, 1, 3, 1, 1, 1, 0, 0, 0] and left == 3
    assert out[0, 4, 0, :, 0].tolist() == [14, 9] and out[0, 6, 0, :, 0].tolist() == [14, 13]


def test_oracle_of_compaction():
    pool = np.arange(4 * 3).reshape(1, 4, 1, 3, 1)
    out, new = compact_ref(pool, np.array([[2, 0, 1]]), np.array([8]), np.array([0, 2, 3, 5, -1, -1]), np.array([3]), None, 5)
    # positions 0..7 hold 6 7 8 0 1 2 3 4; rows 2, 3 and 5 (positions 4, 5, 7) move to positions 3, 4, 5
    assert out[0, :3, 0, :, 0].tolist() == [[1, 2, 4], [3, 4, 5], [6, 7, 8]] and new.tolist() == [6]
