"""Argument checks of the calls on trees of guesses: no GPU is needed, nothing
here reaches a launch."""
import ctypes as C

import pytest
import torch

from tree_util import walk_ref

FAKE = 1 << 40  # never dereferenced


@pytest.fixture(scope="module")
def T():
    import os

    from rejection_sampling_verify_07_amd import binding, tree

    if not os.path.exists(binding.LIB_PATH):
        from rejection_sampling_verify_07_amd import build

        build.build()
    binding.load_library()
    return tree


@pytest.fixture(scope="module")
def lib(T):
    return T.load_library()


def _verify(T, lib, name, logits=FAKE, ids=FAKE, parents=FAKE, filters=(1.0, 0, 1.0, 0, 0), o=(FAKE, FAKE, FAKE), ws=None,
            have=0, **kw):
    d = dict(batch=2, max_draft=4, total_draft=8, vocab=1000, dtype=1, target_row_stride=1000, draft_row_stride=0)
    d.update(kw)
    n = C.c_size_t(have)
    f = filters if name == "spec_verify_tree_sample" else ()
    st = getattr(lib, name)(C.byref(T._b.ShapeT(**d)), logits, ids, parents, *f, *o, ws, C.byref(n), None)
    return st, n.value


CALLS = ("spec_verify_tree_greedy", "spec_verify_tree_sample")


@pytest.mark.parametrize("name", CALLS)
@pytest.mark.parametrize("kw,code", [
    (dict(), 0), (dict(batch=0), 1), (dict(vocab=0), 1), (dict(max_draft=-1), 1), (dict(total_draft=7), 1),
    (dict(total_draft=9, cu_draft=FAKE), 1), (dict(cu_draft=FAKE + 2), 1), (dict(target_row_stride=999), 1),
    (dict(dtype=3), 1), (dict(max_draft=129, total_draft=258), 2), (dict(max_draft=128, total_draft=256), 0),
    (dict(vocab=(1 << 20) + 1, target_row_stride=1 << 21), 2), (dict(max_draft=0, total_draft=0), 0)])
def test_verify_shapes(T, lib, name, kw, code):
    st, need = _verify(T, lib, name, **kw)
    assert st == code and (code or (need > 0 and need % 256 == 0))


@pytest.mark.parametrize("filters,code", [((0.0, 0, 1.0, 0, 0), 1), ((float("nan"), 0, 1.0, 0, 0), 1), ((1.0, -1, 1.0, 0, 0), 1),
                                          ((1.0, 1001, 1.0, 0, 0), 1), ((1.0, 0, 0.0, 0, 0), 1), ((1.0, 0, 1.1, 0, 0), 1),
                                          ((1e-39, 0, 1.0, 0, 0), 1), ((0.7, 50, 0.9, 0, 0), 0)])
def test_verify_filters(T, lib, filters, code):
    assert _verify(T, lib, "spec_verify_tree_sample", filters=filters)[0] == code


@pytest.mark.parametrize("name", CALLS)
def test_verify_pointers(T, lib, name):
    need = _verify(T, lib, name)[1]
    ok = dict(ws=FAKE, have=need)
    for bad in (dict(logits=None), dict(logits=FAKE + 1), dict(ids=None), dict(ids=FAKE + 2), dict(parents=FAKE + 2),
                dict(o=(None, FAKE, FAKE)), dict(o=(FAKE, None, FAKE)), dict(o=(FAKE, FAKE, FAKE + 1)),
                dict(o=(FAKE + 2, FAKE, FAKE)), dict(ws=FAKE + 128)):
        assert _verify(T, lib, name, **{**ok, **bad})[0] == 1, bad
    assert _verify(T, lib, name, ws=FAKE, have=need - 1)[0] == 3


def test_verify_binding_refusals(T):
    x, i = torch.zeros(10, 100), torch.zeros(8, dtype=torch.int32)
    with pytest.raises(ValueError, match="2-D"):
        T.verify_tree_greedy(x[0], i)
    with pytest.raises(ValueError, match="GPU"):
        T.verify_tree_greedy(x, i)
    with pytest.raises(ValueError, match="B\\*\\(K\\+1\\)"):
        T.verify_tree_greedy(x, i[:7])
    with pytest.raises(ValueError, match="max_draft"):
        T.verify_tree_sample(x, i, max_draft=3)


def test_oracle_of_walks():
    assert walk_ref([5, 1, 7, 2], [5, 6, 7], [0, 0, 2], 9) == ([5, 1, -1, -1], 1, [0, 1, -1, -1])
    assert walk_ref([6, 1, 7, 2], [5, 6, 7], [0, 0, 2], 9) == ([6, 7, 2, -1], 2, [0, 2, 3, -1])
    assert walk_ref([6], [], [], 9) == ([6], 0, [0]) and walk_ref([6, 1], [9], [0], 9) is None


# ---- spec_adjust_logits
def _adjust(T, lib, logits=FAKE, out=FAKE, **kw):
    sh = dict(batch=2, max_draft=4, total_draft=8, vocab=1000, dtype=1, row_stride=1000, out_row_stride=1000)
    ad = dict(tokens=FAKE, token_stride=50, max_tokens=50, mask_stride=32, num_masks=10)
    for k, v in kw.items():
        (sh if k in {n for n, _ in T.AdjustShapeT._fields_} else ad)[k] = v
    return lib.spec_adjust_logits(C.byref(T.AdjustShapeT(**sh)), C.byref(T.AdjustT(**ad)), logits, out, None)


@pytest.mark.parametrize("kw,code", [
    (dict(batch=0), 1), (dict(vocab=0), 1), (dict(max_draft=-1), 1), (dict(total_draft=7), 1), (dict(total_draft=-1), 1),
    (dict(total_draft=9, cu_draft=FAKE), 1), (dict(dtype=3), 1), (dict(row_stride=999), 1), (dict(out_row_stride=999), 1),
    (dict(cu_draft=FAKE + 2), 1), (dict(draft_ids=FAKE + 1), 1), (dict(parents=FAKE + 2), 1), (dict(tokens=FAKE + 2), 1),
    (dict(token_stride=49), 1), (dict(max_tokens=-1), 1), (dict(total_bias=-1), 1), (dict(total_bias=3), 1),
    (dict(total_bias=3, bias_ids=FAKE), 1), (dict(total_bias=3, bias_ids=FAKE, bias_values=FAKE + 2), 1),
    (dict(masks=FAKE, mask_stride=31), 1), (dict(masks=FAKE, num_masks=9), 1), (dict(masks=FAKE, num_masks=0, mask_rows=FAKE), 1),
    (dict(masks=FAKE + 2), 1), (dict(repetition=FAKE + 1), 1), (dict(mask_rows=FAKE + 2), 1), (dict(lengths=FAKE + 3), 1),
    (dict(logits=None), 1), (dict(out=None), 1), (dict(logits=FAKE + 1), 1), (dict(out=FAKE + 1), 1),
    (dict(out=FAKE + 2), 1), (dict(out=FAKE + 19998), 1), (dict(out_row_stride=1008), 1), (dict(logits=FAKE + 19998), 1),
    (dict(vocab=(1 << 20) + 1, row_stride=1 << 21, out_row_stride=1 << 21), 2), (dict(max_draft=129, total_draft=258), 2),
    (dict(max_tokens=(1 << 30) + 1, token_stride=1 << 31), 2), (dict(row_stride=1 << 62, out_row_stride=1 << 62), 2),
    (dict(token_stride=1 << 62), 2), (dict(masks=FAKE, mask_stride=1 << 62), 2)])
def test_adjust_refusals(T, lib, kw, code):
    assert _adjust(T, lib, **kw) == code


def test_adjust_longest_text(T, lib):
    """A count of 2^30 would be a table entry's flag.  (Logits that overlap the output are what the longest text that is
    taken is refused for: nothing is launched.)"""
    for n, code in (((1 << 30) - 1, 1), (1 << 30, 2), ((1 << 31) - 1, 2)):
        assert _adjust(T, lib, out=FAKE + 2, max_tokens=n, token_stride=1 << 31) == code
    assert _adjust(T, lib, out=FAKE + 2, tokens=None, max_tokens=1 << 30) == 1


def test_adjust_null(T, lib):
    assert lib.spec_adjust_logits(None, C.byref(T.AdjustT()), FAKE, FAKE, None) == 1
    assert lib.spec_adjust_logits(C.byref(T.AdjustShapeT()), None, FAKE, FAKE, None) == 1


def test_adjust_binding_refusals(T):
    x, i = torch.zeros(10, 100), torch.zeros(8, dtype=torch.int32)
    with pytest.raises(ValueError, match="GPU"):
        T.adjust_logits(x)
    with pytest.raises(ValueError, match="2-D"):
        T.adjust_logits(x[0], draft_ids=i)


# ---- spec_tree_attention
def _tree(T, lib, q=FAKE, k=(FAKE, 4096, 256, 128), v=(FAKE, 4096, 256, 128), scale=0.1, out=FAKE, lse=None, ws=None, have=0,
          **kw):
    d = dict(batch=4, max_draft=5, total_draft=20, q_heads=8, kv_heads=2, head_dim=128, pages=50, page_size=16, max_pages=9,
             dtype=1, table_stride=9, q_row_stride=1024, q_head_stride=128, out_row_stride=1024, out_head_stride=128,
             page_table=FAKE)
    d.update(kw)
    n = C.c_size_t(have)
    st = lib.spec_tree_attention(C.byref(T.TreeShapeT(**d)), q, C.byref(T.CacheT(*k)) if k else None,
                                 C.byref(T.CacheT(*v)) if v else None, scale, out, lse, ws, C.byref(n), None)
    return st, n.value


@pytest.mark.parametrize("kw,code", [
    (dict(), 0), (dict(batch=0), 1), (dict(max_draft=-1), 1), (dict(total_draft=19), 1), (dict(total_draft=-1), 1),
    (dict(total_draft=21, cu_draft=FAKE), 1), (dict(total_draft=7, cu_draft=FAKE), 0), (dict(q_heads=7), 1), (dict(kv_heads=0), 1),
    (dict(pages=0), 1), (dict(page_size=0), 1), (dict(max_pages=0), 1), (dict(table_stride=8), 1), (dict(batch=1, max_draft=20, table_stride=0), 0),
    (dict(page_table=None), 1), (dict(page_table=None, max_pages=1, pages=3), 1), (dict(page_table=None, max_pages=1, page_size=77), 0),
    (dict(page_size=8), 2), (dict(page_size=40), 2), (dict(page_size=48), 0), (dict(dtype=0), 2), (dict(dtype=5), 1), (dict(head_dim=96), 2),
    (dict(head_dim=0), 1), (dict(max_draft=129, total_draft=516), 2), (dict(max_draft=128, total_draft=512), 0),
    (dict(max_pages=(1 << 26) + 1, table_stride=1 << 27), 2), (dict(max_pages=1 << 26, table_stride=1 << 26), 0),
    (dict(max_pages=1 << 26, table_stride=1 << 26, batch=1 << 8, max_draft=0, total_draft=0), 2), (dict(table_stride=1 << 62), 2),
    (dict(cu_draft=FAKE + 2, total_draft=7), 1), (dict(parents=FAKE + 2), 1), (dict(lengths=FAKE + 1), 1), (dict(page_table=FAKE + 2), 1),
    (dict(scale=0.0), 1), (dict(scale=-1.0), 1), (dict(scale=float("nan")), 1), (dict(scale=3e38), 1), (dict(q_heads=1 << 24, kv_heads=1), 2)])
def test_tree_shapes(T, lib, kw, code):
    st, need = _tree(T, lib, **kw)
    assert st == code and (code or (need > 0 and need % 256 == 0))


def test_tree_workspace_does_not_grow_with_the_caches(T, lib):
    assert _tree(T, lib, max_pages=1 << 20, table_stride=1 << 20)[1] == _tree(T, lib, max_pages=1 << 14, table_stride=1 << 14)[1]


def test_tree_pointers(T, lib):
    need = _tree(T, lib)[1]
    ok = dict(ws=FAKE, have=need)
    for bad in (dict(q=None), dict(q=FAKE + 8), dict(out=None), dict(out=FAKE + 4), dict(lse=FAKE + 2), dict(k=None), dict(v=None),
                dict(k=(None, 4096, 256, 128)), dict(k=(FAKE + 8, 4096, 256, 128)), dict(v=(FAKE, 4097, 256, 128)),
                dict(v=(FAKE, 4096, 252, 128)), dict(k=(FAKE, 4096, 256, -128)), dict(q_row_stride=1020), dict(q_head_stride=-8),
                dict(out_row_stride=1022), dict(out_head_stride=64), dict(out_row_stride=512), dict(ws=FAKE + 128)):
        assert _tree(T, lib, **{**ok, **bad})[0] == 1, bad
    assert _tree(T, lib, **ok, k=(FAKE, 1 << 40, 1 << 25, 128))[0] == 2
    assert _tree(T, lib, ws=FAKE, have=need - 1)[0] == 3


def test_tree_strides_that_64_bits_do_not_hold(T, lib):
    """Counted in bytes they would wrap.  (The workspace is too small: nothing is launched.)"""
    need = _tree(T, lib)[1]
    short = dict(ws=FAKE, have=need - 1)
    for far in (1 << 62, (1 << 63) - 8, 1 << 58):
        for at in range(3):
            cache = [4096, 256, 128]
            cache[at] = far
            for name in ("k", "v"):
                assert _tree(T, lib, **short, **{name: (FAKE, *cache)})[0] == 2, (name, at, far)
        for name in ("q_row_stride", "q_head_stride", "out_row_stride", "out_head_stride"):
            assert _tree(T, lib, **short, **{name: far})[0] == 2, (name, far)
    # what is still counted
    for name in ("q_row_stride", "q_head_stride", "out_row_stride", "out_head_stride"):
        assert _tree(T, lib, **short, **{name: 1 << 50})[0] == 3
    for at, stride in ((0, 1 << 50), (1, 1 << 24), (2, 1 << 50)):
        cache = [4096, 256, 128]
        cache[at] = stride
        assert _tree(T, lib, **short, k=(FAKE, *cache))[0] == 3


def test_tree_binding_refusals(T):
    q, k = torch.zeros(6, 4, 64, dtype=torch.bfloat16), torch.zeros(9, 16, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="GPU"):
        T.tree_attention(q, k, k)
    with pytest.raises(ValueError, match="q must be"):
        T.tree_attention(q[0], k, k)
    with pytest.raises(ValueError, match="k must be"):
        T.tree_attention(q, k[0], k)
    with pytest.raises(ValueError, match="do not fit"):
        T.tree_attention(q[:, :3], k, k)
