"""A step of fixed size that holds fewer guesses: cu_draft ends before total_draft.  The sequences get what they get
without the rows behind the last one, and those are left as they were, in every call of the step."""
import numpy as np
import pytest
import torch

import test_gpu_adjust as adjust
import test_gpu_tree_verify as verify
from test_gpu_tree_attention import Case, ints, sv  # noqa: F401

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
PAD = 5


def padded(t, fill):
    """`t` with PAD more rows of `fill`."""
    return torch.cat([t, torch.full((PAD, *t.shape[1:]), fill, dtype=t.dtype, device=t.device)])


@pytest.mark.parametrize("context,drafts,q_heads,kv_heads,dim,size,dtype", [
    ([3000, 40, 900], [2, 0, 4], 8, 2, 128, 16, "bf16"),
    ([100, 40], [3, 1], 8, 2, 128, 16, "f16"),             # a workgroup per pair
    ([5000, 700], [63, 40], 8, 2, 64, 64, "bf16"),         # several row tiles
    ([900], [0], 4, 1, 256, 32, "f16"),
])
def test_attention(sv, context, drafts, q_heads, kv_heads, dim, size, dtype):  # noqa: F811
    c = Case(context, drafts, q_heads, kv_heads, dim, size, dtype, seed=dim)
    most = max(drafts) + PAD
    want = c.run(sv, cu_draft=ints(c.cu), max_draft=most)
    rows = c.q.shape[0]
    out = {"out": torch.full((rows + PAD, q_heads, dim), 7.0, dtype=c.q.dtype, device=DEV),
           "lse": torch.full((rows + PAD, q_heads), 7.0, device=DEV)}
    got = sv.tree_attention(padded(c.q, float("nan")), c.k, c.v,
                            **c.kw(cu_draft=ints(c.cu), max_draft=most, parents=padded(ints(c.parents), 0), out=out))
    for n in ("out", "lse"):
        assert torch.equal(got[n][:rows], want[n])
        assert bool((got[n][rows:] == 7.0).all())
    c.check(want)


@pytest.mark.parametrize("inplace", [False, True])
def test_edits(sv, inplace):  # noqa: F811
    c = adjust.Case([5, 0, 12, 1], 32003, "f16", bias=300, masked="some")
    want = c.call(sv, max_draft=12 + PAD)
    rows = want.shape[0]
    x = padded(c.logits, 3.0)
    out = x if inplace else torch.full_like(x, 7.0)
    a = c.a
    got = c.call(sv, logits=x, out=out, max_draft=12 + PAD, draft_ids=padded(ints(a["ids"]), 0),
                 parents=padded(ints(a["parents"]), 0), mask_rows=padded(ints(a["mask_rows"]), 0))
    assert torch.equal(got[:rows].view(torch.int16), want.view(torch.int16))
    assert bool((got[rows:] == (3.0 if inplace else 7.0)).all())


@pytest.mark.parametrize("how", ["greedy", "sample"])
def test_verify(sv, how):  # noqa: F811
    c = verify.Case([4, 0, 9, 2], 5003, "bf16", seed=3)
    call = sv.verify_tree_greedy if how == "greedy" else sv.verify_tree_sample
    kw = dict(max_draft=9 + PAD, **({} if how == "greedy" else dict(temperature=0.8, top_k=50, top_p=0.9, seed=3)))
    want = call(c.logits, ints(c.ids), **c.kw(), **kw)
    rows = c.logits.shape[0]
    out = {"tokens": torch.full((rows + PAD,), 7, dtype=torch.int32, device=DEV),
           "path": torch.full((rows + PAD,), 7, dtype=torch.int32, device=DEV),
           "num_accepted": torch.full((4,), 7, dtype=torch.int32, device=DEV)}
    got = call(padded(c.logits, 1.0), padded(ints(c.ids), 0), padded(ints(c.parents), 0), cu_draft=ints(c.cu), out=out, **kw)
    assert torch.equal(got["num_accepted"], want["num_accepted"])
    for n in ("tokens", "path"):
        assert torch.equal(got[n][:rows], want[n])
        assert bool((got[n][rows:] == 7).all())


def test_compact(sv):  # noqa: F811
    g = torch.Generator(DEV).manual_seed(1)
    pool = torch.randn(3, 40, 16, 64, generator=g, device=DEV)
    table = ints(np.random.default_rng(1).permutation(40)[:36].reshape(3, 12))
    cu, lengths, taken = ints([0, 4, 4, 10]), ints([60, 170, 100]), ints([2, 0, 4])
    path = ints([0, 2, 4, -1, -1, 0, 0, 1, 3, 4, 6, -1, -1])
    one, two = pool.clone(), pool.clone()
    want = sv.compact_cache(one, path, taken, lengths, table, cu, max_draft=11)
    got = sv.compact_cache(two, padded(path, 3), taken, lengths, table, cu, max_draft=11)
    assert torch.equal(got, want) and torch.equal(one, two) and not torch.equal(one, pool)
