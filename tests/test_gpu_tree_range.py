"""The calls on trees and pages at the ends of their ranges: stretches of many rounds, memory further apart than 32 bits
count, most rows."""
import numpy as np
import pytest
import torch

from test_gpu_tree_attention import Case, ints, sv  # noqa: F401
from tree_util import compact_ref, fork_ref, random_tree

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
GIB = 2 ** 30


@pytest.mark.parametrize("context,drafts,q_heads,kv_heads,dim,size,dtype", [
    # pairs of a sequence and a key head times 64 keys, over 512 workgroups: at least 8 rounds each
    ([5300, 4900, 0, 6100, 64, 5100, 4000, 5700, 3900], [0, 2, 1, 0, 3, 0, 1, 0, 0], 8, 8, 64, 16, "bf16"),
    ([9000, 8100, 70, 7999], [1, 0, 2, 0], 12, 12, 128, 32, "f16"),
    ([2300, 3100, 190, 2100, 2900], [2, 0, 1, 1, 0], 16, 16, 256, 48, "bf16"),        # over 256
    ([4200, 1, 3900, 2600, 3500, 2700], [20, 30, 12, 18, 0, 9], 64, 16, 64, 16, "f16"),  # two 16-row tiles per wave
])
def test_long_stretches(sv, context, drafts, q_heads, kv_heads, dim, size, dtype):
    c = Case(context, drafts, q_heads, kv_heads, dim, size, dtype, seed=dim + len(context))
    assert (-(-c.lengths // 64)).sum() * kv_heads >= 8 * (256 if dim == 256 else 512)
    # some rows of each sequence, checked alone: the others' share is in the run all the same
    got = c.run(sv)
    keep = [int(c.cu[b]) + b + r for b, k in enumerate(drafts) for r in sorted({0, k // 2, k})]
    heads = sorted({0, 1, q_heads // 2, q_heads - 1})
    rep = q_heads // kv_heads
    for h in heads:
        one = Case.__new__(Case)
        one.__dict__ = dict(c.__dict__, q=c.q[:, h:h + 1], k=c.k[:, :, h // rep:h // rep + 1], v=c.v[:, :, h // rep:h // rep + 1])
        out, lse, b_out, b_lse = one.ref()
        o = got["out"][:, h:h + 1].double().cpu().numpy()[keep]
        z = got["lse"][:, h:h + 1].double().cpu().numpy()[keep]
        assert np.all(np.abs(o - out[keep]) <= b_out[keep]), h
        assert np.all(np.abs(z - lse[keep]) <= b_lse[keep]), h


@pytest.mark.parametrize("dim,q_heads", [(64, 8), (256, 4)])
def test_most_rows(sv, dim, q_heads):
    """129 rows of 8 or 4 heads on one key head: nine and nine row tiles."""
    c = Case([150, 3], [128, 128], q_heads, 1, dim, 16, "bf16", seed=dim, wide=9)
    c.check(c.run(sv))


def far_apart(shape, strides, dtype):
    """An uninitialised tensor of these strides."""
    extent = sum((n - 1) * s for n, s in zip(shape, strides)) + 1
    return torch.empty(extent, dtype=dtype, device=DEV).as_strided(shape, strides)


@pytest.mark.parametrize("paged", [True, False])
def test_attention_past_32_bits(sv, paged):
    """Pages more than 4 GiB apart; one piece whose positions reach past 4 GiB: the results of the same values packed."""
    if paged:
        c = Case([70, 40], [3, 3], 4, 2, 128, 16, "bf16", seed=1)
        k, v = (far_apart(t.shape, (GIB // 2 // 2, 2 * 128, 128, 1), t.dtype) for t in (c.k, c.v))
    else:  # (position strides of 2 MiB: 2300 positions are 4.5 GiB)
        c = Case([2296], [3], 4, 2, 128, 0, "f16", seed=2)
        c.k, c.v = c.k[:1].contiguous(), c.v[:1].contiguous()
        k, v = (far_apart(t.shape, (0, 2 ** 20, 128, 1), t.dtype) for t in (c.k, c.v))
    assert (k.shape[0] - 1) * k.stride(0) * 2 + (k.shape[1] - 1) * k.stride(1) * 2 > 4 * GIB
    k.copy_(c.k), v.copy_(c.v)
    ref, got = c.run(sv), sv.tree_attention(c.q, k, v, **c.kw())
    torch.cuda.synchronize()
    c.check(ref)
    assert torch.equal(got["out"], ref["out"]) and torch.equal(got["lse"], ref["lse"])


def test_caches_past_32_bits(sv):
    """compact and fork on a pool of two slabs whose pages lie further apart than 4 GiB."""
    rng = np.random.default_rng(3)
    slabs, pages, size, row = 2, 10, 4, 24
    a = rng.integers(-100, 100, (slabs, pages, 1, size, row)).astype(np.int16)
    pool = far_apart((slabs, pages, size, row), (GIB // 8, GIB // 4 + 64, 32, 1), torch.int16)
    assert (pages - 1) * pool.stride(1) * 2 > 4 * GIB
    pool.copy_(torch.from_numpy(a[:, :, 0]))
    table = np.array([[9, 0, 5], [2, 8, 1]])
    lengths, nacc, path = np.array([12, 9]), np.array([2, 3]), np.array([0, 2, 5, -1, -1, -1, 0, 1, 3, 5, -1, -1])
    got = sv.compact_cache(pool, ints(path), ints(nacc), ints(lengths), ints(table))
    want, new = compact_ref(a, table, lengths, path, nacc, None, 5)
    assert np.array_equal(got.cpu().numpy(), new) and np.array_equal(pool.cpu().numpy(), want[:, :, 0])
    refs = np.bincount(table.reshape(-1), minlength=pages)
    lengths, parents = np.array([10, 9]), np.array([1, 0, 0, 1])
    res = sv.fork_pages(pool, ints(table), ints(lengths), ints(parents), ints(refs))
    out, tab, cnt, left = fork_ref(want, table, lengths, parents, refs)
    assert np.array_equal(res["page_table"].cpu().numpy(), tab) and np.array_equal(res["refs"].cpu().numpy(), cnt)
    assert int(res["free"].item()) == left and np.array_equal(pool.cpu().numpy(), out[:, :, 0])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_logits_past_32_bits(sv, dtype):
    """Edits and verifies of rows more than 4 GiB apart: the results of the same rows packed."""
    rng = np.random.default_rng(5)
    K, V = 4, 5003
    ids, ups = ints(rng.integers(0, V, K)), ints(random_tree(rng, K))
    packed = torch.randn(K + 1, V, generator=torch.Generator().manual_seed(1)).to(dtype).to(DEV)
    logits = far_apart((K + 1, V), (GIB + 11, 1), dtype)
    assert K * logits.stride(0) * logits.element_size() > 4 * GIB
    logits.copy_(packed)
    text, rep = ints(rng.integers(0, V, (1, 300))), torch.full((1,), 1.3, device=DEV)
    kw = dict(tokens=text, repetition=rep, presence=rep, draft_ids=ids, parents=ups,
              masks=ints(rng.integers(-2 ** 31, 2 ** 31 - 1, (K + 1, 157))))
    ref = sv.adjust_logits(packed, **kw)
    assert torch.equal(sv.adjust_logits(logits, **kw), ref)
    sv.adjust_logits(logits, out=logits, **kw)
    assert torch.equal(logits, ref)
    for call in (lambda x: sv.verify_tree_greedy(x, ids, ups), lambda x: sv.verify_tree_sample(x, ids, ups, seed=4)):
        a, b = call(logits), call(ref)
        assert all(torch.equal(a[k], b[k]) for k in b)


@pytest.mark.parametrize("context,drafts,q_heads,kv_heads,dim,size,dtype,form", [
    ([100, 37, 0, 5], [0, 3, 1, 7], 8, 2, 128, 16, "bf16", "paged"),
    ([180, 0, 13], [4, 0, 9], 6, 3, 64, 48, "f16", "paged"),
    ([40, 30], [3, 2], 8, 2, 256, 16, "bf16", "paged"),
    ([100, 20], [19, 5], 8, 2, 128, 0, "f16", "piece"),
    ([90, 1], [128, 100], 4, 2, 64, 16, "bf16", "chain"),                      # three row tiles
    (list(range(3, 240, 12)), [k % 4 for k in range(20)], 8, 4, 128, 16, "f16", "paged"),  # 80 workgroups
    (list(range(0, 960, 12)), [k % 3 for k in range(80)], 4, 4, 64, 32, "bf16", "paged"),  # 320
    (list(range(0, 240, 3)), [0] * 80, 4, 4, 256, 16, "bf16", "paged"),
])
def test_pairs_of_one_workgroup(sv, context, drafts, q_heads, kv_heads, dim, size, dtype, form):
    """Tables that hold few positions: a workgroup per pair and no parts, also for empty sequences, pages that are none and
    values that are not finite."""
    c = Case(context, drafts, q_heads, kv_heads, dim, size, dtype, form != "chain", seed=dim + len(context))
    plan = sv.TreeAttentionPlan(c.q, c.k, c.v, **c.kw())
    assert plan.workspace.numel() < 65536  # (no parts)
    plan.out["out"].fill_(7), plan.out["lse"].fill_(7)
    c.check(plan())
    # in the graph's replays too, with other lengths in the same tensor
    graph = torch.cuda.CUDAGraph()
    lengths = ints(c.lengths)
    held = sv.TreeAttentionPlan(c.q, c.k, c.v, **c.kw(lengths=lengths))
    with torch.cuda.graph(graph):
        held()
    for cut in (3, 0, 10 ** 6):
        c.lengths = np.maximum(c.lengths - cut, 0)
        c.lengths[0] = 0
        lengths.copy_(ints(c.lengths))
        held.out["out"].fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        c.check(held.out)
    assert not held.out["out"].any() and bool((held.out["lse"] == -float("inf")).all())


def test_pairs_of_one_workgroup_with_holes(sv):
    c = Case([70, 50, 90], [4, 9, 0], 4, 2, 128, 16, "bf16", seed=3)
    c.table[0, 1], c.table[1, 2], c.table[2, :] = -1, c.k.shape[0], -7
    assert sv.TreeAttentionPlan(c.q, c.k, c.v, **c.kw()).workspace.numel() < 65536
    c.check(c.run(sv))
    # values that are not finite behind the lengths and in other pages reach nobody; in a guess's row the rows that see it
    ref = c.run(sv)
    spare = sorted(set(range(c.k.shape[0])) - set(c.table.reshape(-1).tolist()))
    for t in (c.k, c.v):
        t[spare] = float("nan")
    page, at = int(c.table[1, (c.lengths[1] - 1) // 16]), int((c.lengths[1] - 1) % 16)
    c.v[page, at] = float("inf")  # the last guess's
    c.k[page, at + 1:], c.v[page, at + 1:] = float("nan"), float("inf")
    got = c.run(sv)
    last = int(c.cu[2]) + 1  # its row
    assert torch.equal(got["out"][:last], ref["out"][:last]) and torch.equal(got["out"][last + 1:], ref["out"][last + 1:])
    assert bool(got["out"][last].isinf().all())


@pytest.mark.parametrize("dtype,V", [(torch.float32, 140001), (torch.bfloat16, 280003), (torch.float16, 280000)])
def test_edits_of_many_bytes(sv, dtype, V):
    """Logits of more than 64 MB, in place and apart: what the same sequences get in calls of fewer."""
    rng = np.random.default_rng(6)
    B, K = 30, 3
    rows = B * (K + 1)
    assert rows * V * torch.finfo(dtype).bits // 8 > 64e6 > rows // 2 * V * torch.finfo(dtype).bits // 8
    logits = torch.randn(rows, V, generator=torch.Generator(DEV).manual_seed(2), device=DEV).to(dtype)
    text, ids = rng.integers(0, V, (B, 700)), rng.integers(0, V, B * K)
    ups = np.concatenate([random_tree(rng, K) for _ in range(B)])
    bits = torch.rand(rows, (V + 31) // 32, 32, generator=torch.Generator(DEV).manual_seed(3), device=DEV)
    bits = bits < torch.tensor([0.02, 0.98, 1.0], device=DEV)[torch.arange(rows, device=DEV) % 3][:, None, None]
    words = (bits.long() << torch.arange(32, device=DEV)).sum(2)
    masks = torch.where(words >= 2 ** 31, words - 2 ** 32, words).int()
    rep = 1 + torch.rand(B, device=DEV)

    def call(b0, b1, x, out=None):
        r = slice(b0 * (K + 1), b1 * (K + 1))
        return sv.adjust_logits(x[r], ints(text[b0:b1]), repetition=rep[b0:b1], frequency=rep[b0:b1], masks=masks[r],
                                draft_ids=ints(ids[b0 * K:b1 * K]), parents=ints(ups[b0 * K:b1 * K]), out=out)

    want = torch.cat([call(i, i + B // 2, logits) for i in (0, B // 2)])
    assert torch.equal(call(0, B, logits), want)
    call(0, B, logits, out=logits)
    assert torch.equal(logits, want)
