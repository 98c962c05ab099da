"""spec_tree_attention against the 64-bit form, with the tolerances it derives."""
import numpy as np
import pytest
import torch

from beam_util import DTYPES, widen
from tree_util import random_tree, tree_attention_ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
EPS = {"bf16": 2.0 ** -7, "f16": 2.0 ** -10}
# the smallest weight a kernel keeps whole is far below a row's sum: half of fp16's smallest step under a largest weight
# of 2^10 or more, bf16 has fp32's range
TINY = {"bf16": 0.0, "f16": 2.0 ** -35}


@pytest.fixture(scope="module")
def sv():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import rejection_sampling_verify_07_amd as sv

    sv.load_library()
    return sv


def ints(a):
    return torch.from_numpy(np.ascontiguousarray(a, np.int32)).to(DEV)


class Case:
    """context: positions before the newest rows of each sequence; size 0: one piece per sequence."""

    def __init__(self, context, drafts, q_heads, kv_heads, dim, size, dtype, tree=True, seed=0, spread=2.0, wide=4):
        g = torch.Generator().manual_seed(seed)
        rng = np.random.default_rng(seed)
        b = len(drafts)
        self.drafts, self.dtype, self.dim = list(drafts), dtype, dim
        self.cu = np.concatenate([[0], np.cumsum(drafts)]).astype(np.int64)
        self.lengths = np.array(context) + np.array(drafts) + 1
        rows = int(self.cu[-1]) + b
        mk = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
        dt = DTYPES[dtype]
        self.q = (mk(rows, q_heads, dim) * spread).to(dt).to(DEV)
        longest = int(self.lengths.max())
        if size:
            most = -(-longest // size) + 1
            pages = b * most + 2
            self.table = rng.permutation(pages)[:b * most].reshape(b, most)
            self.table[np.arange(most)[None] * size >= self.lengths[:, None]] = -1
        else:
            size, pages, self.table = longest + 3, b + 1, None
        self.k, self.v = (mk(pages, size, kv_heads, dim).to(dt).to(DEV) for _ in range(2))
        self.parents = np.concatenate([random_tree(rng, k, wide) for k in drafts] + [np.zeros(0, np.int64)]) if tree else None
        self.scale = float(np.float32(dim ** -0.5))

    def kw(self, **kw):
        d = dict(page_table=None if self.table is None else ints(self.table), lengths=ints(self.lengths),
                 parents=None if self.parents is None else ints(self.parents),
                 cu_draft=ints(self.cu) if len(set(self.drafts)) > 1 else None, scale=self.scale, return_lse=True)
        d.update(kw)
        return d

    def run(self, sv, **kw):
        return sv.tree_attention(self.q, self.k, self.v, **self.kw(**kw))

    def ref(self, **kw):
        d = dict(table=self.table, lengths=self.lengths, parents=self.parents, cu=self.cu, scale=self.scale,
                 eps=EPS[self.dtype], tiny=TINY[self.dtype])
        d.update(kw)
        return tree_attention_ref(widen(self.q), widen(self.k), widen(self.v), **d)

    def check(self, got, **kw):
        out, lse, b_out, b_lse = self.ref(**kw)
        o, z = widen(got["out"]), got["lse"].double().cpu().numpy()
        empty = np.isneginf(lse)
        assert np.array_equal(np.isneginf(z), empty)
        far = np.abs(o - out)
        assert np.all(far <= b_out), (far / np.maximum(b_out, 1e-300)).max()
        far = np.abs(z[~empty] - lse[~empty])
        assert np.all(far <= b_lse[~empty]), far.max()


CASES = [
    # context, drafts, q heads, kv heads, dim, page, type
    ([0], [0], 1, 1, 64, 16, "bf16"),
    ([1], [0], 4, 4, 64, 16, "f16"),
    ([500, 37], [0, 0], 8, 8, 64, 16, "f16"),
    ([127, 128, 129, 0], [0] * 4, 8, 2, 128, 32, "bf16"),
    ([1000, 3, 17], [5, 0, 8], 8, 2, 128, 16, "bf16"),
    ([300, 0, 900], [2, 7, 1], 6, 2, 64, 48, "f16"),
    ([700], [15], 2, 1, 128, 64, "f16"),           # 32 rows per key head
    ([33, 400], [16, 3], 4, 2, 128, 16, "bf16"),   # 34: through LDS
    ([63, 64, 65, 1], [20, 9, 31, 0], 8, 2, 64, 16, "f16"),
    ([500, 90], [63, 40], 8, 2, 128, 64, "bf16"),  # two row tiles
    ([10], [128], 2, 1, 64, 16, "bf16"),
    ([257, 100], [128, 64], 5, 1, 128, 112, "f16"),  # six row tiles
    ([200, 31], [3, 1], 8, 2, 256, 16, "bf16"),
    ([300, 64], [12, 30], 4, 2, 256, 32, "f16"),
    ([100], [40], 8, 1, 256, 80, "bf16"),
    ([5, 0, 2000, 1, 0, 600], [1] * 6, 3, 1, 128, 16, "bf16"),
    ([4000], [4], 2, 1, 64, 16, "bf16"),           # one pair over many workgroups
]


@pytest.mark.parametrize("context,drafts,q_heads,kv_heads,dim,size,dtype", CASES)
@pytest.mark.parametrize("form", ["paged", "piece", "chain"])
def test_attention(sv, context, drafts, q_heads, kv_heads, dim, size, dtype, form):
    c = Case(context, drafts, q_heads, kv_heads, dim, 0 if form == "piece" else size, dtype, form != "chain",
             seed=sum(context) + dim)
    c.check(c.run(sv))


def test_many_sequences(sv):
    """More sequences than a workgroup has threads, most of them short, some empty."""
    rng = np.random.default_rng(4)
    context = rng.integers(0, 60, 700)
    context[[5, 300, 699]] = [1500, 900, 2100]
    c = Case(context, [0] * 700, 2, 1, 64, 16, "bf16", seed=4)
    c.lengths[rng.permutation(700)[:100]] = 0
    c.check(c.run(sv))


def test_shapes_against_each_other(sv):
    """A sequence's result does not depend on what else is in the batch but for the borders of parts."""
    c = Case([900, 40, 300], [6, 6, 6], 8, 2, 128, 16, "bf16", seed=9)
    got = c.run(sv)
    one = sv.tree_attention(c.q[7:14], c.k, c.v, **c.kw(page_table=ints(c.table[1:2]), lengths=ints(c.lengths[1:2]),
                                                        parents=ints(c.parents[6:12])))
    tol = 2.0 ** -6 * got["out"][7:14].float().abs().max()
    assert torch.all((one["out"].float() - got["out"][7:14].float()).abs() <= tol)


def test_lengths_and_pages_that_are_none(sv):
    """Lengths out of range, below the newest rows' number, tables with entries that are no pages."""
    c = Case([100, 5, 60, 20, 200], [4, 4, 4, 4, 4], 4, 2, 64, 16, "bf16", seed=5)
    c.lengths = np.array([105, 3, -7, 999, 205])
    c.table[0, [1, 3]] = [-1, 2 ** 31 - 1]
    c.table[4, 12] = c.k.shape[0]  # of the newest rows
    c.check(c.run(sv))
    c.table[0] = -1
    got = c.run(sv)
    c.check(got)
    assert torch.all(got["out"][:5] == 0) and torch.all(got["lse"][:5] == -float("inf"))
    many = Case([100, 300], [40, 40], 4, 1, 128, 16, "f16", seed=6)  # through LDS
    many.table[0, [0, 6]] = -5
    many.table[1, 18] = 10 ** 6
    many.check(many.run(sv))
    many.lengths = np.array([12, 0])
    many.check(many.run(sv))
    # no lengths: all positions
    piece = Case([50, 50], [3, 3], 4, 2, 64, 0, "bf16", seed=7)
    piece.check(piece.run(sv, lengths=None, cu_draft=ints(piece.cu)), lengths=None)


def test_parents_out_of_range(sv):
    c = Case([70], [9], 4, 2, 128, 16, "bf16", seed=8)
    c.parents[[2, 5, 8]] = [-3, 6, 100]
    c.check(c.run(sv))


@pytest.mark.parametrize("dtype,dim,drafts", [("bf16", 64, [5, 5]), ("f16", 128, [40, 12]), ("bf16", 256, [3, 3]),
                                              ("f16", 256, [30, 2]), ("bf16", 128, [20, 20])])
def test_values_that_are_not_finite(sv, dtype, dim, drafts):
    """They reach the rows that see them and no others; what lies behind a length or in another page reaches nobody."""
    c = Case([90, 130], drafts, 4, 2, dim, 16, dtype, seed=dim)
    clean = c.run(sv)
    inf, nan = float("inf"), float("nan")

    def at(b, p):
        return int(c.table[b, p // 16]), p % 16

    first = [int(n) - k - 1 for n, k in zip(c.lengths, c.drafts)]
    # behind the length, in the same page; in a page of nobody
    used = set(c.table.reshape(-1).tolist())
    spare = next(p for p in range(c.k.shape[0]) if p not in used)
    for t in (c.k, c.v):
        t[spare] = nan
        page, off = at(1, int(c.lengths[1]) - 1)
        t[page, off + 1:] = nan
    got = c.run(sv)
    assert torch.equal(got["out"], clean["out"]) and torch.equal(got["lse"], clean["lse"])
    # a value of guess 1's row of sequence 0 (infinite) and of guess 2's (NaN); a NaN key of the last guess of sequence 1
    page, off = at(0, first[0] + 2)
    c.v[page, off, 0, 3] = inf
    page, off = at(0, first[0] + 3)
    c.v[page, off, 1, 7] = nan
    page, off = at(1, first[1] + drafts[1])
    c.k[page, off, 0, 0] = nan
    got = c.run(sv)
    rep = 2
    anc = [set()]
    for j in range(drafts[0]):
        anc.append(anc[int(c.parents[j])] | {j + 1})
    o = got["out"].float().cpu()
    for r in range(drafts[0] + 1):
        want = clean["out"][r].float().cpu().clone()
        if 2 in anc[r]:
            want[:rep, 3] = inf
        if 3 in anc[r]:
            want[rep:, 7] = nan
        assert torch.equal(torch.nan_to_num(o[r], nan=-1e30), torch.nan_to_num(want, nan=-1e30)), r
    row1 = drafts[0] + 1
    assert torch.equal(got["out"][row1:row1 + drafts[1]], clean["out"][row1:row1 + drafts[1]])
    last = o[row1 + drafts[1]]
    assert torch.isnan(last[:rep]).all() and torch.equal(last[rep:], clean["out"][row1 + drafts[1]].float().cpu()[rep:])
    # an infinite value of the context reaches every row
    page, off = at(1, 3)
    c.v[page, off, 1, 0] = -inf
    o = c.run(sv)["out"].float().cpu()
    assert torch.all(o[row1:, rep:, 0] == -inf) and torch.isfinite(o[row1:, rep:, 1:]).all()


def test_strides_and_alignment(sv):
    """Queries, caches and outputs inside larger tensors, heads before positions in the cache, a wide table."""
    for dim, drafts in ((64, [3, 0]), (128, [30, 20]), (256, [2, 5])):
        c = Case([77, 140], drafts, 4, 2, dim, 16, "bf16", seed=11)
        ref = c.run(sv)
        rows = c.q.shape[0]
        wide = torch.zeros(rows, 6, dim + 8, dtype=torch.bfloat16, device=DEV)
        q = wide[:, 1:5, :dim]
        q.copy_(c.q)
        caches = []
        for t in (c.k, c.v):
            big = torch.full((t.shape[0], 3, 16, dim + 16), 9.0, dtype=torch.bfloat16, device=DEV)
            part = big[:, :2, :, 8:8 + dim].transpose(1, 2)
            part.copy_(t)
            caches.append(part)
        table = torch.full((2, c.table.shape[1] + 3), 3, dtype=torch.int32, device=DEV)
        table[:, :-3] = ints(c.table)
        held = torch.full((rows, 5, dim + 4), 7.0, dtype=torch.bfloat16, device=DEV)
        out = {"out": held[:, :4, :dim], "lse": torch.empty(rows, 4, device=DEV)}
        got = sv.tree_attention(q, *caches, **c.kw(page_table=table[:, :-3], out=out))
        assert torch.equal(got["out"], ref["out"]) and torch.equal(got["lse"], ref["lse"])
        assert torch.all(held[:, 4:] == 7.0) and torch.all(held[:, :, dim:] == 7.0)
        # in place of the queries
        got = sv.tree_attention(c.q, c.k, c.v, **c.kw(out={"out": c.q}, return_lse=False))
        assert torch.equal(got["out"], ref["out"])


def test_scores_of_any_size(sv):
    """Large scores and long sums: references move, and far ones stay exact enough."""
    for dtype, spread in (("bf16", 60.0), ("f16", 40.0), ("bf16", 3e5)):
        for drafts in ([2, 1], [30, 33]):
            c = Case([900, 333], drafts, 4, 2, 64, 16, dtype, seed=13, spread=spread)
            c.check(c.run(sv))


def test_against_the_prefix_call(sv):
    """A chain over one-piece caches is spec_prefix_attention without a prefix."""
    c = Case([300, 41], [4, 4], 8, 2, 128, 0, "bf16", tree=False, seed=14)
    got = c.run(sv)
    none = torch.empty(1, 0, 2, 128, dtype=torch.bfloat16, device=DEV)
    ref = sv.prefix_attention(c.q, none, none, c.k[:2], c.v[:2], suffix_lengths=ints(c.lengths), scale=c.scale,
                              return_lse=True)
    assert (got["out"].float() - ref["out"].float()).abs().max() <= 2.0 ** -6 * ref["out"].float().abs().max()
    assert (got["lse"] - ref["lse"]).abs().max() < 1e-4


def test_captured_with_other_lengths(sv):
    """A captured call replayed with other lengths, tables and trees in the same tensors, eager work between; the same
    workspace for two plans in turn."""
    c = Case([900, 40, 300], [6, 6, 6], 8, 2, 128, 16, "bf16", seed=15)
    t = c.kw(lengths=ints(c.lengths))
    plan = sv.TreeAttentionPlan(c.q, c.k, c.v, **t)
    other = sv.TreeAttentionPlan(c.q, c.k, c.v, **c.kw(parents=None, workspace=plan.workspace))
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        plan()
        other()
    rng = np.random.default_rng(1)
    for turn in range(4):
        if turn:
            c.lengths = np.array([int(x) for x in rng.integers(7, 900, 3)])
            c.table = rng.permutation(c.table.reshape(-1)).reshape(c.table.shape)
            c.parents = np.concatenate([random_tree(rng, 6) for _ in range(3)])
            for n, a in (("lengths", c.lengths), ("page_table", c.table), ("parents", c.parents)):
                t[n].copy_(ints(a))
        graph.replay()
        torch.cuda.synchronize()
        c.check(plan.out)
        eager = c.run(sv)
        assert torch.equal(plan.out["out"], eager["out"]) and torch.equal(plan.out["lse"], eager["lse"])


def test_runs_are_equal(sv):
    c = Case([3000, 40, 700], [20, 3, 9], 8, 2, 128, 16, "bf16", seed=16)
    ref = c.run(sv)
    for _ in range(3):
        got = c.run(sv)
        assert torch.equal(got["out"], ref["out"]) and torch.equal(got["lse"], ref["lse"])
