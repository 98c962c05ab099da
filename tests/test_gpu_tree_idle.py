"""spec_tree_attention where sequences of a batch are empty, as a step with idle slots has them: at the head of the
batch, between others, behind them, or all of them.  Tables that hold many positions, so that the work is dealt and
joined."""
import numpy as np
import pytest
import torch

from test_gpu_tree_attention import Case, ints, sv  # noqa: F401

pytestmark = pytest.mark.gpu


def run(c, sv):  # noqa: F811
    """The call into outputs that hold something else before."""
    plan = sv.TreeAttentionPlan(c.q, c.k, c.v, **c.kw())
    assert plan.workspace.numel() > 65536  # (parts)
    plan.out["out"].fill_(7), plan.out["lse"].fill_(7)
    return plan()


def check(c, got):
    c.check(got)
    for b in np.nonzero(c.lengths <= 0)[0]:
        rows = slice(int(c.cu[b] + b), int(c.cu[b + 1] + b + 1))
        assert not got["out"][rows].any() and bool((got["lse"][rows] == -float("inf")).all())


SHAPES = [
    # drafts, q heads, kv heads, dim, page, type
    ([0, 0, 0, 0], 8, 2, 64, 16, "f16"),
    ([3, 0, 5, 1], 8, 2, 128, 16, "bf16"),
    ([40, 63, 40, 9], 8, 2, 128, 64, "bf16"),  # two row tiles
    ([2, 2, 2, 2], 4, 1, 256, 32, "bf16"),
    ([20, 30, 0, 7], 4, 2, 256, 16, "f16"),
]


@pytest.mark.parametrize("drafts,q_heads,kv_heads,dim,size,dtype", SHAPES)
@pytest.mark.parametrize("lengths", [[0, 0, 0, 0], [0, 4000, 0, 4000], [0, 0, 0, 70], [4000, 0, 0, 0], [-5, 65, 0, 2500]])
def test_empty_sequences(sv, drafts, q_heads, kv_heads, dim, size, dtype, lengths):  # noqa: F811
    c = Case([4000 - k - 1 for k in drafts], drafts, q_heads, kv_heads, dim, size, dtype, seed=dim + len(lengths))
    c.lengths = np.array(lengths)
    check(c, run(c, sv))


@pytest.mark.parametrize("longest", [600, 9000])
def test_many_empty_sequences(sv, longest):  # noqa: F811
    """More sequences than a workgroup has threads, the first 300 of them idle."""
    c = Case([600] + [30] * 699, [0] * 700, 2, 1, 64, 16, "bf16", seed=longest)
    c.lengths = np.zeros(700, np.int64)
    c.lengths[[300, 301, 650]] = [31, longest, 17]
    pages = np.random.default_rng(1).permutation(c.k.shape[0])
    c.table = np.full((700, 600), -1)
    c.table[300, :2], c.table[301], c.table[650, :2] = pages[:2], pages[2:602], pages[602:604]
    check(c, run(c, sv))


def test_empty_sequences_beside_a_long_one(sv):  # noqa: F811
    """So many rounds that every pair, also an empty one, counts some beyond its own."""
    c = Case([5000] * 4, [1, 0, 2, 0], 8, 8, 256, 16, "bf16", seed=2)
    c.table = np.tile(c.table.reshape(1, -1), (4, 1))
    c.table[c.table < 0] = 0
    c.lengths = np.array([0, 20000, 0, 0])
    check(c, run(c, sv))


def test_slots_that_fall_idle_in_a_graph(sv):  # noqa: F811
    c = Case([3000, 500, 2000, 900], [4, 4, 4, 4], 8, 2, 128, 16, "bf16", seed=3)
    full, lengths = c.lengths.copy(), ints(c.lengths)
    plan = sv.TreeAttentionPlan(c.q, c.k, c.v, **c.kw(lengths=lengths))
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        plan()
    for idle in ([], [0], [0, 1], [0, 1, 2, 3], [3], [1, 2]):
        c.lengths = full.copy()
        c.lengths[idle] = 0
        lengths.copy_(ints(c.lengths))
        plan.out["out"].fill_(7), plan.out["lse"].fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        check(c, plan.out)
