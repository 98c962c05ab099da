"""spec_beam_select at scores of every size: masks of the type's lowest value,
start scores of unused beams, scores whose fp64 steps are coarse.  Tokens and
parents against the plain 64-bit form, bit for bit."""
import numpy as np
import pytest
import torch

from beam_util import DTYPES, select_ref, widen
from test_gpu_beam import check, make_logits, sv  # noqa: F401

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def masked(rows, V, dtype, live, seed):
    """Rows whose logits are the type's lowest value but for `live` tokens from the middle of the row."""
    x = torch.full((rows, V), torch.finfo(DTYPES[dtype]).min, dtype=DTYPES[dtype])
    g = torch.Generator().manual_seed(seed)
    at = V // 3 + torch.randint(0, V // 3, (rows, live), generator=g)
    x.scatter_(1, at, torch.randn(rows, live, generator=g).to(DTYPES[dtype]))
    return x.to(DEV)


@pytest.mark.parametrize("T", [0.5, 0.75, 1.0, 1.5])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("G,W,V,n,live", [(3, 2, 5000, 8, 1), (1, 4, 4001, 128, 3), (2, 1, 700, 64, 2)])
def test_select_fewer_unmasked_tokens_than_places(sv, dtype, T, G, W, V, n, live):
    """The places left go to masked tokens, lowest w * V + v first, also where (l - m) / T passes fp32's range."""
    logits = masked(G * W, V, dtype, live, V + n)
    scores = -torch.rand(G * W, generator=torch.Generator().manual_seed(n)) * 4
    check(sv, logits, scores.to(DEV), W, n, T)


def test_select_lowest_value_masks_past_the_lists(sv):
    """More masked blocks than the pick's lists hold."""
    logits = masked(4, 151936, "f32", 3, 1)
    check(sv, logits, torch.tensor([-1.0, -1.5, -0.5, -4.0], device=DEV), 4, 16, 0.7)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("n", [6, 64])
def test_select_smallest_temperature(sv, dtype, n):
    """Every logit but the largest scores below fp32's range (f16 and bf16: with ties)."""
    logits = make_logits(6, 3001, dtype, 13)
    check(sv, logits, torch.tensor([-3.0, -2.0, -5.5, -0.5, -0.25, -4.0], device=DEV), 3, n, 1e-38)


@pytest.mark.parametrize("start", [-1e9, -3e38, -1e4])
@pytest.mark.parametrize("dtype,V", [("f32", 151936), ("bf16", 50304)])
def test_select_start_scores(sv, dtype, V, start):
    """The first step of a search: one beam in use, the others at a score that no candidate reaches."""
    logits = make_logits(2 * 8, V, dtype, 17)
    scores = torch.full((2, 8), start, device=DEV)
    scores[0, 0], scores[1, 3] = 0.0, -1.0
    check(sv, logits, scores.view(-1), 8, 16)


def test_select_start_scores_cost_no_more_than_others(sv):
    """The unused beams' scores leave the filters of the beam in use alone: a call with them takes the time of any
    other (it took several times that when a group shared one error margin)."""
    logits = make_logits(8, 151936, "f32", 19)

    def us(scores):
        plan = sv.BeamSelectPlan(logits, torch.tensor(scores, device=DEV), 8, 16)
        times = []
        for _ in range(9):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            for _ in range(10):
                plan()
            b.record()
            torch.cuda.synchronize()
            times.append(a.elapsed_time(b) * 100)
        return min(times)

    usual, start = us([-0.3 * i for i in range(8)]), us([0.0] + [-1e9] * 7)
    print(f"select: usual scores {usual:.1f} us, start scores {start:.1f} us", flush=True)
    assert start < 2 * usual


def test_select_scores_of_coarse_steps(sv):
    """Scores around -4e10, whose fp64 steps (7.6e-6) are coarser than the window of the near ties.  A group's second
    beam holds the first one's logits in another order: the exact scores tie in pairs, while the two beams' fp32 sums
    differ and may put their scores one step apart."""
    G, V, n = 32768, 300, 4
    g = torch.Generator().manual_seed(23)
    x = torch.randn(G, V, generator=g) * 1.5
    logits = torch.stack([x, x[:, torch.randperm(V, generator=g)]], 1).view(2 * G, V).to(DEV)
    scores = (-4e10 - 1e9 * torch.rand(G, 1, generator=g)).repeat(1, 2).view(-1).to(DEV)
    out = sv.beam_select(logits, scores, 2, n)
    torch.cuda.synchronize()
    _, rt, rp = select_ref(widen(logits), widen(scores), 2, n)
    wrong = (out["tokens"].cpu().numpy() != rt).any(1) | (out["parents"].cpu().numpy() != rp).any(1)
    assert not wrong.any(), f"{wrong.sum()} of {G} groups: {np.argwhere(wrong)[:5].ravel()}"
