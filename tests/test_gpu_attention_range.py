"""spec_prefix_attention at the edges of its types' ranges: weights far below a
row's largest, scores far below zero, infinite values next to a cache's end."""
import numpy as np
import pytest
import torch

from beam_util import DTYPES, attention_ref, widen
from test_gpu_attention import Case, sv  # noqa: F401

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
# (sizes, K, Hq, Hk): single rows that walk keys wave by wave, and rows past one wave that share tiles
FEW, MANY = ([4], 0, 4, 2), ([10], 1, 8, 2)


@pytest.mark.parametrize("gap", [9.0, 12.0, 15.0, 16.5, 18.0])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("sizes,K,Hq,Hk", [FEW, MANY])
def test_attention_sink_keys_of_no_value(sv, sizes, K, Hq, Hk, dtype, D, gap):
    """Keys that take nearly all of a row's weight and hold zeros, `gap` above all others: out is what is left of the
    others, each of which has a weight of e^-gap.  In every run of 32 keys, so that no split or wave is without one."""
    P = 2048
    c = Case(sizes, [K] * sum(sizes), Hq, Hk, D, P, K + 1, dtype, seed=int(10 * gap) + D)
    dt = DTYPES[dtype]
    # score = scale * q . k = k[0] + noise of spread 0.1
    c.q = torch.cat([torch.full_like(c.q[..., :1], D ** 0.5), c.q[..., 1:].float() * 0.05], -1).to(dt)
    for k, v in ((c.pk, c.pv), (c.sk, c.sv)):
        k[..., 0] = -gap
        v.copy_((512 + 64 * v.float()).to(dt))
    c.pk[:, ::32, :, 0], c.pv[:, ::32] = 0.0, 0.0
    c.sk[:, ::32, :, 0], c.sv[:, ::32] = 0.0, 0.0
    got = c.run(sv)
    torch.cuda.synchronize()
    # A weight is rounded where its row's largest is 2^10 at least (f16), half a step of the smallest being 2^-25;
    # outputs are far above the smallest step.
    tiny = 2.0 ** -35 if dtype == "f16" else 0.0
    out, lse, b_out, b_lse = attention_ref(
        *(widen(x) for x in (c.q, c.pk, c.pv, c.sk, c.sv)), c.plen, c.slen, c.drafts, c.groups,
        float(np.float32(c.scale)), torch.finfo(dt).eps, tiny)
    assert np.abs(out).min() > 2.0 ** -14
    err = np.abs(widen(got["out"]) - out)
    assert (err <= b_out).all(), (err.max(), (err / np.abs(out)).max())
    assert (np.abs(widen(got["lse"]) - lse) <= b_lse).all()


@pytest.mark.parametrize("power", [20, 56])
@pytest.mark.parametrize("sign", [-1, 1])
@pytest.mark.parametrize("P", [1, 300])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("sizes,K,Hq,Hk", [FEW, MANY])
def test_attention_scores_far_from_zero(sv, sizes, K, Hq, Hk, D, P, sign, power):
    """Every score at +-2^40 or +-2^112 and more: copies of one key, so that all weights are equal."""
    c = Case(sizes, [K] * sum(sizes), Hq, Hk, D, P, 0, "bf16")
    c.q.fill_(1.25 * 2.0 ** power)
    c.pk.fill_(sign * 1.375 * 2.0 ** power)
    score = sign * 1.25 * 1.375 * 2.0 ** (2 * power) * D * float(np.float32(c.scale))
    got = c.run(sv)
    torch.cuda.synchronize()
    v = widen(c.pv)[0].repeat(Hq // Hk, axis=1)  # [P, Hq, D]
    # equal weights (one power of 2, and an exact sum of them): P terms added in fp32, a reciprocal, a product and the
    # rounding of out
    want = np.broadcast_to(v.mean(0), got["out"].shape)
    bound = (2.0 ** -8 * np.abs(want) + (P + 4) * 2.0 ** -24 * np.abs(v).mean(0)) * 1.01
    assert (np.abs(widen(got["out"]) - want) <= bound).all()
    # log2(e) scale, its product with the score, the sum with log2(l), ln 2 and its product: rounded once each
    assert np.abs(widen(got["lse"]) / score - 1).max() <= 5 * 2.0 ** -24


@pytest.mark.parametrize("sizes,K,Hq,Hk", [FEW, MANY])
@pytest.mark.parametrize("dtype,power", [("bf16", 20), ("f16", 14)])
def test_attention_far_scores_choose_one_key(sv, sizes, K, Hq, Hk, dtype, power):
    """Scores of 2^30 and more that grow key by key: all weight is the last key's (or the first one's)."""
    c = Case(sizes, [K] * sum(sizes), Hq, Hk, 64, 200, 0, dtype)
    c.q.fill_(2.0 ** power)
    grow = torch.arange(1, 201, device=DEV).view(1, 200, 1, 1).expand_as(c.pk)
    for sign, at in ((1, 199), (-1, 0)):
        c.pk.copy_(sign * 2.0 ** (power - 7) * grow)
        got = c.run(sv)
        torch.cuda.synchronize()
        want = c.pv[0, at].repeat_interleave(Hq // Hk, 0).expand_as(got["out"])
        assert torch.equal(got["out"], want), (sign, got["out"][0, 0, :4], want[0, 0, :4])


@pytest.mark.parametrize("wild", [float("inf"), float("-inf")])
@pytest.mark.parametrize("P", [1, 70, 321])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("sizes,K,Hq,Hk", [FEW, MANY])
def test_attention_infinite_value_of_the_last_position(sv, sizes, K, Hq, Hk, D, P, wild):
    """The last position in use ends inside a block of keys: its infinite value is every row's, in its column alone."""
    c = Case(sizes, [K] * sum(sizes), Hq, Hk, D, P + 9, 0, "bf16", plen=[P])
    ref = c.run(sv)
    c.pv[0, P - 1, 1, 5] = wild
    got = c.run(sv)
    torch.cuda.synchronize()
    heads = slice(Hq // Hk, None)
    assert (got["out"][:, heads, 5] == wild).all(), got["out"][:2, :, 5]
    got["out"][:, heads, 5] = ref["out"][:, heads, 5]
    assert torch.equal(got["out"], ref["out"]) and torch.equal(got["lse"], ref["lse"])


def test_attention_infinite_value_of_the_newest_row(sv):
    """The same in the suffix of a plain decode step."""
    c = Case([3], [0] * 3, 4, 2, 64, 40, 9, "f16", slen=[9, 1, 5])
    ref = c.run(sv)
    for b in range(3):
        c.sv[b, c.slen[b] - 1, 0, 7] = float("inf")
    got = c.run(sv)
    torch.cuda.synchronize()
    assert (got["out"][:, :2, 7] == float("inf")).all()
    got["out"][:, :2, 7] = ref["out"][:, :2, 7]
    assert torch.equal(got["out"], ref["out"])
