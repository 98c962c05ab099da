"""spec_adjust_logits against the 64-bit form.

Tolerance: a touched element takes at most 5 fp32 roundings (the quotient or product,
frequency * n, two differences, the bias) of values no larger than the sum of its
terms, then one to the element type, eps / 2 of the result (half the smallest
step near 0): 5 * 2^-24 * terms * 1.01 + eps / 2 * |x| + tiny.  Others keep their bits."""
import numpy as np
import pytest
import torch

from beam_util import DTYPES
from tree_util import adjust_ref, random_tree

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
EPS = {"f32": 2.0 ** -23, "bf16": 2.0 ** -7, "f16": 2.0 ** -10}
TINY = {"f32": 2.0 ** -150, "bf16": 2.0 ** -134, "f16": 2.0 ** -25}
INT = {"f32": torch.int32, "bf16": torch.int16, "f16": torch.int16}


@pytest.fixture(scope="module")
def sv():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import rejection_sampling_verify_07_amd as sv

    sv.load_library()
    return sv


def dev(a, dtype=np.int32):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a, dtype)).to(DEV)


class Case:
    def __init__(self, drafts, vocab, dtype, history=50, bias=0, masked=None, tree=True, prompt=True, pad=0, seed=0,
                 guesses=True, shared_bias=False):
        rng = np.random.default_rng(seed)
        b = len(drafts)
        self.drafts, self.V, self.dtype, self.history = list(drafts), vocab, dtype, history
        self.cu = np.concatenate([[0], np.cumsum(drafts)]).astype(np.int64)
        total, rows = int(self.cu[-1]), int(self.cu[-1]) + b
        x = (rng.standard_normal((rows, vocab + pad)) * 4).astype(np.float32)
        self.logits = torch.from_numpy(x).to(DTYPES[dtype]).to(DEV)[:, :vocab]
        self.a = dict(tokens=None, lengths=None, prompt=None, rep=1 + 0.5 * rng.random(b), pres=rng.random(b) - 0.3,
                      freq=0.3 * rng.random(b), ids=None, parents=None)
        if history:
            # a few tokens often, some that are none
            t = (vocab * rng.random((b, history)) ** 3).astype(np.int64)
            t[rng.random((b, history)) < 0.05] = rng.choice([-1, vocab, 2 ** 31 - 1, -2 ** 31])
            self.a.update(tokens=t, lengths=rng.integers(-2, history + 3, b))
            self.a["lengths"][0] = history
            if prompt:
                self.a["prompt"] = rng.integers(-1, history + 2, b)
        if guesses and total:
            self.a["ids"] = (vocab * rng.random(total) ** 3).astype(np.int64)
            if history:  # guesses that are in the text already
                again = rng.random(total) < 0.4
                self.a["ids"][again] = self.a["tokens"][0, 0]
            if tree:
                self.a["parents"] = np.concatenate([random_tree(rng, k) for k in drafts])
        if bias:
            n = bias if shared_bias else bias * b
            cut = np.sort(rng.integers(0, n + 1, b - 1)) if b > 1 else np.zeros(0, int)
            self.a.update(bias_ids=rng.integers(-2, min(vocab, 3 * bias) + 2, n), bias_values=rng.standard_normal(n) * 5,
                          cu_bias=None if shared_bias else np.concatenate([[0], cut, [n]]))
        if masked is not None:
            words = (vocab + 31) // 32 + 1
            bits = rng.random((rows if masked == "rows" else 5, words * 32)) < rng.choice([0.02, 0.5, 0.99, 1.0], (rows if masked == "rows" else 5, 1))
            self.a["masks"] = np.packbits(bits, axis=1, bitorder="little").view(np.int32)
            if masked == "some":
                self.a["mask_rows"] = rng.integers(-2, 7, rows)

    def call(self, sv, logits=None, out=None, plan=False, **kw):
        a = self.a
        ragged = len(set(self.drafts)) > 1
        args = dict(tokens=dev(a["tokens"]), lengths=dev(a["lengths"]), prompt_lengths=dev(a["prompt"]),
                    repetition=dev(a["rep"], np.float32), presence=dev(a["pres"], np.float32),
                    frequency=dev(a["freq"], np.float32), bias_ids=dev(a.get("bias_ids")),
                    bias_values=dev(a.get("bias_values"), np.float32), cu_bias=dev(a.get("cu_bias")),
                    masks=dev(a.get("masks")), mask_rows=dev(a.get("mask_rows")), draft_ids=dev(a["ids"]),
                    parents=dev(a["parents"]), cu_draft=dev(self.cu) if ragged else None, out=out)
        args.update(kw)
        return (sv.AdjustLogitsPlan if plan else sv.adjust_logits)(self.logits if logits is None else logits, **args)

    def check(self, got, before=None):
        before = self.logits if before is None else before
        a = dict(self.a)
        for n in ("rep", "pres", "freq", "bias_values"):  # as the call gets them
            if a.get(n) is not None:
                a[n] = np.asarray(a[n], np.float32)
        want, size = adjust_ref(before.double().cpu().numpy(), self.cu, **a)
        g = got.double().cpu().numpy()
        masked = np.isneginf(want)
        assert np.array_equal(np.isneginf(g), masked)
        same = (size == 0) & ~masked
        assert torch.equal(got.view(INT[self.dtype]).cpu()[torch.from_numpy(same)],
                           before.view(INT[self.dtype]).cpu()[torch.from_numpy(same)])
        far = np.abs(g[~masked] - want[~masked])
        tol = (5 * 2.0 ** -24 * size * 1.01 + EPS[self.dtype] / 2 * np.abs(want) * 1.01 + TINY[self.dtype])[~masked]
        assert np.all(far <= tol), (far / tol).max()
        return size


CASES = {
    "one_row": dict(drafts=[0], vocab=50304, dtype="f32"),
    "one_token": dict(drafts=[0, 0], vocab=1, dtype="bf16"),
    "no_history": dict(drafts=[3, 3], vocab=1000, dtype="f16", history=0),
    "nothing": dict(drafts=[2], vocab=100, dtype="f32", history=0, guesses=False),
    "ragged_tree": dict(drafts=[5, 0, 12, 1], vocab=32003, dtype="f16", bias=300, masked="some", pad=5),
    "chains": dict(drafts=[4] * 6, vocab=9001, dtype="bf16", tree=False, masked="rows"),
    "deep": dict(drafts=[128, 100], vocab=8193, dtype="bf16", bias=3),
    "deep_chain": dict(drafts=[128], vocab=300, dtype="f32", tree=False, bias=1000),
    "shared_bias": dict(drafts=[1, 2], vocab=16390, dtype="f16", bias=70, shared_bias=True, history=1500),
    "long_text": dict(drafts=[2] * 3, vocab=151936, dtype="bf16", history=9001, masked="some"),
    "words_only": dict(drafts=[7] * 5, vocab=4095, dtype="f32", masked="rows", history=0, guesses=False, pad=3),
    "many": dict(drafts=[0] * 700, vocab=501, dtype="f32", history=33, bias=2),
}


@pytest.mark.parametrize("name", sorted(CASES))
@pytest.mark.parametrize("inplace", [False, True])
def test_adjust(sv, name, inplace):
    c = Case(**CASES[name], seed=len(name))
    before = c.logits.clone()
    out = c.logits if inplace else None
    got = c.call(sv, out=out)
    assert (got is c.logits) == inplace
    size = c.check(got, before)
    if name not in ("one_token", "nothing", "words_only"):
        assert (size > 0).any()
    if not inplace:
        assert torch.equal(c.logits.view(INT[c.dtype]), before.view(INT[c.dtype]))


def test_surroundings_are_left(sv):
    """Rows in the middle of wider ones, out of place with another stride and in place: nothing beside them changes."""
    for dtype in ("f32", "bf16", "f16"):
        c = Case([3, 1], 1001, dtype, masked="rows", bias=5, seed=3)
        wide = torch.full((6, 1001 + 24), 7.0, dtype=DTYPES[dtype], device=DEV)
        part = wide[:, 11:1012]
        c.check(c.call(sv, out=part))
        assert torch.all(wide[:, :11] == 7.0) and torch.all(wide[:, 1012:] == 7.0)
        part.copy_(c.logits)
        got = c.call(sv, logits=part, out=part)
        c.check(got)
        assert torch.all(wide[:, :11] == 7.0) and torch.all(wide[:, 1012:] == 7.0)


def test_values_that_are_not_finite(sv):
    """Infinities and NaN keep their places; the type's lowest values follow its rounding; a biased ban is one."""
    for dtype in ("f32", "bf16", "f16"):
        low = torch.finfo(DTYPES[dtype]).min
        x = torch.zeros(1, 64, dtype=DTYPES[dtype])
        x[0, :8] = torch.tensor([float("inf"), -float("inf"), float("nan"), low, low, 1.0, 2.0, -0.0])
        nan_bits = x.view(INT[dtype])[0, 2].item()
        call = dict(tokens=dev([[0, 1, 3, 5, 7]]), repetition=dev([2.0], np.float32), presence=dev([0.5], np.float32),
                    bias_ids=dev([6]), bias_values=dev([-np.inf], np.float32))
        got = sv.adjust_logits(x.to(DEV), **call).cpu()
        assert got[0, 0] == float("inf") and got[0, 1] == -float("inf")
        assert got.view(INT[dtype])[0, 2].item() == nan_bits and got[0, 4] == low  # untouched
        assert got[0, 3] == -float("inf")  # twice the lowest value
        assert got[0, 5] == 0.0 and got[0, 6] == -float("inf") and got[0, 7] == -0.5
        # a NaN that is touched stays one
        got = sv.adjust_logits(x.to(DEV), tokens=dev([[2]]), repetition=dev([2.0], np.float32)).cpu()
        assert torch.isnan(got[0, 2])
        # all masked: the row is -inf whatever it held
        got = sv.adjust_logits(x.to(DEV), masks=dev([[0, 0]])).cpu()
        assert torch.all(got == -float("inf"))


def test_bad_sequences_and_parents(sv):
    """cu_draft entries out of range leave the sequence's rows; parents out of range count as row 0."""
    c = Case([4, 4, 4], 500, "f32", seed=7)
    c.a["parents"][[1, 6]] = [-1, 9]
    c.check(c.call(sv, cu_draft=dev(c.cu), max_draft=4))
    cu = np.array([0, 4, 8, 13])
    out = torch.full_like(c.logits, 7.0)
    got = c.call(sv, cu_draft=dev(cu), max_draft=5, out=out)
    assert torch.all(got[10:] == 7.0) and not torch.any(got[:10] == 7.0)


def test_counts_and_bias_twins(sv):
    """How often a token was written counts exactly, prompt tokens for repetition alone, the last of two biases."""
    x = torch.full((2, 40), 10.0, device=DEV)
    kw = dict(tokens=dev([[3] * 1000 + [4, 5]]), prompt_lengths=dev([1000]), frequency=dev([0.25], np.float32),
              draft_ids=dev([4]))
    got = sv.adjust_logits(x, repetition=dev([2.0], np.float32), bias_ids=dev([9, 9, 9]),
                           bias_values=dev([1.0, 5.0, -2.0], np.float32), **kw)
    assert got[0, 3:6].tolist() == [5.0, 4.75, 4.75] and got[1, 3:6].tolist() == [5.0, 4.5, 4.75]
    assert got[:, 9].tolist() == [8.0, 8.0] and got[:, 10].tolist() == [10.0, 10.0]
    # no penalties: the text changes nothing
    plain = sv.adjust_logits(x, tokens=kw["tokens"], repetition=dev([1.0], np.float32), presence=dev([0.0], np.float32),
                             draft_ids=dev([4]))
    assert torch.equal(plain, x)


def test_captured_and_on_another_stream(sv):
    c = Case([3, 0, 6], 3001, "bf16", masked="some", bias=9, seed=11)
    ref = c.call(sv)
    work = c.logits.clone()
    plan = c.call(sv, logits=work, out=work, plan=True)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        plan()
    for _ in range(3):
        work.copy_(c.logits)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(work.view(torch.int16), ref.view(torch.int16))
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = c.call(sv, stream=s)
    s.synchronize()
    assert torch.equal(got.view(torch.int16), ref.view(torch.int16))
