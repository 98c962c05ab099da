"""The verify, draft and likelihood calls on a stream that is busy: the sizes they read back, and the workspace that they
allocate, belong to the stream of the call."""
import pytest
import torch

from test_gpu_beam_streams import busy

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module")
def sv():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import rejection_sampling_verify_07_amd as sv

    sv.load_library()
    return sv


def inputs():
    g = torch.Generator().manual_seed(6)
    drafts = [0, 9, 3, 6]
    cu = torch.tensor([0, 0, 9, 12, 18], dtype=torch.int32, device=DEV)
    V = 5003
    t = torch.randn(sum(drafts) + 4, V, generator=g).to(DEV)
    d = torch.randn(sum(drafts), V, generator=g).to(DEV)
    ids = torch.randint(0, V, (sum(drafts),), generator=g).int().to(DEV)
    return t, d, ids, cu


def calls(sv, t, d, ids, cu, **kw):
    """The calls as f(stream) -> tensors, and their plans."""
    return {
        "sample": (lambda s: sv.verify_sample(t, d, ids, cu_draft=cu, seed=3, stream=s, **kw),
                   lambda s: sv.SamplePlan(t, d, ids, cu_draft=cu, seed=3, stream=s, **kw)),
        "noalloc": (lambda s: sv.verify_sample_noalloc(t, d, ids, cu_draft=cu, seed=3, stream=s, **kw), None),
        "greedy": (lambda s: sv.verify_greedy(t, ids, cu_draft=cu, stream=s, **kw),
                   lambda s: sv.GreedyPlan(t, ids, cu_draft=cu, stream=s, **kw)),
        "draft": (lambda s: {"ids": sv.draft_sample(d, cu_draft=cu, seed=3, stream=s, **kw)},
                  lambda s: sv.DraftPlan(d, cu_draft=cu, seed=3, stream=s, **kw)),
        "likelihood": (lambda s: sv.token_likelihood(t[:18], d, ids, cu_draft=cu, stream=s, **kw),
                       lambda s: sv.LikelihoodPlan(t[:18], d, ids, cu_draft=cu, stream=s, **kw)),
    }


@pytest.mark.parametrize("name", ["sample", "noalloc", "greedy", "draft", "likelihood"])
def test_sizes_read_back_on_the_stream_of_the_call(sv, name):
    args = inputs()
    cu = args[3]
    call = calls(sv, *args)[name][0]
    ref = call(None)
    torch.cuda.synchronize()
    after = cu.clone()
    cu.copy_(torch.tensor([0, 4, 9, 13, 18], dtype=torch.int32))  # at most 5 a sequence
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    done = busy(s)
    with torch.cuda.stream(s):
        cu.copy_(after)
    assert not done.query()  # (otherwise this shows nothing)
    got = call(s)
    torch.cuda.synchronize()
    for k in ref:
        assert torch.equal(got[k], ref[k]), k


def stream_beside_the_current_one():
    """A stream whose work does not hold the current one's up (several streams may share one hardware queue)."""
    for _ in range(8):
        s = torch.cuda.Stream()
        torch.cuda.synchronize()
        done = busy(s, 6)
        torch.zeros(1, device=DEV)
        torch.cuda.current_stream().synchronize()
        if not done.query():
            return s
    pytest.skip("no stream runs beside the current one")


@pytest.mark.parametrize("name", ["sample", "greedy", "draft", "likelihood"])
def test_workspace_allocated_on_the_stream_of_the_call(sv, name):
    """A workspace that the call allocates and drops is not handed out to others while its stream still works."""
    args = inputs()
    call, plan = calls(sv, *args, max_draft=9)[name]
    ref, size = call(None), plan(None).workspace.numel()
    s = stream_beside_the_current_one()
    warm = [torch.empty(size, dtype=torch.uint8, device=DEV) for _ in range(9)]  # (nothing below waits for memory)
    with torch.cuda.stream(s):
        warm.append(torch.empty(size, dtype=torch.uint8, device=DEV))
    del warm
    torch.cuda.synchronize()
    done = busy(s)
    got = call(s)
    fresh = [torch.full((size,), 7, dtype=torch.uint8, device=DEV) for _ in range(8)]
    torch.cuda.current_stream().synchronize()
    assert not done.query()  # (otherwise this shows nothing)
    torch.cuda.synchronize()
    assert all(bool((f == 7).all()) for f in fresh)
    for k in ref:
        assert torch.equal(got[k], ref[k]), k
