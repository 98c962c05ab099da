"""The beam-decoding calls on streams that are busy: what is read back, allocated
and freed belongs to the stream of the call."""
import numpy as np
import pytest
import torch

from test_gpu_attention import Case, sv  # noqa: F401

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def busy(stream, n=80):
    """About n milliseconds of work queued on `stream`; an event behind it."""
    with torch.cuda.stream(stream):
        x = torch.full((8192, 8192), 2.0 ** -13, dtype=torch.bfloat16, device=DEV)
        for _ in range(n):
            x = x @ x
        done = torch.cuda.Event()
        done.record()
    return done


@pytest.mark.parametrize("what", ["cu_draft", "cu_groups"])
def test_attention_reads_sizes_back_on_its_stream(sv, what):
    """cu_draft and cu_groups that the call's stream still has to write."""
    if what == "cu_draft":
        c = Case([3], [0, 9, 3], 16, 2, 64, 300, 20, "bf16")
        cu, before = c.cu, [0, 4, 8, 12]
    else:
        c = Case([1, 11], [1] * 12, 16, 2, 64, 300, 20, "bf16")
        cu, before = c.cug, [0, 6, 12]
    ref = c.run(sv)
    torch.cuda.synchronize()
    c.check(ref)
    after = cu.clone()
    cu.copy_(torch.tensor(before, dtype=torch.int32))
    plen, slen = torch.from_numpy(c.plen).to(DEV), torch.from_numpy(c.slen).to(DEV)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    done = busy(s)
    with torch.cuda.stream(s):
        cu.copy_(after)
    assert not done.query()  # (otherwise this shows nothing)
    got = sv.prefix_attention(c.q, c.pk, c.pv, c.sk, c.sv, plen, slen, cu_draft=c.cu, cu_groups=c.cug, scale=c.scale,
                              return_lse=True, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(got["out"], ref["out"]) and torch.equal(got["lse"], ref["lse"])


def test_attention_lse_beside_a_given_out(sv):
    """return_lse with an out that holds none: the call adds one and leaves the caller's dict alone."""
    c = Case([3], [1] * 3, 4, 2, 64, 100, 8, "bf16")
    ref = c.run(sv)
    for given in ({}, {"lse": None}):
        mine = {"out": torch.empty_like(ref["out"]), **given}
        got = c.run(sv, out=mine)
        torch.cuda.synchronize()
        assert got["out"] is mine["out"] and mine.get("lse") is None
        assert torch.equal(got["out"], ref["out"]) and torch.equal(got["lse"], ref["lse"])
    assert "lse" not in c.run(sv, return_lse=False)


def test_memory_of_plans_outlives_their_work_on_other_streams(sv):
    """Plans made for one stream, called on another that is busy, and dropped: none of their memory is handed out
    before that stream has done its work, and the results are those of a quiet call."""
    g = torch.Generator().manual_seed(4)
    logits = torch.randn(32, 20000, generator=g).to(DEV)
    scores = -torch.rand(32, generator=g).to(DEV)
    c = Case([4], [1] * 4, 8, 2, 64, 900, 20, "bf16")
    select, attn = sv.beam_select(logits, scores, 4, 8), c.run(sv)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    done = busy(s)
    plans = [sv.BeamSelectPlan(logits, scores, 4, 8), sv.PrefixAttentionPlan(c.q, c.pk, c.pv, c.sk, c.sv,
                                                                             return_lse=True)]
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = [{k: v.clone() for k, v in p().items()} for p in plans]
    blocks = {t.data_ptr(): t.numel() * t.element_size() for p in plans for t in (p.workspace, *p.out.values())}
    del plans
    fresh = [torch.full((size,), 7, dtype=torch.uint8, device=DEV) for size in blocks.values() for _ in range(4)]
    assert not done.query()  # (otherwise this shows nothing)
    assert not blocks.keys() & {t.data_ptr() for t in fresh}
    torch.cuda.synchronize()
    assert all(torch.equal(got[0][k], select[k]) for k in select)
    assert all(torch.equal(got[1][k], attn[k]) for k in attn)
