"""The beam-decoding calls on streams that are busy: what is read back, allocated
and freed belongs to the stream of the call."""
import numpy as np
import pytest
import torch

from test_gpu_attention import Case, sv  # noqa: F401

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def busy(stream, n=24):
    """Some tens of milliseconds of work queued on `stream`; an event behind it."""
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
