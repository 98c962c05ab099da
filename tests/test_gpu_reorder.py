"""spec_state_reorder on the GPU: bytes are moved, so every result is compared
bit for bit with the out-of-place form, what must not change included."""
import numpy as np
import pytest
import torch

from beam_util import reorder_ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module")
def sv():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import rejection_sampling_verify_07_amd as sv

    sv.load_library()
    return sv


def bits(shape, seed, dtype=torch.int16):
    g = torch.Generator().manual_seed(seed)
    return torch.randint(-(1 << 7) if dtype == torch.int8 else -(1 << 15), 1 << 7 if dtype == torch.int8 else 1 << 15,
                         shape, generator=g).to(dtype)


def check(sv, host, parents, beams, lengths=None, view=lambda t: t, dtype=None):
    """host: the whole storage tensor; view: the states inside it, 5-D."""
    print(f"reorder {tuple(host.shape)} beams={beams} {host.dtype}", flush=True)
    want = host.clone()
    view(want).copy_(reorder_ref(view(host), parents.reshape(-1), beams, lengths))
    dev = host.to(DEV)
    st = view(dev)
    arg = st if dtype is None else st.view(dtype)
    got = sv.reorder_states(arg, parents.to(DEV), beams, None if lengths is None else lengths.to(DEV))
    torch.cuda.synchronize()
    assert got is arg
    assert torch.equal(dev.cpu(), want)


def parents_for(G, W, seed, low=0, high=None):
    return torch.from_numpy(np.random.default_rng(seed).integers(low, high or W, (G, W)).astype(np.int32))


@pytest.mark.parametrize("slabs,G,W,heads,positions,row", [
    (1, 1, 1, 1, 1, 1), (2, 1, 2, 1, 1, 1), (3, 2, 4, 1, 37, 64), (12, 1, 4, 1, 5, 512), (2, 3, 5, 7, 11, 90),
    (2, 2, 8, 2, 129, 128), (1, 2, 9, 1, 33, 80), (3, 1, 16, 3, 17, 65), (1, 2, 17, 1, 20, 64), (2, 1, 64, 2, 9, 40),
    (1, 1, 64, 1, 3, 7), (1, 40, 3, 1, 0, 8), (5, 7, 6, 4, 1, 8)])
@pytest.mark.parametrize("with_lengths", [False, True])
def test_reorder_sizes(sv, slabs, G, W, heads, positions, row, with_lengths):
    host = bits((slabs, G * W, heads, positions, row), 3 * W + row)
    lengths = None
    if with_lengths:
        lengths = torch.from_numpy(np.random.default_rng(W).integers(-2, positions + 3, G * W).astype(np.int32))
    check(sv, host, parents_for(G, W, W), W, lengths)
    check(sv, host, parents_for(G, W, W + 1, -2, W + 2), W, lengths)  # some parents are none


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32, torch.float16, torch.int32])
def test_reorder_moves_every_type(sv, dtype):
    host = bits((2, 6, 1, 10, 32), 1)
    check(sv, host, parents_for(2, 3, 5), 3, dtype=dtype)


def test_reorder_permutations_and_repeats(sv):
    host = bits((2, 8, 1, 50, 64), 2)
    for p in ([1, 2, 3, 4, 5, 6, 7, 0], [7, 6, 5, 4, 3, 2, 1, 0], [3] * 8, list(range(8)), [1, 0, 2, 2, 5, 4, -1, 0]):
        check(sv, host, torch.tensor([p], dtype=torch.int32), 8)


def test_reorder_ranks_of_states(sv):
    """[batch, row], [batch, positions, row], [slabs, batch, positions, row]."""
    W, par = 4, torch.tensor([2, 2, 0, 3, 1, 0, 3, 2], dtype=torch.int32)
    for shape, five in (((8, 6), lambda t: t[None, :, None, None]), ((8, 9, 6), lambda t: t[None, :, None]),
                        ((3, 8, 9, 6), lambda t: t[:, :, None])):
        host = bits(shape, 9)
        want = reorder_ref(five(host), par, W).reshape(shape)
        dev = host.to(DEV)
        sv.reorder_states(dev, par.to(DEV), W)
        assert torch.equal(dev.cpu(), want)


def test_reorder_strided_views(sv):
    """Views of larger storages: other batch places, other positions, padding
    between rows and odd offsets stay untouched."""
    G, W = 2, 3
    par = parents_for(G, W, 4)
    lens = torch.tensor([4, 0, 7, 5, 5, 9], dtype=torch.int32)
    # [slabs, batch, positions, heads, row] seen as [slabs, batch, heads, positions, row]
    host = bits((2, G * W + 2, 12, 4, 24), 6)
    check(sv, host, par, W, lens, lambda t: t[:, 1:1 + G * W, 1:10].permute(0, 1, 3, 2, 4))
    # batch outermost, rows cut on both sides: 2-byte pieces
    host = bits((G * W, 2, 12, 27), 7)
    check(sv, host, par, W, lens, lambda t: t[..., 1:24].permute(1, 0, 2, 3)[:, :, None])
    # 4-byte pieces
    host = bits((G * W, 2, 12, 26), 8)
    check(sv, host, par, W, lens, lambda t: t[..., 2:24].permute(1, 0, 2, 3)[:, :, None])
    # bytes
    host = bits((2, G * W, 1, 12, 27), 8, torch.int8)
    check(sv, host, par, W, lens, lambda t: t[..., 1:])


def test_reorder_offsets_past_32_bits(sv):
    """Slabs 5 GB apart in one allocation of 10 GB."""
    W, rows = 2, 1 << 12
    big = torch.empty((2, W, 5 * (1 << 28)), dtype=torch.int16, device=DEV)
    st = big[:, :, -rows * 8:].view(2, W, 1, rows, 8)
    host = bits((2, W, 1, rows, 8), 12)
    st.copy_(host)
    par = torch.tensor([1, 0], dtype=torch.int32)
    sv.reorder_states(st, par.to(DEV), W)
    torch.cuda.synchronize()
    assert torch.equal(st.cpu(), reorder_ref(host, par, W))


def test_reorder_on_another_stream_and_in_a_graph(sv):
    host = bits((4, 6, 1, 100, 64), 13)
    par = parents_for(2, 3, 8)
    dev, dpar = host.to(DEV), par.to(DEV)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    sv.reorder_states(dev, dpar, 3, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    want = reorder_ref(host, par.reshape(-1), 3)
    assert torch.equal(dev.cpu(), want)
    plan = sv.StateReorderPlan(dev, dpar, 3)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        sv.reorder_states(dev, dpar, 3)
    for seed in (8, 9, 10):
        dpar.copy_(parents_for(2, 3, seed))
        now = dev.cpu()
        g.replay()
        torch.cuda.synchronize()
        want = reorder_ref(now, dpar.cpu().reshape(-1), 3)
        assert torch.equal(dev.cpu(), want)
        plan()  # eager work between the replays
        assert torch.equal(dev.cpu(), reorder_ref(want, dpar.cpu().reshape(-1), 3))
