"""What a caller hands to the 8-bit and 4-bit blocks is checked before anything of
the call runs: buffers of another call's sizes, streams of another device."""
import types

import pytest
import torch

from mixture_experts_projections_b200 import rom

BF16, F32 = torch.bfloat16, torch.float32
gpu = pytest.mark.gpu


def test_a_stream_of_another_device_is_refused():
    on = lambda i: types.SimpleNamespace(device=torch.device("cuda", i))  # noqa: E731
    with pytest.raises(rom.RomError, match="the stream is one of cuda:1"):
        rom._scope(on(0), on(1))


@pytest.fixture()
def block():
    """Inputs of 8 tokens, 128 -> 256 -> 128 over 4 experts."""
    T, Dm, De, E = 8, 128, 256, 4
    g = torch.Generator().manual_seed(0)
    w = [torch.randn(E, n, k, generator=g).to(BF16).cuda() for n, k in ((De, Dm), (De, Dm), (Dm, De))]
    x = torch.randn(T, Dm, generator=g).to(BF16).cuda()
    return T, Dm, De, E, x, (0.1 * torch.randn(Dm, E, generator=g)).cuda(), w


def untouched(t):
    """The tensor with its bytes set, and whether they still are."""
    t.view(torch.uint8).fill_(0x5a)
    return lambda: bool((t.view(torch.uint8) == 0x5a).all())


@gpu
@pytest.mark.parametrize("k", [1, 2])
def test_buffers_of_other_sizes_are_refused_before_the_first_launch(block, k):
    T, Dm, De, E, x, w_r, w = block
    q8, w4 = ([c.quantize(t) for t in w] for c in (rom.Q8Weights, rom.W4Weights))
    wrong = [(T - 1, Dm, De, E, k), (T, Dm, De, E, 3 - k), (T, Dm, 128, E, k), (T, 256, De, E, k)]
    for t, dm, de, e, kk in wrong + [(T, Dm, De, 2, k)]:
        b = rom.Q8BlockBuffers(t, dm, de, e, kk, "cuda")
        same = untouched(b.routing.topk_idx)
        with pytest.raises(rom.RomError, match="must be"):
            rom.block_forward_q8(x, w_r, None, *q8, k, bufs=b)
        assert same()
    for t, dm, de, _, kk in wrong:
        b = rom.W4BlockBuffers(t, dm, de, kk, "cuda")
        same = untouched(b.topk_idx)
        with pytest.raises(rom.RomError, match="must be"):
            rom.block_forward_w4(x, w_r, None, *w4, k, bufs=b)
        assert same()
    # buffers of these sizes are taken
    for f, qw, b in ((rom.block_forward_q8, q8, rom.Q8BlockBuffers(T, Dm, De, E, k, "cuda")),
                     (rom.block_forward_w4, w4, rom.W4BlockBuffers(T, Dm, De, k, "cuda"))):
        assert torch.equal(f(x, w_r, None, *qw, k, bufs=b).out, f(x, w_r, None, *qw, k).out)


@gpu
@pytest.mark.parametrize("k", [1, 2])
def test_inproj_outputs_of_other_sizes_are_refused(block, k):
    T, Dm, De, E, x, w_r, w = block
    w4 = rom.W4Weights.quantize(w[0])
    for bad in (torch.empty(T - 1, De, dtype=BF16, device="cuda"), torch.empty(T, De, device="cuda"),
                torch.empty(De, T, dtype=BF16, device="cuda").t()):
        with pytest.raises(rom.RomError, match="out must be"):
            rom.inproj_forward(x, w_r, None, k, w_q4=w4, out=bad)
    with pytest.raises(rom.RomError, match="topk_idx must be"):
        rom.inproj_forward(x, w_r, None, k, w_q4=w4, bufs=rom.RoutingBuffers(T + 1, Dm, E, k, BF16, "cuda"))
    out = torch.empty(T, De, dtype=BF16, device="cuda")
    got, _ = rom.inproj_forward(x, w_r, None, k, w_q4=w4, out=out, bufs=rom.RoutingBuffers(T, Dm, E, k, BF16, "cuda"))
    ref, _ = rom.inproj_forward(x, w_r, None, k, w_q4=w4)
    assert got is out and torch.equal(out, ref)


@gpu
def test_a_larger_workspace_is_taken(block):
    """(A caller may share one over calls of several sizes.)"""
    T, Dm, De, E, x, w_r, w = block
    q8 = [rom.Q8Weights.quantize(t) for t in w]
    b = rom.Q8BlockBuffers(T, Dm, De, E, 1, "cuda")
    b.routing.ws = torch.empty(4096, dtype=torch.int32, device="cuda")
    assert torch.equal(rom.block_forward_q8(x, w_r, None, *q8, 1, bufs=b).out, rom.block_forward_q8(x, w_r, None, *q8, 1).out)
