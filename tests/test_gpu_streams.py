"""GPU tests of calls queued on the current stream and on another one with no
wait between them, each with memory that the binding takes for it: both give
the bits of a call that ran alone. The inputs are complete before the first
call, and no call reads what another writes, so that nothing but memory that
the calls would share could order or mix them.
"""
import numpy as np
import pytest

import oracle
from group_wise_affine_qlinear_amd import inputs
from group_wise_affine_qlinear_amd import qlinear as ql

from gpu_helpers import dev, torch_or_skip

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    t = torch_or_skip()
    ql.load_library()
    return t


def in_turn(torch, calls, outs, want, rounds=8):
    """calls[i](stream) on the current stream and on a side stream in turn, the side stream as an object and a handle."""
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for r in range(rounds):
        for o in outs:
            o.fill_(float("nan"))
        torch.cuda.synchronize()
        calls[0](None)
        calls[1](side if r % 2 else side.cuda_stream)
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            assert torch.equal(o, w), r
    # the legacy default stream by its handle, behind the side stream's call
    with torch.cuda.stream(side):
        calls[0](None)
        calls[1](0)
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert torch.equal(o, w)


@pytest.mark.parametrize("M,N,K,rank", [(1500, 1024, 1024, 32), (40, 512, 4608, 64)])
def test_adapters(torch, M, N, K, rank):
    calls, outs, want = [], [], []
    for seed in (1, 2):
        g = torch.Generator().manual_seed(seed)
        x = torch.randn((M, K), generator=g).to(torch.bfloat16).cuda()
        a = (torch.randn((4, rank, K), generator=g) / K ** 0.5).to(torch.bfloat16).cuda()
        b = (torch.randn((4, N, rank), generator=g) / rank ** 0.5).to(torch.bfloat16).cuda()
        ids = torch.sort(torch.randint(0, 4, (M,), generator=g)).values.to(torch.int32).cuda()
        out = torch.empty((M, N), device="cuda")
        call = lambda stream, args=(x, a, b, ids, M, N, K, out): ql.qlinear_adapters(*args, stream=stream)  # noqa: E731
        call(None)
        torch.cuda.synchronize()
        calls.append(call)
        outs.append(out)
        want.append(out.clone())
    in_turn(torch, calls, outs, want)


@pytest.mark.parametrize("M,N,K,bits", [(1024, 512, 1024, 4), (12, 512, 4608, 4)])
def test_forward(torch, M, N, K, bits):
    calls, outs, want = [], [], []
    for seed in (1, 2):
        q, s16, b16 = oracle.quantize_rtn(inputs.weights(N, K, seed), bits)
        x = dev(torch, inputs.activations_bf16(M, K, seed))
        p, s, b = dev(torch, oracle.pack(q, bits)), dev(torch, s16), dev(torch, b16)
        out = torch.empty((M, N), device="cuda")
        call = lambda stream, args=(x, p, s, b, bits, M, N, K, out): ql.qlinear_forward_ex(*args, stream=stream)  # noqa: E731
        call(None)
        torch.cuda.synchronize()
        assert np.isfinite(out.cpu().numpy()).all()
        calls.append(call)
        outs.append(out)
        want.append(out.clone())
    in_turn(torch, calls, outs, want)


def test_results_of_a_call_on_another_stream(torch):
    """The FAST activations that a call takes memory for: made on a side stream while the current one still works
    on a block of the same size that was just freed, then read and freed on the current stream."""
    M, K = 2048, 4608
    x = dev(torch, inputs.activations_bf16(M, K, 3))
    want, want_scale = (t.clone() for t in ql.qlinear_fast_activations(x, M, K))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for r in range(6):
        busy = torch.zeros((M, K), dtype=torch.float16, device="cuda")
        for _ in range(4):
            busy += 1
        kept = busy.clone()
        del busy
        x16, scale = ql.qlinear_fast_activations(x, M, K, stream=side if r % 2 else side.cuda_stream)
        torch.cuda.current_stream().wait_stream(side)
        got, got_scale = x16.clone(), scale.clone()
        del x16, scale
        ql.qlinear_fast_activations(x * 2, M, K, stream=None)
        torch.cuda.synchronize()
        assert torch.equal(got, want) and torch.equal(got_scale, want_scale), r
        assert bool((kept == 4).all()), r


def test_captured_on_the_stream_that_is_given(torch):
    """A call that is given the capturing stream, as an object or a handle, takes its scratch from the graph's memory."""
    M, N, K, rank = 300, 512, 1024, 32
    g = torch.Generator().manual_seed(5)
    x = torch.randn((M, K), generator=g).to(torch.bfloat16).cuda()
    a = (torch.randn((4, rank, K), generator=g) / K ** 0.5).to(torch.bfloat16).cuda()
    b = (torch.randn((4, N, rank), generator=g) / rank ** 0.5).to(torch.bfloat16).cuda()
    ids = torch.randint(0, 4, (M,), generator=g).to(torch.int32).cuda()
    want = ql.qlinear_adapters(x, a, b, ids, M, N, K, torch.empty((M, N), device="cuda"))
    side = torch.cuda.Stream()
    graphs, outs = [], []
    for stream in (side, side.cuda_stream):
        side.wait_stream(torch.cuda.current_stream())
        outs.append(torch.empty((M, N), device="cuda"))
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1], stream=side):
            ql.qlinear_adapters(x, a, b, ids, M, N, K, outs[-1], stream=stream)
    for r in range(4):
        for out in outs:
            out.fill_(float("nan"))
        eager = ql.qlinear_adapters(x, a, b, ids, M, N, K, torch.empty((M, N), device="cuda"), stream=side)
        torch.cuda.synchronize()
        for graph in graphs:
            graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(eager, want) and all(torch.equal(out, want) for out in outs), r
