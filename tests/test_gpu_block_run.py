"""GPU test of the operators of one block branch together, as a program runs
them: the norm before the block with its AdaLN modulation into FAST
activations and bf16, the quantized projection, the adapters of a ragged batch
of requests beside it with SwiGLU, the down projection with its adapters, and
the norm after with gate and residual, eager and as a captured graph.

The whole is compared with the branch in 64 bits on the same quantized
weights. The branch output is normalised to about 1 and enters the stream
times a gate below 1. What separates the two: h in bf16 (half a step, 2^-8 of
each value) before the first products, the MLP's activation in bf16 (2^-8)
before the second, FAST weights (2^-11), fp32 sums. Independent roundings of
relative size at most 2^-8, uniform (so 2^-8 / sqrt(3) in the mean square),
pass through a product with the mean-square size they had: h's rounding
reaches gate and up (relative 2^-8 / sqrt(3) = 2.3e-3 each, so at most their
sum through silu(g) u with |g silu'(g) / silu(g)| below 1 + |g|, taken as 3),
then the activation's own 2.3e-3: below 3 * 2.3e-3 + 2.3e-3 + 2.3e-3 = 1.2e-2
of the branch in the Frobenius norm. The stream's bf16 rounding adds 2^-8 / sqrt(3)."""
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


@pytest.mark.parametrize("M", [9, 330])
def test_branch(torch, M):
    D, F, bits, rank, n = 512, 640, 4, 16, 3
    g = torch.Generator().manual_seed(M)
    rand = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    weights = {}
    for i, (name, N, K) in enumerate((("up", 2 * F, D), ("down", D, F))):
        q, s16, b16 = oracle.quantize_rtn(inputs.weights(N, K, 40 + i), bits)
        weights[name] = (dev(torch, oracle.pack(q, bits)), dev(torch, s16), dev(torch, b16),
                         oracle.dequantize(q, s16, b16).astype(np.float64))
    stream0 = (rand(M, D) * 2).to(torch.bfloat16).cuda()
    pad = M // 8
    lengths = [M // 3, M // 4, M - pad - M // 3 - M // 4, pad]
    sample = torch.repeat_interleave(torch.tensor([0, 1, 2, -1]), torch.tensor(lengths)).to(torch.int32).cuda()
    ids = torch.repeat_interleave(torch.tensor([2, -1, 0, -1]), torch.tensor(lengths)).to(torch.int32).cuda()
    mod = torch.empty((3, 3 * D)).copy_(torch.cat([0.3 * rand(3, D), 0.2 * rand(3, D), torch.tanh(rand(3, D))], 1)).cuda()
    scale, shift, gate = mod[:, :D], mod[:, D:2 * D], mod[:, 2 * D:]
    w_pre, w_post = (1 + 0.1 * rand(D)).cuda(), (1 + 0.1 * rand(D)).cuda()
    tables = {"up": ((rand(n, rank, D) / D ** 0.5).to(torch.bfloat16).cuda(), (rand(n, 2 * F, rank) * 0.1).to(torch.bfloat16).cuda()),
              "down": ((rand(n, rank, F) / F ** 0.5).to(torch.bfloat16).cuda(), (rand(n, D, rank) * 0.1).to(torch.bfloat16).cuda())}
    scaling = torch.tensor([1.0, 0.5, 2.0]).cuda()
    h = torch.zeros((M, D), dtype=torch.bfloat16, device="cuda")
    x16 = torch.zeros((M, D), dtype=torch.float16, device="cuda")
    rowscale = torch.ones(M, device="cuda")
    y_up = torch.empty((M, 2 * F), device="cuda")
    act = torch.empty((M, F), dtype=torch.bfloat16, device="cuda")
    y_down = torch.empty((M, D), device="cuda")
    stream = stream0.clone()
    sizes = [ql.qlinear_workspace_bytes(bits, M, 2 * F, D), ql.qlinear_workspace_bytes(bits, M, D, F),
             ql.qlinear_adapters_workspace_bytes(M, 2 * F, D, rank, n), ql.qlinear_adapters_workspace_bytes(M, D, F, rank, n)]
    ws = torch.empty(max(sizes), dtype=torch.uint8, device="cuda")

    def branch():
        ql.qlinear_block_norm(stream, M, D, pre_norm=ql.QL_NORM_RMS, pre_weight=w_pre, scale=scale, shift=shift,
                              row_sample=sample, h=h, x16=x16, rowscale=rowscale)
        p, s, b, _ = weights["up"]
        # M <= 16 runs the skinny kernel, which takes the bf16 h alone
        fast = dict(x16=x16, rowscale=rowscale) if M > 16 else {}
        ql.qlinear_forward_ex(h, p, s, b, bits, M, 2 * F, D, y_up, workspace=ws, **fast)
        ql.qlinear_adapters(h, *tables["up"], ids, M, 2 * F, D, act, y=y_up, scaling=scaling,
                            epilogue=ql.QL_EPI_SWIGLU, workspace=ws)
        p, s, b, _ = weights["down"]
        ql.qlinear_forward_ex(act, p, s, b, bits, M, D, F, y_down, workspace=ws)
        ql.qlinear_adapters(act, *tables["down"], ids, M, D, F, y_down, y=y_down, scaling=scaling, workspace=ws)
        ql.qlinear_block_norm(stream, M, D, y=y_down, post_norm=ql.QL_NORM_RMS, post_weight=w_post, gate=gate,
                              row_sample=sample, residual_out=stream)

    branch()
    torch.cuda.synchronize()
    eager = stream.clone()

    live = sample.cpu().numpy() >= 0
    per_row = lambda t: t.double().cpu().numpy()[np.where(live, sample.cpu().numpy(), 0)]  # noqa: E731
    num = lambda t: t.double().cpu().numpy()  # noqa: E731
    r0 = num(stream0)
    _, hr = oracle.block_norm(r0, pre="rms", pre_weight=num(w_pre), scale=per_row(scale), shift=per_row(shift))
    ids_h, s_h = ids.cpu().numpy(), num(scaling)
    up = hr @ weights["up"][3].T + oracle.adapter_delta(hr, num(tables["up"][0]), num(tables["up"][1]), ids_h, None, s_h)
    ar = oracle.swiglu(up, F)
    down = ar @ weights["down"][3].T + oracle.adapter_delta(ar, num(tables["down"][0]), num(tables["down"][1]), ids_h, None, s_h)
    want, _ = oracle.block_norm(r0, down, post="rms", post_weight=num(w_post), gate=per_row(gate))
    got = num(eager)
    branch_size = np.linalg.norm((want - r0)[live])
    err = np.linalg.norm((got - want)[live])
    assert err <= 1.2e-2 * branch_size + 2.0 ** -8 / np.sqrt(3) * np.linalg.norm(want[live]), (err, branch_size)
    # rows behind the last sequence: the stream is left as it was
    assert torch.equal(eager[sample < 0], stream0[sample < 0])

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        branch()
    for _ in range(4):
        stream.copy_(stream0)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(stream, eager)
