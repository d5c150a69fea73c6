"""GPU tests of qlinear_attention's sums over long runs of keys that nothing cuts."""
import math

import pytest

from group_wise_affine_qlinear_amd import qlinear as ql

from gpu_helpers import torch_or_skip

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    t = torch_or_skip()
    ql.load_library()
    return t


CASES = [
    # queries, log2 of the keys, D, weight in 128ths, kernel
    (40, 22, 64, 148, "rows128"), (40, 22, 128, 156, "rows128"), (200, 22, 256, 132, "rows256"),
    (32768, 21, 64, 162, "rows256"), (200, 21, 192, 154, "rows256"), (3, 23, 64, 162, "rows32"), (2, 24, 128, 148, "rows32"),
]


@pytest.mark.parametrize("nq,lg,D,weight,kernel", CASES)
def test_equal_weights_of_millions_of_keys(torch, nq, lg, D, weight, kernel):
    """A sum that is rounded the same way with every addition loses more than the output's own rounding.

    The first 128 keys (each wave's first chunk) have the score 0 and the others log(p), p = weight / 128, less than what
    the maximum follows: so the weights are 1 and p exactly (exp2 is off by far less than bf16's half step). The values
    are 1 for the first 8192 keys and 0 behind them, so that their sum ends early: its terms are multiples of 2^-7 and it
    stays below 2^14, exact in fp32. A half of a wave adds up the weights of 16 keys at a time, multiples of
    gcd(weight, 8) / 8, to less than 2^24 of these, as asserted: exact too. What is left is the division (a few 2^-24) and
    the output's rounding, 2^-8. Two weights at a time, the sum is off by 0.8 % (2^21 keys) to 1.7 % (2^22)."""
    n, p = 1 << lg, weight / 128
    share = n // (8 if kernel == "rows32" else 2)  # keys of one half of a wave
    step = math.gcd(weight, 8) / 8                  # sums of 16 weights are multiples of it
    assert share * p < 2 ** 24 * step
    q = torch.zeros((nq, 1, D), dtype=torch.bfloat16, device="cuda")
    q[:, :, 0] = 1.0
    k = torch.zeros((n, 1, D), dtype=torch.bfloat16, device="cuda")
    k[128:, :, 0] = 1.0
    v = torch.zeros_like(k)
    v[:8192] = 1.0
    out = torch.empty_like(q)
    ql.qlinear_attention(q, k, v, out, scale=math.log(p), workspace=None)
    assert ql.qlinear_last_path() == f"attention_{kernel}_slots0"
    want = (128 + 8064 * p) / (128 + (n - 128) * p)
    assert ((out.double() - want).abs() <= (2.0 ** -8 + 2.0 ** -20) * want).all(), (out.double() / want - 1).abs().max().item()


@pytest.mark.parametrize("nq,lg,D,kernel", [(40, 22, 64, "rows128"), (200, 22, 256, "rows256"), (3, 24, 64, "rows32"),
                                            (40, 20, 128, "rows128")])
@pytest.mark.parametrize("weight", [129, 181, 213])
def test_equal_values_stay_within_the_stated_loss(torch, nq, lg, D, kernel, weight):
    """Equal weights of equal values, a different one in each column: sums of 16 products are added n / 16 times (n keys
    of a wave), each rounded by at most 2^-24 of the sum so far: n * 2^-28 in all. The weights' sum is added to n / 32
    times: half of that. The output's rounding is 2^-8 more."""
    n, p = 1 << lg, weight / 128
    q = torch.zeros((nq, 1, D), dtype=torch.bfloat16, device="cuda")
    q[:, :, 0] = 1.0
    k = torch.zeros((n, 1, D), dtype=torch.bfloat16, device="cuda")
    k[128:, :, 0] = 1.0
    value = 1.0 + torch.arange(D, device="cuda") / 128 % 1.0
    v = value.to(torch.bfloat16).expand(n, 1, D).contiguous()
    out = torch.empty_like(q)
    ql.qlinear_attention(q, k, v, out, scale=math.log(p), workspace=None)
    assert ql.qlinear_last_path() == f"attention_{kernel}_slots0"
    run = n // 4 if kernel == "rows32" else n
    off = (out.double() / value - 1).abs().max().item()
    assert off <= 2.0 ** -8 + 1.5 * run * 2.0 ** -28 + 2.0 ** -20, off
