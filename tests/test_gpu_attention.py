"""GPU tests of qlinear_attention against its definition in 64 bits.

Tolerance, elementwise, from the arithmetic; u = 2^-24 (fp32, half a step). A
score is a sum of D products in fp32: off by at most (D + 4) u S, with S =
scale * max_j sum_d |q_d k_jd|, the conversion to powers of two, the maximum's
subtraction and the exponential included (3 more roundings of what is at most
2 S, and 2 u of the exponential): a weight is off by the factor 1 + d_s, d_s
<= (D + 16) u S + 4 u to first order, doubled here for the higher orders. Its
rounding to bf16 adds 2^-8, weights below 2^-126 of the largest underflow
(nothing beside the sums). The sum is taken of the rounded weights, so
out = sum p'_j v_j / sum p'_j with p'_j = p_j (1 + d_j), |d_j| <= d, is off by

  sum p_j d_j (v_j - out) / sum p'_j,  at most  d / (1 - d) * A,  A = sum p_j |v_j - out| / sum p_j.

fp32 sums over n keys (and their rescaling by powers that are rounded: one
rounding of each of at most n / 32 followings) add (n + n / 32 + 16) u of sum
p |v| / sum p, the division and the factors of joined pieces a few more, in
the 16. The output is rounded once: 2^-8 of it.
"""
import numpy as np
import pytest

import oracle
from group_wise_affine_qlinear_amd import qlinear as ql

from gpu_helpers import torch_or_skip

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.fixture(scope="module")
def torch():
    t = torch_or_skip()
    ql.load_library()
    return t


def reference(q, k, v, scale, q_offsets=None, k_offsets=None, key_mask=None):
    """(out, tolerance, live) in 64 bits."""
    want, live = oracle.attention(q, k, v, scale, q_offsets, k_offsets, key_mask)
    tol = np.zeros_like(want)
    if q_offsets is None:
        q_offsets, k_offsets = [0, q.shape[0]], [0, k.shape[0]]
    group, D = q.shape[1] // k.shape[1], q.shape[2]
    for q0, q1, k0, k1 in zip(q_offsets[:-1], q_offsets[1:], k_offsets[:-1], k_offsets[1:]):
        keys = np.arange(k0, k1)
        if key_mask is not None:
            keys = keys[key_mask[k0:k1] != 0]
        if len(keys) == 0 or q1 == q0:
            continue
        for h in range(q.shape[1]):
            x, kk, vv = q[q0:q1, h], k[keys, h // group], v[keys, h // group]
            s = scale * (x @ kk.T)
            size = scale * (np.abs(x) @ np.abs(kk).T).max(axis=1, keepdims=True)
            p = np.exp(s - s.max(axis=1, keepdims=True))
            p /= p.sum(axis=1, keepdims=True)
            d = 2.0 ** -8 + 2 * ((D + 16) * U * size + 4 * U)
            o = want[q0:q1, h]
            spread = np.empty_like(o)
            for c in range(0, q1 - q0, 64):  # [queries, keys, D] at once would not fit
                spread[c:c + 64] = np.einsum("qk,qkd->qd", p[c:c + 64], np.abs(vv[None] - o[c:c + 64, None]))
            n = len(keys)
            e = d / (1 - d) * spread + (n + n / 32 + 16) * U * (p @ np.abs(vv))
            tol[q0:q1, h] = e + 2.0 ** -8 * (np.abs(o) + e)
    return want, tol, live


def num(t):
    return t.double().cpu().numpy()


def edges(lengths, first=0):
    return np.cumsum([first] + list(lengths))


def make(torch, nq, nk, hq, hkv, D, seed, spread=2.0):
    g = torch.Generator().manual_seed(seed)
    rand = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    q = (rand(nq, hq, D) * spread).to(torch.bfloat16).cuda()
    k = (rand(nk, hkv, D) + 0.5 * rand(1, hkv, D)).to(torch.bfloat16).cuda()
    v = (rand(nk, hkv, D) + 0.5 * rand(1, hkv, D)).to(torch.bfloat16).cuda()
    return q, k, v


def check(torch, q, k, v, q_len=None, k_len=None, mask=None, first=(0, 0), scale=None, workspace=ql.TORCH_WORKSPACE,
          out=None, keep=None):
    """Runs the call and compares it; q_len, k_len: lengths of samples behind the rows first[0], first[1]."""
    D = q.shape[2]
    out = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device="cuda") if out is None else out
    before = out.clone()
    kw, offsets = {}, (None, None)
    if q_len is not None:
        offsets = edges(q_len, first[0]), edges(k_len, first[1])
        kw = {"q_offsets": torch.tensor(offsets[0], dtype=torch.int32, device="cuda"),
              "k_offsets": torch.tensor(offsets[1], dtype=torch.int32, device="cuda")}
    if mask is not None:
        kw["key_mask"] = torch.tensor(mask, device="cuda")
    inputs = [num(q), num(k), num(v)]
    ql.qlinear_attention(q, k, v, out, scale=scale, workspace=workspace, **kw)
    want, tol, live = reference(*inputs, D ** -0.5 if scale is None else scale, *offsets, mask)
    got = num(out)
    err = np.abs(got - want)[live]
    assert np.isfinite(got[live]).all()
    assert (err <= tol[live]).all(), ((err - tol[live]).max(), err.max())
    assert torch.equal(out[torch.tensor(~live)], before[torch.tensor(~live)])
    return out


SIZES = [
    # queries, keys, query heads, key heads, D: tiles of each height with ends inside, one key, one query, odd groups
    (1, 1, 1, 1, 8), (1, 33, 2, 1, 64), (5, 31, 2, 2, 72), (32, 64, 1, 1, 128), (33, 65, 2, 1, 40), (130, 257, 3, 1, 64),
    (128, 128, 2, 2, 256), (7, 700, 6, 2, 136), (300, 1, 2, 2, 128), (257, 321, 2, 2, 128), (513, 200, 1, 1, 256),
    # tiles behind as many as the card holds, which go 32 rows to a block
    (2500, 70, 26, 26, 128), (1290, 40, 43, 43, 256),
    (260, 515, 2, 1, 96), (400, 700, 2, 2, 192), (130, 300, 2, 1, 160), (9, 3000, 4, 2, 176), (700, 400, 20, 20, 184),
    (33, 1500, 2, 2, 88), (1, 5000, 4, 4, 256), (3, 9001, 8, 1, 64), (140, 3001, 2, 1, 256), (300, 2049, 1, 1, 64),
]


@pytest.mark.parametrize("nq,nk,hq,hkv,D", SIZES)
@pytest.mark.parametrize("workspace", [ql.TORCH_WORKSPACE, None])
def test_one_sample(torch, nq, nk, hq, hkv, D, workspace):
    check(torch, *make(torch, nq, nk, hq, hkv, D, nq + nk), workspace=workspace)


RAGGED = [
    # samples without queries, without keys, of one row, of several tiles
    ([0, 1, 40, 300, 0, 7], [5, 0, 129, 64, 90, 1000]),
    ([257, 3, 128], [31, 65, 700]),
    ([1] * 70, [1 + 37 * i % 400 for i in range(70)]),
    ([0, 0], [3, 4]),
    ([5, 6], [0, 0]),
]


@pytest.mark.parametrize("q_len,k_len", RAGGED)
@pytest.mark.parametrize("hq,hkv,D", [(2, 2, 64), (4, 1, 128), (1, 1, 256), (6, 2, 72), (2, 2, 192)])
@pytest.mark.parametrize("masked", [False, True])
def test_ragged(torch, q_len, k_len, hq, hkv, D, masked):
    """Samples that begin behind rows of no sample and end before others, which stay as they were; what hidden keys,
    and keys of no sample, hold is not seen."""
    q, k, v = make(torch, sum(q_len) + 9, sum(k_len) + 11, hq, hkv, D, len(q_len) + D)
    mask = None
    if masked:
        g = torch.Generator().manual_seed(D)
        mask = (torch.rand(k.shape[0], generator=g) < 0.7).numpy()
        at = edges(k_len, 5)
        mask[at[0]:at[1]] = False           # one sample without any key
        mask[at[-2]:at[-2] + 130] = False   # a run longer than a tile
        hidden = torch.tensor(~mask)
        k[hidden], v[hidden] = float("nan"), float("inf")
    for t in (k, v):
        t[:5], t[5 + sum(k_len):] = float("nan"), float("inf")
    check(torch, q, k, v, q_len, k_len, mask, first=(4, 5))


MANY = [
    # samples, queries of each, keys of each: more samples than a wave has lanes, whose keys are cut into pieces
    (65, lambda i: 1 + i % 3, lambda i: 400 + 97 * i % 3000, 2, 1, 64),
    (131, lambda i: i % 2, lambda i: 1500 + 211 * i % 1000, 1, 1, 128),
    (67, lambda i: 1 + 5 * i % 90, lambda i: 100 + 61 * i % 1200, 1, 1, 72),
    (66, lambda i: 40 if i != 64 else 700, lambda i: 330 + 61 * i % 900, 2, 2, 256),
    (64, lambda i: 40, lambda i: 0 if i % 3 else 1900, 2, 2, 128),
    # one long sample among short ones; two rounds of pieces
    (5, lambda i: 200, lambda i: 6000 if i == 2 else 70, 4, 4, 64),
    (2, lambda i: 260, lambda i: 1500 - 41 * i, 40, 40, 256),
]


@pytest.mark.parametrize("samples,q_of,k_of,hq,hkv,D", MANY)
@pytest.mark.parametrize("workspace", [ql.TORCH_WORKSPACE, None])
def test_many_samples(torch, samples, q_of, k_of, hq, hkv, D, workspace):
    q_len, k_len = [q_of(i) for i in range(samples)], [k_of(i) for i in range(samples)]
    q, k, v = make(torch, sum(q_len) + 6, sum(k_len) + 5, hq, hkv, D, samples)
    assert ql.qlinear_attention_workspace_bytes(q.shape[0], k.shape[0], samples, hq, hkv, D) > 0
    check(torch, q, k, v, q_len, k_len, first=(3, 2), workspace=workspace)


@pytest.mark.parametrize("nq,nk,hq,hkv,D", [(3, 4000, 4, 2, 64), (100, 3000, 2, 2, 128), (300, 3000, 2, 1, 256),
                                            (1290, 40, 43, 43, 256)])
def test_in_place(torch, nq, nk, hq, hkv, D):
    """out is q, also where a tile's keys are cut or its rows go 32 to a block."""
    q, k, v = make(torch, nq, nk, hq, hkv, D, 53)
    want = ql.qlinear_attention(q, k, v, torch.empty_like(q))
    for workspace in (ql.TORCH_WORKSPACE, None):
        again = q.clone()
        check(torch, again, k, v, workspace=workspace, out=again)
        assert workspace is None or torch.equal(again, want)


@pytest.mark.parametrize("nq,nk,D,heads", [(3, 700, 64, 2), (200, 300, 128, 2), (300, 300, 256, 2), (200, 300, 96, 2),
                                           (600, 700, 192, 2), (1290, 50, 256, 43)])
def test_masks(torch, nq, nk, D, heads):
    q, k, v = make(torch, nq, nk, heads, 1 if heads == 2 else heads, D, 5)
    for mask in (np.zeros(nk, bool), np.arange(nk) % 2 == 0, np.arange(nk) == nk - 1, np.arange(nk) >= 256,
                 np.ones(nk, bool), (np.arange(nk) % 3 * 100).astype(np.uint8)):
        check(torch, q, k, v, mask=mask)


@pytest.mark.parametrize("nq", [3, 200, 400])
def test_slices_of_one_projection(torch, nq):
    """q, k, v and out are slices of longer rows; what lies between out's rows stays."""
    D, hq, hkv = 64, 4, 2
    g = torch.Generator().manual_seed(nq)
    full = torch.randn((nq, (hq + 2 * hkv + 1) * D), generator=g).to(torch.bfloat16).cuda()
    cut = lambda a, n: full[:, a * D:(a + n) * D].unflatten(1, (n, D))  # noqa: E731
    long = torch.full((nq, hq + 1, D), 7.0, dtype=torch.bfloat16, device="cuda")
    check(torch, cut(0, hq), cut(hq, hkv), cut(hq + hkv, hkv), out=long[:, :hq])
    assert (long[:, hq] == 7.0).all()
    # in place
    want = long[:, :hq].clone()
    q = cut(0, hq)
    ql.qlinear_attention(q, cut(hq, hkv), cut(hq + hkv, hkv), q)
    assert torch.equal(q, want)


@pytest.mark.parametrize("nq,nk", [(2, 900), (300, 600)])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_wide_scores(torch, nq, nk, D):
    """Scores of some hundreds that grow along the keys, so that the maximum is followed again and again."""
    q, k, v = make(torch, nq, nk, 1, 1, D, 17)
    ramp = torch.linspace(-6, 6, nk, device="cuda")[:, None, None]
    k = (k.float() * 0.3 + ramp * q[:1].float() * 0.3).to(torch.bfloat16)
    check(torch, q, k, v)
    check(torch, q, k.flip(0).contiguous(), v, scale=0.5)
    check(torch, q, k, v, scale=1e-6)
    # the least of scales hides no key more and none less; the largest leaves the best key's value
    mask = np.arange(nk) % 3 != 0
    check(torch, q, k, v, scale=1e-30, mask=mask)
    q, k = torch.ones_like(q), -torch.ones_like(k)
    k[nk // 2] = 1.0
    out = torch.empty_like(q)
    ql.qlinear_attention(q, k, v, out, scale=1e30)
    assert torch.equal(out, v[nk // 2].expand_as(out))


@pytest.mark.parametrize("nq", [2, 40, 300])
@pytest.mark.parametrize("D", [64, 256])
def test_values_that_are_not_finite_stay_with_their_query(torch, nq, D):
    q, k, v = make(torch, nq, 333, 2, 2, D, 23)
    clean = check(torch, q, k, v)
    q[1, 0, 3] = float("nan")
    out = torch.empty_like(clean)
    ql.qlinear_attention(q, k, v, out)
    assert torch.isnan(out[1, 0]).all()
    out[1, 0] = clean[1, 0]
    assert torch.equal(out, clean)
    # an infinite value reaches its head's queries, in its own column
    q[1, 0, 3] = 0.0
    clean = check(torch, q, k, v)
    v[7, 1, 5] = float("inf")
    ql.qlinear_attention(q, k, v, out)
    assert (torch.isinf(out[:, 1, 5]) | torch.isnan(out[:, 1, 5])).all()
    out[:, 1, 5] = clean[:, 1, 5]
    assert torch.equal(out, clean)


@pytest.mark.parametrize("nq,nk,hkv,D", [(1, 4096, 2, 128), (64, 5000, 1, 256), (300, 1000, 3, 64), (2000, 640, 9, 256)])
def test_repeatable_and_same_without_waits(torch, nq, nk, hkv, D):
    """The same bits from call to call, from a side stream, and beside another call with a workspace of its own."""
    q, k, v = make(torch, nq, nk, hkv, hkv, D, 29)
    first = check(torch, q, k, v) if nq * nk <= 400000 else ql.qlinear_attention(q, k, v, torch.empty_like(q))
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [torch.empty_like(q) for _ in streams]
    torch.cuda.synchronize()
    for _ in range(3):
        for s, o in zip(streams, outs):
            ql.qlinear_attention(q, k, v, o, stream=s)
    torch.cuda.synchronize()
    for o in outs:
        assert torch.equal(o, first)


@pytest.mark.parametrize("nq,nk,D", [(4, 2000, 128), (300, 900, 64), (520, 700, 256)])
def test_graph_with_other_lengths(torch, nq, nk, D):
    """A captured call serves other offsets and another mask after they are overwritten."""
    q, k, v = make(torch, nq, nk, 2, 1, D, 31)
    qo = torch.zeros(4, dtype=torch.int32, device="cuda")
    ko, mask = torch.zeros_like(qo), torch.ones(nk, dtype=torch.bool, device="cuda")
    ws = torch.empty(ql.qlinear_attention_workspace_bytes(nq, nk, 3, 2, 1, D) + 16, dtype=torch.uint8, device="cuda")
    out = torch.zeros_like(q)

    def call(o, w):
        ql.qlinear_attention(q, k, v, o, q_offsets=qo, k_offsets=ko, key_mask=mask, workspace=w)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        call(out, ws)
    seen = []
    for a, b in (([0, 1, 2, nq], [0, 500, 600, nk]), ([0, 0, 0, nq], [3, 4, 5, 6]), ([1, 2, 3, 4], [0, nk // 2, nk, nk]),
                 ([0, nq // 2, nq, nq], [0, 100, 400, 400])):
        qo.copy_(torch.tensor(a))
        ko.copy_(torch.tensor(b))
        mask.copy_(torch.arange(nk) % (3 + a[1] % 5) != 0)
        eager = torch.zeros_like(q)
        torch.cuda.synchronize()
        call(eager, ql.TORCH_WORKSPACE)
        out.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, eager)
        seen.append(eager)
    assert not torch.equal(seen[0], seen[1]) and seen[0].abs().sum() > 0


def test_keys_past_4_gib(torch):
    """A cache whose rows lie past 32-bit byte offsets: the last sample's keys and a sample in the middle."""
    D, hkv, nk = 256, 2, 2300000
    k = torch.full((nk, 2 * hkv, D), float("nan"), dtype=torch.bfloat16, device="cuda")  # 4.7 GB, k and v in turn
    q, kk, vv = make(torch, 3, 700, hkv, hkv, D, 37)
    a, b = 1100000, nk - 400
    k[a:a + 300, :hkv], k[a:a + 300, hkv:] = kk[:300], vv[:300]
    k[b:, :hkv], k[b:, hkv:] = kk[300:], vv[300:]
    out = torch.empty_like(q)
    offsets = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    # the second of the samples, without queries, holds what lies between
    ql.qlinear_attention(q, k[:, :hkv], k[:, hkv:], out, q_offsets=offsets(0, 2, 2, 3),
                         k_offsets=torch.tensor([a, a + 300, b, nk], dtype=torch.int32, device="cuda"))
    want, tol, _ = reference(num(q), num(kk), num(vv), D ** -0.5, [0, 2, 3], [0, 300, 700])
    assert (np.abs(num(out) - want) <= tol).all()


def test_one_long_sample(torch):
    """One sample across 4 GiB of keys, all of them hidden but some at its ends."""
    D, nk = 256, 4300000
    kv = torch.full((nk, 2, D), float("nan"), dtype=torch.bfloat16, device="cuda")  # 4.4 GB
    q, kk, vv = make(torch, 2, 200, 1, 1, D, 41)
    mask = torch.zeros(nk, dtype=torch.bool, device="cuda")
    mask[:100], mask[-100:] = True, True
    for rows, part in ((slice(0, 100), slice(0, 100)), (slice(nk - 100, nk), slice(100, 200))):
        kv[rows, :1], kv[rows, 1:] = kk[part], vv[part]
    out = torch.empty_like(q)
    ql.qlinear_attention(q, kv[:, :1], kv[:, 1:], out, key_mask=mask)
    want, tol, _ = reference(num(q), num(kk), num(vv), D ** -0.5)
    assert (np.abs(num(out) - want) <= tol).all()


def test_no_keys_and_no_queries(torch):
    D = 64
    q, k, v = make(torch, 5, 3, 2, 2, D, 43)
    out = torch.full_like(q, 7.0)
    ql.qlinear_attention(q, k[:0], v[:0], out)
    assert (out == 0).all()
    ql.qlinear_attention(q[:0], k, v, out[:0])
    none = torch.zeros(1, dtype=torch.int32, device="cuda")
    out.fill_(7.0)
    ql.qlinear_attention(q, k, v, out, q_offsets=none, k_offsets=none)
    assert (out == 7.0).all()


def test_offsets_that_are_out_of_order_touch_nothing_outside(torch):
    """Such offsets give unspecified values in out, and none elsewhere."""
    D, nq, nk = 64, 40, 300
    q, k, v = make(torch, nq, nk, 2, 2, D, 47)
    space = torch.full((nq + 2, 2, D), 7.0, dtype=torch.bfloat16, device="cuda")
    need = ql.qlinear_attention_workspace_bytes(nq, nk, 4, 2, 2, D)
    ws = torch.full((need + 4096,), 77, dtype=torch.uint8, device="cuda")
    for a, b in (([40, 0, 40, 0, 40], [300, 0, 300, 0, 300]), ([-5, 60, -7, 100, 2000000000], [-5, 600, -700, 1000, 2000000000]),
                 ([2147483647, -2147483648, 0, 0, 40], [0, 300, 0, 300, 0])):
        ql.qlinear_attention(q, k, v, space[1:-1], q_offsets=torch.tensor(a, dtype=torch.int32, device="cuda"),
                             k_offsets=torch.tensor(b, dtype=torch.int32, device="cuda"), workspace=ws[:need] if need else ws[:16])
        torch.cuda.synchronize()
        assert (space[0] == 7.0).all() and (space[-1] == 7.0).all() and (ws[need + 16:] == 77).all()


def test_run_from_projection_to_projection(torch):
    """The operators of a block's attention branch together, on a padded ragged batch: QKV projection, head norms and
    rotation, attention within the samples, the output projection with gate and residual.

    Against the branch in 64 bits on the same quantized weights. Independent roundings of at most 2^-8, uniform (2^-8 /
    sqrt(3) in the mean square): q, k and v in bf16 and the weights of the softmax. A score sums D products, each off by
    two such factors: relative to the scores' spread (about scale * |q| |k| = 1 here) 2 * 2^-8 / sqrt(3), which a weight
    takes as a factor; with the weight's own and v's rounding below 5 * 2.3e-3 of the attention's output in the
    Frobenius norm, its bf16 rounding one more, FAST weights 2^-11 twice: below 6 * 2.3e-3 = 1.4e-2 of the branch. The
    stream's rounding adds 2^-8 / sqrt(3) of the stream."""
    from group_wise_affine_qlinear_amd import inputs
    from gpu_helpers import dev
    bits, H, D, M, pad = 4, 4, 64, 330, 23
    W = H * D
    g = torch.Generator().manual_seed(3)
    rand = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    weights = {}
    for i, (name, N, K) in enumerate((("qkv", 3 * W, W), ("out", W, W))):
        qq, s16, b16 = oracle.quantize_rtn(inputs.weights(N, K, 60 + i), bits)
        weights[name] = (dev(torch, oracle.pack(qq, bits)), dev(torch, s16), dev(torch, b16),
                         oracle.dequantize(qq, s16, b16).astype(np.float64))
    x = rand(M, W).to(torch.bfloat16).cuda()
    stream0 = rand(M, W).to(torch.bfloat16).cuda()
    stream = stream0.clone()
    at = [0, 100, 101, M - pad]
    offsets = torch.tensor(at, dtype=torch.int32, device="cuda")
    gate = torch.tanh(rand(1, W)).cuda()
    wq, wk = (1 + 0.1 * rand(D)).cuda(), (1 + 0.1 * rand(D)).cuda()
    f, a = ql.qlinear_rope_table_host(10000.0, [D // 4, D // 8, D // 8])
    freqs, axis = torch.tensor(f).cuda(), torch.tensor(a).cuda()
    pos = torch.stack([torch.arange(M), torch.arange(M) // 16, torch.arange(M) % 16]).to(torch.int32).cuda()
    y = torch.empty((M, 3 * H, D), device="cuda")
    qkv = torch.zeros((M, 3 * H, D), dtype=torch.bfloat16, device="cuda")
    o = torch.zeros((M, H, D), dtype=torch.bfloat16, device="cuda")
    cut = lambda t: (t[:, :H], t[:, H:2 * H], t[:, 2 * H:])  # noqa: E731
    ws = torch.empty(max(ql.qlinear_workspace_bytes(bits, M, 3 * W, W), ql.qlinear_workspace_bytes(bits, M, W, W),
                         ql.qlinear_attention_workspace_bytes(M, M, 3, H, H, D)), dtype=torch.uint8, device="cuda")

    def branch():
        p, s, b, _ = weights["qkv"]
        ql.qlinear_forward_ex(x, p, s, b, bits, M, 3 * W, W, y.view(M, 3 * W), workspace=ws)
        q, k, v = cut(y)
        qo, ko, vo = cut(qkv)
        ql.qlinear_qk_norm_rope(M, D, q=q, k=k, v=v, q_out=qo, k_out=ko, v_out=vo, norm=ql.QL_NORM_RMS, q_weight=wq,
                                k_weight=wk, freqs=freqs, pair_axis=axis, positions=pos, rows_end=offsets[-1:])
        ql.qlinear_attention(qo, ko, vo, o, q_offsets=offsets, k_offsets=offsets, workspace=ws)
        p, s, b, _ = weights["out"]
        ql.qlinear_forward_ex(o.view(M, W), p, s, b, bits, M, W, W, stream, epilogue=ql.QL_EPI_GATE_RESIDUAL,
                              residual=stream, gate=gate, gate_rows=M, workspace=ws)

    branch()
    torch.cuda.synchronize()
    eager = stream.clone()
    yr = (num(x) @ weights["qkv"][3].T).reshape(M, 3 * H, D)
    qr = oracle.qk_norm_rope(yr[:, :H], num(wq), "rms", 1e-6, num(pos), f, a)
    kr = oracle.qk_norm_rope(yr[:, H:2 * H], num(wk), "rms", 1e-6, num(pos), f, a)
    ar, live = oracle.attention(qr, kr, yr[:, 2 * H:], D ** -0.5, at, at)
    want = num(stream0) + num(gate) * (ar.reshape(M, W) @ weights["out"][3].T)
    err = np.linalg.norm((num(eager) - want)[live])
    size = np.linalg.norm((want - num(stream0))[live])
    assert err <= 1.4e-2 * size + 2.0 ** -8 / np.sqrt(3) * np.linalg.norm(want[live]), (err, size)
    assert torch.equal(eager[~torch.tensor(live)], stream0[~torch.tensor(live)])

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


def test_two_graphs_share_a_workspace(torch):
    """Nothing in a workspace is kept: graphs that share one may be replayed in any order, one after the other."""
    a, b = make(torch, 2, 3000, 2, 1, 128, 59), make(torch, 300, 1500, 2, 2, 256, 61)
    need = [ql.qlinear_attention_workspace_bytes(q.shape[0], k.shape[0], 1, q.shape[1], k.shape[1], q.shape[2])
            for q, k, _ in (a, b)]
    assert min(need) > 0
    ws = torch.empty(max(need), dtype=torch.uint8, device="cuda")
    want = [check(torch, *x) for x in (a, b)]
    outs = [torch.zeros_like(x[0]) for x in (a, b)]
    graphs = []
    for x, o in zip((a, b), outs):
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1], stream=side):
            ql.qlinear_attention(*x, o, workspace=ws)
    for order in ((0, 1), (1, 0), (0, 0), (1, 1)):
        for o in outs:
            o.zero_()
        for i in order:
            graphs[i].replay()
        ws.fill_(255)  # eager work between the replays
        torch.cuda.synchronize()
        for i in set(order):
            assert torch.equal(outs[i], want[i])
