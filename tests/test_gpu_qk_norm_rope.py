"""GPU tests of qlinear_qk_norm_rope against its definition in 64 bits.

Tolerance, elementwise, from the arithmetic. u = 2^-24 is fp32's rounding (at
most half a step). A head's sums are taken by lanes of 8 values and then over
at most 32 lanes, one rounding each: 8 + 5 roundings of the sum of magnitudes,
below 16 u with the products' own. So the mean is off by 16 u * mean|x|, the
variance by 16 u of itself beside the centring's share, and N(x), the
reciprocal square root included, by at most

  e_N = 32 u (|n| + rstd * (|x| + mean|x|)).

The weight adds one u. An angle is a 64-bit product reduced by whole turns and
rounded to fp32 turns: off by at most 2^-25 turns (a magnitude of at most 1/2)
= 2 pi 2^-25 < 4 u, the sine and cosine themselves by at most 4 u: 8 u. A
turned value a c - b s is off by the errors of a and b, 8 u (|a| + |b|) from
the angle and 2 u (|a| + |b|) from its own roundings. The output is rounded
once more: 2^-8 of it (half a step of bf16). Far positions add nothing: the
64-bit product is off by 2^-52 of at most 2^31 turns, 2^-21 turns; the cases
here stay below 2^24 turns (2^-28).
"""
import numpy as np
import pytest

import oracle
from group_wise_affine_qlinear_amd import qlinear as ql

from gpu_helpers import torch_or_skip

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
KIND = {"none": ql.QL_NORM_NONE, "rms": ql.QL_NORM_RMS, "layer": ql.QL_NORM_LAYER}
LAYOUT = {"halves": ql.QL_ROPE_HALVES, "pairs": ql.QL_ROPE_PAIRS}
EPS = 1e-6


@pytest.fixture(scope="module")
def torch():
    t = torch_or_skip()
    ql.load_library()
    return t


def num(t):
    return t.double().cpu().numpy()


def bound(x, weight, norm, positions, freqs, axis, layout):
    """The result in 64 bits and how far the kernel's may be from it."""
    x = np.asarray(x, dtype=np.float64)
    n = oracle.qk_norm_rope(x, None, norm, EPS)
    if norm == "none":
        e = np.zeros_like(x)
    else:
        c = x - x.mean(-1, keepdims=True) if norm == "layer" else x
        rstd = 1 / np.sqrt((c * c).mean(-1, keepdims=True) + EPS)
        e = 32 * U * (np.abs(n) + rstd * (np.abs(x) + np.abs(x).mean(-1, keepdims=True)))
    w = np.ones(x.shape[-1]) if weight is None else weight
    a, e = n * w, e * np.abs(w) + U * np.abs(n * w)
    want = oracle.qk_norm_rope(x, weight, norm, EPS, positions, freqs, axis, layout)
    p = len(freqs)
    if p:
        i, j = (np.arange(p), np.arange(p) + p) if layout == "halves" else (2 * np.arange(p), 2 * np.arange(p) + 1)
        both = e[..., i] + e[..., j] + 10 * U * (np.abs(a[..., i]) + np.abs(a[..., j]))
        e[..., i], e[..., j] = both, both
    return want, 2.0 ** -8 * (np.abs(want) + e) + e


def make(torch, M, hq, hkv, D, dtype, seed, extra=0):
    """q, k and v as slices of one projection output, rows `extra` elements longer than their heads."""
    g = torch.Generator().manual_seed(seed)
    width = (hq + 2 * hkv) * D
    full = torch.randn((M, width + extra), generator=g) * (1 + 6 * (torch.rand(width + extra, generator=g) < 0.03)) + 0.1
    full = full.to(dtype).cuda()
    cut = lambda a, n: full[:, a * D:(a + n) * D].unflatten(1, (n, D))  # noqa: E731
    return cut(0, hq), cut(hq, hkv), cut(hq + hkv, hkv), g


def tables(torch, g, pairs, axes, M, far):
    freqs = 10000.0 ** (-torch.rand(pairs, generator=g))
    axis = torch.randint(0, axes, (pairs,), generator=g, dtype=torch.int32)
    pos = torch.randint(-50, 5000, (axes, M), generator=g, dtype=torch.int32) + far
    return freqs.cuda(), axis.cuda(), pos.cuda()


def check(torch, M, hq, hkv, D, *, dtype="bf16", norm="rms", layout="halves", pairs=None, axes=3, far=0, weights=True,
          extra=0, rows_end=None, seed=0):
    t = torch.float32 if dtype == "f32" else torch.bfloat16
    pairs = D // 2 if pairs is None else pairs
    q, k, v, g = make(torch, M, hq, hkv, D, t, seed + 1000 * M + D, extra)
    wq, wk = ((1 + 0.3 * torch.randn(D, generator=g)).cuda() for _ in range(2)) if weights else (None, None)
    freqs, axis, pos = tables(torch, g, pairs, axes, M, far)
    rope = dict(freqs=freqs, pair_axis=axis, positions=pos) if pairs else {}
    outs = [torch.full((M, n, D), 7.0, dtype=torch.bfloat16, device="cuda") for n in (hq, hkv, hkv)]
    end = None if rows_end is None else torch.tensor([rows_end], dtype=torch.int32, device="cuda")
    ql.qlinear_qk_norm_rope(M, D, q=q, k=k, v=v, q_out=outs[0], k_out=outs[1], v_out=outs[2], norm=KIND[norm], eps=EPS,
                            q_weight=wq, k_weight=wk, rope=LAYOUT[layout], rows_end=end, **rope)
    live = M if rows_end is None else max(0, min(M, rows_end))
    for x, w, o in ((q, wq, outs[0]), (k, wk, outs[1])):
        want, tol = bound(num(x), None if w is None else num(w), norm, num(pos), num(freqs) if pairs else (), num(axis), layout)
        err = np.abs(num(o) - want)[:live]
        assert (err <= tol[:live]).all(), (err - tol[:live]).max()
    assert torch.equal(outs[2][:live], v[:live].to(torch.bfloat16))
    for o in outs:
        assert (o[live:] == 7.0).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("layout", ["halves", "pairs"])
@pytest.mark.parametrize("norm", ["none", "rms", "layer"])
@pytest.mark.parametrize("M,hq,hkv,D,pairs", [(1, 1, 1, 8, 4), (3, 5, 1, 32, 16), (7, 3, 3, 40, 12), (33, 4, 2, 64, 32),
                                              (5, 6, 2, 72, 20), (130, 2, 1, 128, 64), (9, 18, 18, 256, 128),
                                              (600, 3, 1, 136, 8), (17, 2, 2, 256, 0)])
def test_against_definition(torch, M, hq, hkv, D, pairs, norm, layout, dtype):
    check(torch, M, hq, hkv, D, dtype=dtype, norm=norm, layout=layout, pairs=pairs, weights=norm != "none")


@pytest.mark.parametrize("dtype,extra", [("f32", 1), ("bf16", 3), ("f32", 4), ("bf16", 8)])
@pytest.mark.parametrize("layout", ["halves", "pairs"])
def test_pitches(torch, layout, dtype, extra):
    check(torch, 41, 4, 2, 64, dtype=dtype, layout=layout, extra=extra)


@pytest.mark.parametrize("what", ["q", "q_out", "q_weight", "k_weight", "small"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("layout", ["halves", "pairs"])
def test_arrays_aligned_to_their_elements_only(torch, layout, dtype, what):
    """One array one element behind an aligned address gives the same bits; tables and positions may always be such."""
    M, D = 21, 72
    q, k, v, g = make(torch, M, 3, 2, D, torch.float32 if dtype == "f32" else torch.bfloat16, 13)
    freqs, axis, pos = tables(torch, g, 20, 2, M, 0)
    w = {n: (1 + 0.3 * torch.randn(D, generator=g)).cuda() for n in ("q_weight", "k_weight")}

    def behind(t):
        moved = torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")[1:].view(t.shape)
        return moved.copy_(t)

    def call(q, q_out, freqs, axis, pos, weights):
        outs = [torch.empty((M, n, D), dtype=torch.bfloat16, device="cuda") for n in (2, 2)]
        ql.qlinear_qk_norm_rope(M, D, q=q, k=k, v=v, q_out=q_out, k_out=outs[0], v_out=outs[1], norm=KIND["rms"],
                                rope=LAYOUT[layout], freqs=freqs, pair_axis=axis, positions=pos, **weights)
        return [q_out] + outs

    out = lambda: torch.zeros((M, 3, D), dtype=torch.bfloat16, device="cuda")  # noqa: E731
    want = call(q, out(), freqs, axis, pos, w)
    small = behind if what == "small" else lambda t: t  # noqa: E731
    got = call(behind(q) if what == "q" else q, behind(out()) if what == "q_out" else out(), small(freqs), small(axis),
               small(pos), {n: behind(t) if what == n else t for n, t in w.items()})
    for a, b in zip(got, want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("far", [1 << 20, 16000000, -16000000])
def test_far_positions(torch, far):
    check(torch, 33, 2, 1, 128, dtype="f32", far=far)


@pytest.mark.parametrize("rows_end", [-5, 0, 1, 200, 257, 10000])
def test_rows_behind_the_last_sample_stay(torch, rows_end):
    check(torch, 257, 3, 1, 64, rows_end=rows_end)


def test_parts_and_unweighted(torch):
    M, D = 12, 64
    q, k, v, g = make(torch, M, 4, 2, D, torch.bfloat16, 3)
    freqs, axis, pos = tables(torch, g, 32, 1, M, 0)
    whole = [torch.empty((M, n, D), dtype=torch.bfloat16, device="cuda") for n in (4, 2, 2)]
    kw = dict(norm=KIND["rms"], freqs=freqs, positions=pos[0])
    ql.qlinear_qk_norm_rope(M, D, q=q, k=k, v=v, q_out=whole[0], k_out=whole[1], v_out=whole[2], **kw)
    parts = [torch.empty_like(t) for t in whole]
    ql.qlinear_qk_norm_rope(M, D, q=q, q_out=parts[0], **kw)
    ql.qlinear_qk_norm_rope(M, D, k=k, k_out=parts[1], **kw)
    ql.qlinear_qk_norm_rope(M, D, v=v, v_out=parts[2])
    for a, b in zip(whole, parts):
        assert torch.equal(a, b)
    want, tol = bound(num(q), None, "rms", num(pos), num(freqs), None, "halves")
    assert (np.abs(num(whole[0]) - want) <= tol).all()


@pytest.mark.parametrize("layout", ["halves", "pairs"])
@pytest.mark.parametrize("D", [64, 256])
def test_in_place_and_strided_outputs(torch, layout, D):
    M = 77
    q, k, v, g = make(torch, M, 4, 2, D, torch.bfloat16, 5)
    freqs, axis, pos = tables(torch, g, D // 2, 2, M, 0)
    kw = dict(norm=KIND["rms"], rope=LAYOUT[layout], freqs=freqs, pair_axis=axis, positions=pos)
    apart = [torch.empty((M, n, D), dtype=torch.bfloat16, device="cuda") for n in (4, 2, 2)]
    ql.qlinear_qk_norm_rope(M, D, q=q, k=k, v=v, q_out=apart[0], k_out=apart[1], v_out=apart[2], **kw)
    packed = torch.full((M, 9, D), 3.0, dtype=torch.bfloat16, device="cuda")
    ql.qlinear_qk_norm_rope(M, D, q=q, k=k, v=v, q_out=packed[:, :4], k_out=packed[:, 4:6], v_out=packed[:, 6:8], **kw)
    ql.qlinear_qk_norm_rope(M, D, q=q, k=k, v=v, q_out=q, k_out=k, v_out=v, **kw)
    for a, b, c in zip(apart, (packed[:, :4], packed[:, 4:6], packed[:, 6:8]), (q, k, v)):
        assert torch.equal(a, b) and torch.equal(a, c)
    assert (packed[:, 8] == 3.0).all()


def test_axes_outside_are_not_turned(torch):
    M, D = 5, 32
    q, _, _, g = make(torch, M, 2, 1, D, torch.float32, 7)
    freqs, _, pos = tables(torch, g, 16, 2, M, 0)
    axis = torch.tensor([0, 1, 2, -1, 2147483647, -2147483648, 0, 1] * 2, dtype=torch.int32, device="cuda")
    out = torch.empty((M, 2, D), dtype=torch.bfloat16, device="cuda")
    ql.qlinear_qk_norm_rope(M, D, q=q, q_out=out, freqs=freqs, pair_axis=axis, positions=pos)
    want, tol = bound(num(q), None, "none", num(pos), num(freqs), num(axis).astype(int), "halves")
    assert (np.abs(num(out) - want) <= tol).all()


@pytest.mark.parametrize("norm", ["rms", "layer"])
def test_extremes_stay_in_their_head(torch, norm):
    """Heads of huge, tiny, zero, constant, infinite and NaN values among ordinary ones of the same wave."""
    M, H, D = 4, 8, 64
    g = torch.Generator().manual_seed(11)
    x = torch.randn((M, H, D), generator=g)
    x[0, 0] *= 1e30
    x[0, 1] *= 1e-30
    x[0, 2] = 0.0
    x[0, 3] = 5.0
    x[1, 0, 3] = float("inf")
    x[1, 1, 5] = float("nan")
    x[1, 2] *= 3e37
    out = torch.empty((M, H, D), dtype=torch.bfloat16, device="cuda")
    ql.qlinear_qk_norm_rope(M, D, q=x.cuda(), q_out=out, norm=KIND[norm], eps=1e-6)
    got = num(out)
    with np.errstate(all="ignore"):
        want, tol = bound(num(x), None, norm, None, (), None, "halves")
    odd = np.zeros((M, H), dtype=bool)
    odd[1, :2] = True
    assert np.isfinite(got[~odd]).all()
    assert (np.abs(got - want) <= tol)[~odd].all()
    assert np.isnan(got[1, 0, 3]) and np.isnan(got[1, 1]).all()


def test_streams_device_and_graph(torch):
    """On another stream than the tensors' own, and replayed with other positions and another end."""
    M, D = 65, 128
    q, k, v, g = make(torch, M, 4, 2, D, torch.float32, 9)
    freqs, axis, pos = tables(torch, g, 64, 3, M, 0)
    end = torch.tensor([M], dtype=torch.int32, device="cuda")
    outs = [torch.zeros((M, n, D), dtype=torch.bfloat16, device="cuda") for n in (4, 2, 2)]
    weight = torch.ones(D, device="cuda")

    def call(o, stream=None):
        ql.qlinear_qk_norm_rope(M, D, q=q, k=k, v=v, q_out=o[0], k_out=o[1], v_out=o[2], norm=KIND["rms"], q_weight=weight,
                                k_weight=weight, freqs=freqs, pair_axis=axis, positions=pos, rows_end=end, stream=stream)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        call(outs)
    for i, rows in enumerate((M, 10, 0, M)):
        pos.add_(i)
        end.fill_(rows)
        eager = [torch.zeros_like(o) for o in outs]
        torch.cuda.synchronize()
        call(eager, side)
        side.synchronize()
        for o in outs:
            o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(outs, eager):
            assert torch.equal(a, b)
    assert outs[0].abs().sum() > 0


def test_no_rows(torch):
    """An empty batch is nothing to do, with weights, tables and tensors of their own or slices of longer ones."""
    D = 64
    weight, freqs = torch.ones(D, device="cuda"), torch.ones(D // 2, device="cuda")
    full = torch.zeros((3, 8, D), dtype=torch.bfloat16, device="cuda")
    for x in (full[:0], torch.empty((0, 8, D), dtype=torch.bfloat16, device="cuda")):
        outs = [torch.empty((0, n, D), dtype=torch.bfloat16, device="cuda") for n in (4, 2, 2)]
        ql.qlinear_qk_norm_rope(0, D, q=x[:, :4], k=x[:, 4:6], v=x[:, 6:], q_out=outs[0], k_out=outs[1], v_out=outs[2],
                                norm=KIND["rms"], q_weight=weight, k_weight=weight, freqs=freqs,
                                positions=torch.empty((3, 0), dtype=torch.int32, device="cuda"))


def test_most_rows(torch):
    """2^24 - 1 rows of one small head: the largest grid. Values are turned by whole and half turns, which change at most
    the sign; the angle of pi is off by less than 2^-22, the sine with it, and the values are at most 3."""
    M, D = (1 << 24) - 1, 8
    g = torch.Generator(device="cuda").manual_seed(5)
    q = torch.randint(-3, 4, (M, 1, D), generator=g, device="cuda").to(torch.bfloat16)
    out = torch.empty_like(q)
    positions = torch.arange(M, device="cuda", dtype=torch.int32) % 4
    freqs = torch.full((D // 2,), np.pi, dtype=torch.float32, device="cuda")
    ql.qlinear_qk_norm_rope(M, D, q=q, q_out=out, freqs=freqs, positions=positions)
    want = torch.where((positions % 2 == 1)[:, None, None], -q, q).float()
    assert ((out.float() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -18).all()


def test_rows_past_4_gib(torch):
    """Rows whose byte offsets pass 32 bits, in inputs and outputs, give what the same rows give side by side."""
    M, D, pitch = 2100, 64, 1 << 20  # 4.4 GB each
    g = torch.Generator(device="cuda").manual_seed(7)
    x = torch.randn((M, 4, D), generator=g, device="cuda").to(torch.bfloat16)
    far, far_out = (torch.zeros((M, pitch), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    far[:, 3 * D:7 * D].copy_(x.view(M, 4 * D))
    freqs = torch.rand(D // 2, generator=g, device="cuda")
    kw = dict(norm=KIND["rms"], freqs=freqs, positions=torch.arange(M, device="cuda", dtype=torch.int32))
    part = lambda t, n: t[:, n * D:(n + 1) * D].unflatten(1, (1, D))  # noqa: E731
    outs = [torch.empty((M, 1, D), dtype=torch.bfloat16, device="cuda") for _ in range(3)]
    ql.qlinear_qk_norm_rope(M, D, q=x[:, :1], k=x[:, 1:2], v=x[:, 2:3], q_out=outs[0], k_out=outs[1], v_out=outs[2], **kw)
    ql.qlinear_qk_norm_rope(M, D, q=part(far, 3), k=part(far, 4), v=part(far, 5), q_out=part(far_out, 0),
                            k_out=part(far_out, 1), v_out=part(far_out, 2), **kw)
    assert torch.equal(far_out[:, :3 * D], torch.cat(outs, dim=1).view(M, 3 * D))
    assert not far_out[:, 3 * D:].any()
