"""GPU tests of qlinear_block_norm against its definition in 64 bits.

Tolerance, elementwise, from the arithmetic. u = 2^-24 is fp32's rounding (at
most half a step). A row's sums are taken by lanes of at most 64 values, then
over 64 lanes and at most 16 waves, one rounding each: a sum of S terms is off
by at most (64 + 6 + 16) u of the sum of magnitudes, below 96 u with the
products' own roundings. So the mean is off by 96 u * mean|v|, the variance by
96 u of itself beside the centring's share, and N(v) by at most

  e_N = 128 u (|n| + rstd * (|v| + mean|v|))

(reciprocal square root: a few u). An error e of the input of a norm reaches
its output as rstd * (e + mean e) + |n| * rstd * rms(e). Every further
multiplication or addition adds one u of what it yields. Each output is
rounded once more: half a step of its type (fp32 2^-24, bf16 2^-8, relative).
"""
import numpy as np
import pytest

import oracle
from group_wise_affine_qlinear_amd import qlinear as ql

from gpu_helpers import torch_or_skip

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF_STEP = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}
KIND = {"none": ql.QL_NORM_NONE, "rms": ql.QL_NORM_RMS, "layer": ql.QL_NORM_LAYER}


@pytest.fixture(scope="module")
def torch():
    t = torch_or_skip()
    ql.load_library()
    return t


def dtype(torch, name):
    return torch.float32 if name == "f32" else torch.bfloat16


def norm_and_bound(v, e, kind, eps):
    """N(v) in 64 bits and the bound of its fp32 error, v itself being off by at most e."""
    n = oracle.norm_rows(v, kind, eps)
    if kind == "none":
        return n, e
    c = v - v.mean(axis=1, keepdims=True) if kind == "layer" else v
    rstd = 1.0 / np.sqrt((c * c).mean(axis=1, keepdims=True) + np.float64(np.float32(eps)))
    own = 128 * U * (np.abs(n) + rstd * (np.abs(v) + np.abs(v).mean(axis=1, keepdims=True)))
    rms_e = np.sqrt((e * e).mean(axis=1, keepdims=True))
    return n, own + rstd * (e + e.mean(axis=1, keepdims=True)) + np.abs(n) * rstd * rms_e


def reference(p):
    """r, h in 64 bits with the bounds of their fp32 errors (before the outputs' own rounding)."""
    f = {k: None if p.get(k) is None else np.asarray(p[k], dtype=np.float64) for k in
         ("residual", "y", "post_weight", "post_bias", "pre_weight", "pre_bias", "gate", "scale", "shift")}
    r = f["residual"] * np.float64(np.float32(p["residual_scale"]))
    e = 2 * U * np.abs(r)
    one = lambda t, other: np.float64(other) if t is None else t  # noqa: E731
    if f["y"] is not None:
        n, en = norm_and_bound(f["y"], np.zeros_like(f["y"]), p["post"], p["post_eps"])
        gate, bias = one(f["gate"], 1.0), one(f["post_bias"], 0.0)
        mul, add = one(f["post_weight"], 1.0) * gate, bias * gate
        z = n * mul + add
        r = r + z
        e = e + np.abs(mul) * en + U * (2 * np.abs(n * mul) + np.abs(add) + np.abs(z) + np.abs(r))
    n, en = norm_and_bound(r, e, p["pre"], p["pre_eps"])
    scale, bias, shift = 1.0 + one(f["scale"], 0.0), one(f["pre_bias"], 0.0), one(f["shift"], 0.0)
    mul, add = one(f["pre_weight"], 1.0) * scale, bias * scale + shift
    h = n * mul + add
    eh = np.abs(mul) * en + U * (3 * np.abs(n * mul) + np.abs(bias * scale) + np.abs(add) + np.abs(h))
    want_r, want_h = oracle.block_norm(
        p["residual"], p.get("y"), residual_scale=p["residual_scale"], post=p["post"], post_eps=p["post_eps"],
        post_weight=f["post_weight"], post_bias=f["post_bias"], gate=f["gate"], pre=p["pre"], pre_eps=p["pre_eps"],
        pre_weight=f["pre_weight"], pre_bias=f["pre_bias"], scale=f["scale"], shift=f["shift"])
    assert np.allclose(r, want_r, rtol=1e-12, atol=1e-12) and np.allclose(h, want_h, rtol=1e-12, atol=1e-12)
    return r, e, h, eh


def close(got, want, err, out):
    got = np.asarray(got.double().cpu().numpy())
    assert np.all(np.isfinite(got))
    # the output's rounding is relative to the fp32 value, itself within err of `want`
    bound = err + HALF_STEP[out] * (np.abs(want) + err) + 1e-37
    worst = np.max(np.abs(got - want) / bound)
    assert worst <= 1.0, worst


class Problem:
    """Inputs on the device and their values in 64 bits."""

    def __init__(self, torch, M, D, parts, post="rms", pre="rms", y="bf16", residual="bf16", affine=True, samples=2,
                 seed=0, residual_scale=1.0, eps=1e-6, amplitude=1.0, mean=0.25):
        g = torch.Generator().manual_seed(1000 * M + D + seed)
        rand = lambda *s: torch.randn(s, generator=g)  # noqa: E731
        self.torch, self.M, self.D, self.parts = torch, M, D, parts
        self.before, self.after = parts != "after", parts != "before"
        self.types = {"y": y, "residual": residual}
        t = {"residual": ((rand(M, D) + mean) * 3 * amplitude).to(dtype(torch, residual))}
        if self.after:
            t["y"] = ((rand(M, D) - mean) * amplitude).to(dtype(torch, y))
        self.samples = samples
        self.mod_rows = -(-M // samples)
        if affine:
            if self.after:
                t["post_weight"], t["post_bias"] = 1 + 0.2 * rand(D), 0.3 * rand(D)
            if self.before:
                t["pre_weight"], t["pre_bias"] = 1 + 0.2 * rand(D), 0.3 * rand(D)
        mod = {}
        if self.after:
            mod["gate"] = torch.tanh(rand(samples, D))
        if self.before:
            mod["scale"], mod["shift"] = 0.3 * rand(samples, D), 0.2 * rand(samples, D)
        self.host, self.mod_host = t, mod
        self.dev = {k: v.cuda() for k, v in t.items()}
        self.mod = {k: v.cuda() for k, v in mod.items()}
        self.kw = dict(residual_scale=residual_scale)
        if self.after:
            self.kw.update(post_norm=KIND[post], post_eps=eps)
        if self.before:
            self.kw.update(pre_norm=KIND[pre], pre_eps=eps)
        sample = np.arange(M) // self.mod_rows
        self.values = {k: v.double().numpy() for k, v in t.items()}
        self.values.update({k: v.double().numpy()[sample] for k, v in mod.items()})
        self.values.update(residual_scale=residual_scale, post=post if self.after else "none", post_eps=eps,
                           pre=pre if self.before else "none", pre_eps=eps)

    def outputs(self):
        torch = self.torch
        out = {}
        if self.after:
            out["residual_out"] = torch.full((self.M, self.D), 77.0, dtype=dtype(torch, self.types["residual"]), device="cuda")
        if self.before:
            out["h"] = torch.full((self.M, self.D), 77.0, dtype=torch.bfloat16, device="cuda")
        return out

    def call(self, out=None, **more):
        out = self.outputs() if out is None else out
        kw = dict(self.kw, mod_rows=self.mod_rows, **{k: v for k, v in self.dev.items() if k != "residual"}, **self.mod)
        kw.update(out)
        kw.update(more)
        residual = kw.pop("residual", self.dev["residual"])
        ql.qlinear_block_norm(residual, self.M, self.D, **kw)
        return out

    def check(self, out):
        r, er, h, eh = reference(self.values)
        if "residual_out" in out:
            close(out["residual_out"], r, er, self.types["residual"])
        if "h" in out:
            close(out["h"], h, eh, "bf16")
        return r, er, h, eh


SHAPES = [(1, 1), (3, 7), (2, 8), (5, 64), (1, 65), (4, 512), (9, 520), (2, 1003), (6, 1152), (3, 2048), (2, 4100),
          (5, 4608), (1, 4608), (2, 8200), (3, 12288), (2, 16392), (1, 30001), (2, 40000), (2, 53248), (1, 65535),
          (1, 65536), (300, 128), (260, 1000)]


@pytest.mark.parametrize("parts", ["before", "after", "between"])
@pytest.mark.parametrize("M,D", SHAPES)
def test_every_length(torch, M, D, parts):
    """Row lengths from one value to the longest, whole and odd; both norms, all stream types over the lengths."""
    i = SHAPES.index((M, D))
    kinds = [("rms", "rms"), ("layer", "layer"), ("rms", "layer"), ("layer", "rms")][i % 4]
    types = [("bf16", "bf16"), ("f32", "bf16"), ("bf16", "f32"), ("f32", "f32")][(i // 2) % 4]
    p = Problem(torch, M, D, parts, post=kinds[0], pre=kinds[1], y=types[0], residual=types[1], affine=i % 3 != 0,
                samples=min(M, 1 + i % 3), residual_scale=1.0 if i % 2 else 0.5)
    p.check(p.call())


@pytest.mark.parametrize("y", ["f32", "bf16"])
@pytest.mark.parametrize("residual", ["f32", "bf16"])
@pytest.mark.parametrize("post", ["none", "rms", "layer"])
@pytest.mark.parametrize("pre", ["none", "rms", "layer"])
@pytest.mark.parametrize("D", [72, 77])
def test_every_norm_and_type(torch, y, residual, post, pre, D):
    p = Problem(torch, 11, D, "between", post=post, pre=pre, y=y, residual=residual, samples=3, residual_scale=0.75)
    p.check(p.call())


@pytest.mark.parametrize("D", [520, 515])
def test_every_part_may_be_left_out(torch, D):
    full = Problem(torch, 7, D, "between", post="layer", pre="rms", samples=2)
    for gone in ("post_weight", "post_bias", "gate", "pre_weight", "pre_bias", "scale", "shift"):
        v = full.values.pop(gone)
        full.check(full.call(**{gone: None}))
        full.values[gone] = v
    # the plain gated update, and a plain copy to bf16 with the modulation alone
    p = Problem(torch, 5, D, "after", post="none", affine=False)
    p.check(p.call())
    p = Problem(torch, 5, D, "before", pre="none", affine=False, residual="f32")
    p.check(p.call())


@pytest.mark.parametrize("D", [512, 500, 4608])
def test_slices_of_one_modulation_output(torch, D):
    """gate, scale and shift as column ranges of one [samples, 6 D] tensor, aligned to 16 bytes or not."""
    for off in (0, 1, 4):
        p = Problem(torch, 9, D, "between", samples=3, seed=off)
        wide = torch.full((3, 6 * D + 8), float("nan"), device="cuda")
        views = {}
        for i, (k, v) in enumerate(p.mod.items()):
            views[k] = wide[:, off + 2 * i * D:off + (2 * i + 1) * D]
            views[k].copy_(v)
        plain = p.call()
        sliced = p.call(**views)
        p.check(sliced)
        for k in plain:
            # 16-byte and element-wise access sum a row in another order: bit-equal only within one of them
            if D % 8 == 0 and off % 4 == 0:
                assert torch.equal(plain[k], sliced[k]), (k, off)


@pytest.mark.parametrize("D,shift", [(512, 1), (4608, 1), (64, 3)])
def test_unaligned_streams(torch, D, shift):
    """Streams that start one element into a buffer take the element-wise path."""
    p = Problem(torch, 4, D, "between", y="f32", residual="f32")

    def moved(t):
        flat = torch.empty(t.numel() + shift, dtype=t.dtype, device="cuda")
        view = flat[shift:].view(t.shape)
        view.copy_(t)
        return view

    out = {k: moved(v) for k, v in p.outputs().items()}
    p.check(p.call(out, y=moved(p.dev["y"]), residual=moved(p.dev["residual"]), gate=moved(p.mod["gate"])))


@pytest.mark.parametrize("parts", ["before", "after", "between"])
@pytest.mark.parametrize("D", [128, 131])
def test_rows_outside_every_sample_stay(torch, parts, D):
    """Ragged samples in any order; rows of no sample are neither read into others nor written."""
    M, S = 37, 4
    p = Problem(torch, M, D, parts, samples=S)
    idx = torch.tensor([3, 3, 0, -1, 2] + [1] * 9 + [4, 5, -7, 2 ** 31 - 1, -2 ** 31] + [2] * 10 + [0] * 3 + [-1] * 5,
                       dtype=torch.int32)
    assert len(idx) == M
    live = ((idx >= 0) & (idx < S)).numpy()
    for k in ("y", "residual"):
        if k in p.dev:
            p.dev[k][~torch.from_numpy(live).cuda()] = float("nan")
            p.host[k] = p.dev[k].cpu()
    out = p.call(row_sample=idx.cuda())
    sample = np.where(live, idx.numpy(), 0)
    values = dict(p.values)
    for k in ("residual", "y"):
        if k in p.host:
            values[k] = p.host[k].double().numpy()[live]
    for k, v in p.mod_host.items():
        values[k] = v.double().numpy()[sample][live]
    r, er, h, eh = reference(values)
    rows = torch.from_numpy(live).cuda()
    for name, want, err, kind in (("residual_out", r, er, p.types["residual"]), ("h", h, eh, "bf16")):
        if name in out:
            close(out[name][rows], want, err, kind)
            assert bool((out[name][~rows] == 77.0).all()), name
    # all rows outside
    out = p.call(row_sample=torch.full((M,), -1, dtype=torch.int32, device="cuda"))
    assert all(bool((v == 77.0).all()) for v in out.values())


def test_row_sample_without_modulation(torch):
    p = Problem(torch, 6, 64, "before", affine=False)
    p.values.update(scale=None, shift=None)
    idx = torch.tensor([0, 1, 2, 0, 1, 2], dtype=torch.int32, device="cuda")
    out = p.call(scale=None, shift=None, row_sample=idx, samples=3)
    p.check(out)
    with pytest.raises(ValueError):
        p.call(scale=None, shift=None, row_sample=idx)


@pytest.mark.parametrize("residual", ["f32", "bf16"])
@pytest.mark.parametrize("D", [4608, 333])
def test_update_in_place(torch, residual, D):
    p = Problem(torch, 6, D, "between", residual=residual)
    apart = p.call()
    stream = p.dev["residual"].clone()
    out = dict(p.outputs(), residual_out=stream)
    p.call(out, residual=stream)
    assert torch.equal(stream, apart["residual_out"]) and torch.equal(out["h"], apart["h"])


@pytest.mark.parametrize("D", [4608, 1000, 777, 40000])
def test_one_pass_is_the_two_calls(torch, D):
    """With an fp32 stream nothing is rounded in between: the pass between two blocks gives the bits of the
    norm after followed by the norm before."""
    p = Problem(torch, 8, D, "between", residual="f32", y="f32", post="layer", pre="rms")
    both = p.call()
    mid = torch.empty_like(p.dev["residual"])
    kw = {k: p.dev[k] for k in ("y", "post_weight", "post_bias")}
    ql.qlinear_block_norm(p.dev["residual"], 8, D, residual_out=mid, post_norm=ql.QL_NORM_LAYER, gate=p.mod["gate"],
                          mod_rows=p.mod_rows, **kw)
    assert torch.equal(mid, both["residual_out"])
    h = torch.empty_like(both["h"])
    ql.qlinear_block_norm(mid, 8, D, h=h, pre_norm=ql.QL_NORM_RMS, pre_weight=p.dev["pre_weight"],
                          pre_bias=p.dev["pre_bias"], scale=p.mod["scale"], shift=p.mod["shift"], mod_rows=p.mod_rows)
    assert torch.equal(h, both["h"])


@pytest.mark.parametrize("D", [4608, 515, 12288])
def test_a_row_does_not_depend_on_the_others(torch, D):
    p = Problem(torch, 13, D, "between", samples=1)
    whole = p.call()
    for m in (0, 6, 12):
        one = {k: torch.empty((1, D), dtype=v.dtype, device="cuda") for k, v in whole.items()}
        kw = {k: v for k, v in p.dev.items() if k not in ("residual", "y")}
        ql.qlinear_block_norm(p.dev["residual"][m:m + 1], 1, D, y=p.dev["y"][m:m + 1], **kw, **p.mod, **p.kw, **one)
        for k in whole:
            assert torch.equal(one[k][0], whole[k][m]), (k, m)


@pytest.mark.parametrize("D", [64, 4608, 1001])
def test_fast_activations_of_the_same_pass(torch, D):
    """x16 * rowscale is the unrounded h to fp16's half step: |x16 * 2^e - h| <= 2^-11 |h| above the smallest
    normal of the row's scale, 2^-25 * 2^e below it, beside h's own fp32 bound."""
    p = Problem(torch, 9, D, "between")
    x16 = torch.zeros((9, D), dtype=torch.float16, device="cuda")
    rowscale = torch.zeros(9, device="cuda")
    out = p.call(x16=x16, rowscale=rowscale)
    _, _, h, eh = p.check(out)
    scale = rowscale.double().cpu().numpy()[:, None]
    got = x16.double().cpu().numpy() * scale
    assert np.all(np.abs(got - h) <= eh + np.maximum(HALF_STEP["f16"] * (np.abs(h) + eh), 2.0 ** -25 * scale))
    top = np.abs(x16.double().cpu().numpy()).max(axis=1)
    assert np.all((top >= 2.0 ** 14) & (top <= 2.0 ** 15))
    # without the bf16 h the same bits
    again, rs = torch.zeros_like(x16), torch.zeros_like(rowscale)
    ql_out = {"residual_out": torch.empty_like(out["residual_out"])}
    p.call(ql_out, x16=again, rowscale=rs)
    assert torch.equal(again, x16) and torch.equal(rs, rowscale)


def test_fast_activations_match_the_prepass(torch):
    """A modulation alone (no norm): the bits of qlinear_fast_activations_adaln."""
    M, D = 6, 4608
    g = torch.Generator().manual_seed(3)
    x = torch.randn((M, D), generator=g).to(torch.bfloat16).cuda()
    x[2] = 0
    scale = (0.3 * torch.randn((2, D), generator=g)).cuda()
    want, want_rs = ql.qlinear_fast_activations_adaln(x, scale, 3, M, D)
    x16, rs = torch.empty_like(want), torch.empty_like(want_rs)
    ql.qlinear_block_norm(x, M, D, scale=scale, mod_rows=3, x16=x16, rowscale=rs)
    assert torch.equal(x16, want) and torch.equal(rs, want_rs)


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("D", [64, 777, 4608])
def test_extremes(torch, kind, D):
    """Rows of zeros and of one value, and rows whose squares pass fp32 in either direction."""
    rows = [np.zeros(D), np.full(D, 3.0), np.full(D, 2.0 ** 127)]
    g = np.random.default_rng(D)
    base = g.standard_normal(D)
    base /= np.abs(base).max()
    for p in (2.0 ** 126, 1e30, 1e19, 1e-3, 1e-18, 1e-30, 2.0 ** -140):
        rows.append(base * p)
    v = torch.from_numpy(np.stack(rows)).to(torch.float32)
    M = len(rows)
    for eps in (1e-6, 1e-30):
        h = torch.full((M, D), float("nan"), dtype=torch.bfloat16, device="cuda")
        ql.qlinear_block_norm(v.cuda(), M, D, pre_norm=KIND[kind], pre_eps=eps, h=h)
        x = v.double().numpy()
        n, e = norm_and_bound(x, np.zeros_like(x), kind, eps)
        # Among subnormal numbers fp32 rounds to multiples of 2^-149, not relative to the value: sums and
        # differences of such numbers are exact, but the mean, the sum times 1 / D, is off by half a step
        # beside the factor's own u, below 2^-149 in all. Every centred value is off by as much, times rstd in
        # the output. The squares of such rows vanish beside eps >= 1e-30. A subnormal output is within
        # 2^-126 of anything of its size.
        c = x - x.mean(axis=1, keepdims=True) if kind == "layer" else x
        rstd = 1.0 / np.sqrt((c * c).mean(axis=1, keepdims=True) + np.float64(np.float32(eps)))
        close(h, n, e + 2.0 ** -126 + 2.0 ** -149 * rstd, "bf16")


@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_infinities_and_nan_stay_in_their_row(torch, kind):
    for bad in (float("inf"), float("-inf"), float("nan")):
        p = Problem(torch, 6, 520, "between", post=kind, pre=kind)
        clean = p.call()
        p.dev["y"][2, 100] = bad
        out = p.call()
        rows = torch.tensor([0, 1, 3, 4, 5], device="cuda")
        for k in clean:
            assert torch.equal(out[k][rows], clean[k][rows])
            assert not bool(torch.isfinite(out[k][2]).all())


def test_layer_norm_of_a_far_mean(torch):
    """The mean is removed before squaring: a mean of 1000 standard deviations cancels nothing but its rounding."""
    p = Problem(torch, 4, 4608, "before", pre="layer", residual="f32", mean=1000.0)
    p.check(p.call())


def test_graph_replays(torch):
    p = Problem(torch, 33, 4608, "between")
    idx = torch.arange(33, dtype=torch.int32, device="cuda") % 2
    want = p.call(row_sample=idx)
    out = p.outputs()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        p.call(out, row_sample=idx)
    for i in range(4):
        for v in out.values():
            v.fill_(5.0)
        torch.cuda.synchronize()
        graph.replay()
        eager = p.call(row_sample=idx)
        torch.cuda.synchronize()
        for k in want:
            assert torch.equal(out[k], want[k]) and torch.equal(eager[k], want[k]), (i, k)


def test_two_streams(torch):
    probs = [Problem(torch, 700, 4608, "between", seed=s) for s in (1, 2)]
    want = [p.call() for p in probs]
    streams = [torch.cuda.Stream() for _ in probs]
    outs = [p.outputs() for p in probs]
    torch.cuda.synchronize()
    for _ in range(3):
        for p, s, o in zip(probs, streams, outs):
            p.call(o, stream=s)
    torch.cuda.synchronize()
    for w, o in zip(want, outs):
        assert all(torch.equal(w[k], o[k]) for k in w)


def test_refused_tensors(torch):
    p = Problem(torch, 4, 64, "between")
    wrong = [
        dict(y=p.dev["y"][:, :32]), dict(y=p.dev["y"].double()), dict(y=p.dev["y"].cpu()),
        dict(y=torch.empty((64, 4), dtype=torch.bfloat16, device="cuda").T),
        dict(gate=p.mod["gate"][:1]), dict(gate=p.mod["gate"][:, :63]), dict(gate=p.mod["gate"].to(torch.bfloat16)),
        dict(gate=p.mod["gate"][:1].expand(2, 64)), dict(scale=torch.empty((64, 2), device="cuda").T),
        dict(scale=p.mod["scale"].cpu()), dict(post_weight=torch.ones(63, device="cuda")),
        dict(residual_out=torch.empty((4, 64), device="cuda")), dict(h=torch.empty((4, 64), device="cuda")),
        dict(row_sample=torch.zeros(3, dtype=torch.int32, device="cuda")),
        dict(row_sample=torch.zeros(4, dtype=torch.int64, device="cuda")),
        dict(row_sample=torch.zeros(4, dtype=torch.int32, device="cuda"), samples=3),
        dict(x16=torch.empty((4, 64), dtype=torch.float16, device="cuda")),
        dict(pre_eps=0.0), dict(post_norm=9),
    ]
    for kw in wrong:
        with pytest.raises((ValueError, TypeError, ql.QLinearError)):
            p.call(**kw)
    torch.cuda.synchronize()
