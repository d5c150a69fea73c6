"""GPU tests of qlinear_block_norm where a block has several rows, and of wide
and odd rows in every use, against the definition in 64 bits with the bounds
that test_gpu_block_norm derives.

A block of 16-byte rows up to 8192 values takes as many consecutive rows as
leave each CU its share of waves: of 4608 values 3 before a block from 1537
rows on, 3 after it from 1025, 4 between two from 769; of 128 values, where a
wave has rows of its own, 3 from 16385, 10241 and 8193. Such a block keeps the
factors of a sample over its rows, reads the next row while it works on one,
and goes past rows of no sample.
"""
import numpy as np
import pytest

from group_wise_affine_qlinear_amd import qlinear as ql

from gpu_helpers import torch_or_skip
from test_gpu_block_norm import HALF_STEP, KIND, Problem, close, norm_and_bound, reference

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    t = torch_or_skip()
    ql.load_library()
    return t


# rows, row length, rows of a block before, after and between
ROWS = [(1600, 4608, (3, 4, 7)), (1100, 4600, (2, 3, 5)), (17001, 128, (3, 4, 5)), (9001, 1000, (3, 4, 5))]
PARTS = ["before", "after", "between"]


def rows_of_a_block(M, D, parts):
    """The rule on sizes that the library follows (256 CUs)."""
    waves = {"before": 32, "after": 20, "between": 16}[parts]
    W = -(-D // 512)
    per_block = 4 if W == 1 else 1
    return -(-M // (256 * max(1, waves // (W * per_block)) * per_block))


@pytest.mark.parametrize("parts", PARTS)
@pytest.mark.parametrize("M,D,rows", ROWS)
def test_samples_that_change_inside_a_block(torch, M, D, rows, parts):
    i = ROWS.index((M, D, rows)) + PARTS.index(parts)
    assert rows_of_a_block(M, D, parts) == rows[PARTS.index(parts)] >= 2
    types = [("bf16", "bf16"), ("f32", "bf16"), ("bf16", "f32"), ("f32", "f32")][i % 4]
    # samples of 5 rows: of 2 to 7 rows of a block, a sample ends in almost every one
    p = Problem(torch, M, D, parts, post=["rms", "layer"][i % 2], pre=["layer", "rms"][i // 2 % 2], y=types[0],
                residual=types[1], affine=i % 3 != 0, samples=-(-M // 5), residual_scale=0.5)
    assert p.mod_rows == 5
    p.check(p.call())


@pytest.mark.parametrize("parts", PARTS)
@pytest.mark.parametrize("M,D,rows", ROWS)
def test_rows_of_no_sample_inside_a_block(torch, M, D, rows, parts):
    """Runs of rows that are left alone among live ones, at the ends of the batch too, with the stream updated in place."""
    S = 7
    p = Problem(torch, M, D, parts, samples=S, post="layer", pre="rms")
    g = torch.Generator().manual_seed(M + D)
    runs = torch.randint(1, 6, (M,), generator=g)
    which = torch.randint(-2, S + 1, (M,), generator=g)
    which[::3] = -1
    idx = torch.repeat_interleave(which, runs)[:M].to(torch.int32)
    idx[-1] = 2 ** 31 - 1
    live = ((idx >= 0) & (idx < S)).numpy()
    assert 0.2 * M < live.sum() < 0.8 * M
    dead = ~torch.from_numpy(live)
    for k in ("y", "residual"):
        if k in p.dev:
            p.host[k][dead] = float("nan")
            p.dev[k].copy_(p.host[k])
    out, kw = p.outputs(), {}
    if p.after:
        kw["residual"] = out["residual_out"] = p.dev["residual"].clone()
    p.call(out, row_sample=idx.cuda(), **kw)
    values = dict(p.values)
    for k in ("residual", "y"):
        if k in p.host:
            values[k] = p.host[k][~dead].double().numpy()
    for k, v in p.mod_host.items():
        values[k] = v.double().numpy()[idx.numpy()[live]]
    r, er, h, eh = reference(values)
    if p.after:
        close(out["residual_out"][~dead.cuda()], r, er, p.types["residual"])
        left = out["residual_out"][dead.cuda()]
        assert bool(torch.isnan(left).all())  # what the stream held there
    if p.before:
        close(out["h"][~dead.cuda()], h, eh, "bf16")
        assert bool((out["h"][dead.cuda()] == 77.0).all())


@pytest.mark.parametrize("M,D,rows", ROWS)
def test_in_place_is_apart(torch, M, D, rows):
    p = Problem(torch, M, D, "between", samples=-(-M // 5))
    apart = p.call()
    stream = p.dev["residual"].clone()
    out = dict(p.outputs(), residual_out=stream)
    p.call(out, residual=stream)
    assert torch.equal(stream, apart["residual_out"]) and torch.equal(out["h"], apart["h"])


@pytest.mark.parametrize("parts", ["before", "between"])
@pytest.mark.parametrize("M,D", [(1600, 4608), (17001, 128), (5, 1001), (3, 12288), (2, 20001), (2, 40000)])
def test_fast_activations(torch, M, D, parts):
    """x16 and rowscale of rows in one chunk and several, whole and odd, with and without an update: the bound of
    test_fast_activations_of_the_same_pass; the same bits without the bf16 h."""
    p = Problem(torch, M, D, parts, pre="layer", residual=["bf16", "f32"][D % 3 == 0])
    x16 = torch.zeros((M, D), dtype=torch.float16, device="cuda")
    rowscale = torch.zeros(M, device="cuda")
    out = p.call(x16=x16, rowscale=rowscale)
    _, _, h, eh = p.check(out)
    scale = rowscale.double().cpu().numpy()[:, None]
    got = x16.double().cpu().numpy()
    assert np.all(np.abs(got * scale - h) <= eh + np.maximum(HALF_STEP["f16"] * (np.abs(h) + eh), 2.0 ** -25 * scale))
    top = np.abs(got).max(axis=1)
    assert np.all((top >= 2.0 ** 14) & (top <= 2.0 ** 15))
    again, rs = torch.zeros_like(x16), torch.zeros_like(rowscale)
    alone = {k: torch.empty_like(v) for k, v in out.items() if k == "residual_out"}
    p.call(alone, x16=again, rowscale=rs)
    assert torch.equal(again, x16) and torch.equal(rs, rowscale)


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("residual", ["f32", "bf16"])
@pytest.mark.parametrize("D", [12288, 20001, 40000])
def test_extremes_of_wide_rows(torch, kind, residual, D):
    """Rows of zeros and of one value, and rows whose squares pass fp32 in either direction, several chunks to a
    lane; the bound of test_extremes."""
    g = np.random.default_rng(D)
    base = g.standard_normal(D)
    base /= np.abs(base).max()
    rows = [np.zeros(D), np.full(D, 3.0), np.full(D, 2.0 ** 127)]
    rows += [base * s for s in (2.0 ** 126, 1e30, 1e19, 1e-3, 1e-18, 1e-30, 2.0 ** -140)]
    v = torch.from_numpy(np.stack(rows)).to(torch.float32 if residual == "f32" else torch.bfloat16)
    M = len(rows)
    for eps in (1e-6, 1e-30):
        h = torch.full((M, D), float("nan"), dtype=torch.bfloat16, device="cuda")
        ql.qlinear_block_norm(v.cuda(), M, D, pre_norm=KIND[kind], pre_eps=eps, h=h)
        x = v.double().numpy()
        n, e = norm_and_bound(x, np.zeros_like(x), kind, eps)
        c = x - x.mean(axis=1, keepdims=True) if kind == "layer" else x
        rstd = 1.0 / np.sqrt((c * c).mean(axis=1, keepdims=True) + np.float64(np.float32(eps)))
        close(h, n, e + 2.0 ** -126 + 2.0 ** -149 * rstd, "bf16")


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("M,D", [(4, 12288), (4, 20001), (3, 40000), (1100, 4608)])
def test_infinities_and_nan_stay_in_their_row(torch, kind, M, D):
    for parts, where in (("between", "y"), ("before", "residual")):
        p = Problem(torch, M, D, parts, post=kind, pre=kind)
        clean = p.call()
        keep = torch.arange(M, device="cuda") != 2
        for bad in (float("inf"), float("-inf"), float("nan")):
            p.dev[where][2, D // 3] = bad
            out = p.call()
            for k in clean:
                assert torch.equal(out[k][keep], clean[k][keep])
                assert not bool(torch.isfinite(out[k][2]).all())
