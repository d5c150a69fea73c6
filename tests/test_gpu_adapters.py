"""GPU tests of qlinear_adapters against its definition in 64 bits.

Tolerance, elementwise, from the arithmetic. u = 2^-24 is fp32's rounding.
v = A x: products of bf16 (or the two terms of fp16) are exact in fp32, K of
them are added in some order, so |dv| <= (2 K + 32) u * |A| |x| (2 K: fp16
tables enter as two terms). The second product takes v to 24 bits (u),
scaled (u), as three terms against one or two of B, added over the rank:
|dd| <= s |B| |dv| + (6 rank + 8) u * s |B| |v|. The base and each step of an
epilogue add one u of what they yield; silu's exponential and reciprocal are
good to a few u (8 are allowed, times 1 + |g| for the exponential's argument).
The output's own rounding is half a step (fp32 2^-24, bf16 2^-8, relative).
"""
import copy

import numpy as np
import pytest

import oracle
from group_wise_affine_qlinear_amd import qlinear as ql

from gpu_helpers import torch_or_skip

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF_STEP = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}
EPI = {"none": ql.QL_EPI_NONE, "swiglu": ql.QL_EPI_SWIGLU, "gate": ql.QL_EPI_GATE_RESIDUAL}


@pytest.fixture(scope="module")
def torch():
    t = torch_or_skip()
    ql.load_library()
    return t


def f64(t):
    return t.double().cpu().numpy()


class Problem:
    def __init__(self, torch, M, N, K, rank, adapters, ids="mixed", y="f32", out="f32", table="bf16", epilogue="none",
                 ranks=None, scaling=True, seed=0):
        g = torch.Generator().manual_seed(7919 * M + 31 * N + K + rank + seed)
        rand = lambda *s: torch.randn(s, generator=g)  # noqa: E731
        types = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
        self.torch, self.M, self.N, self.K, self.rank, self.n = torch, M, N, K, rank, adapters
        self.out_type, self.epilogue = out, epilogue
        self.x = rand(M, K).to(torch.bfloat16).cuda()
        self.a = (rand(adapters, rank, K) / max(K, 1) ** 0.5).to(types[table]).cuda()
        self.b = (rand(adapters, N, rank) / rank ** 0.5).to(types[table]).cuda()
        self.y = rand(M, N).to(types[y]).cuda() if y else None
        if isinstance(ids, str):
            if ids == "mixed":        # any order, some rows without an adapter, some indices outside the table
                ids = torch.randint(-1, adapters + 1, (M,), generator=g)
            elif ids == "sorted":     # runs, as requests in order
                ids = torch.sort(torch.randint(0, max(adapters, 1), (M,), generator=g)).values
            elif ids == "distinct":
                ids = torch.arange(M) % max(adapters, 1)
        self.ids = torch.as_tensor(ids).to(torch.int32).cuda()
        self.ranks = None if ranks is None else torch.as_tensor(ranks, dtype=torch.int32).cuda()
        self.scaling = (0.5 + torch.rand(adapters, generator=g)).cuda() if scaling else None
        self.width = N // 2 if epilogue == "swiglu" else N
        self.gate_rows = max(1, M // 3)
        if epilogue == "gate":
            self.residual = rand(M, N).to(types[out]).cuda()
            self.gate = torch.tanh(rand(-(-M // self.gate_rows), N)).cuda()
        self.dtype = types[out]

    def call(self, out=None, **more):
        if out is None:
            out = self.torch.full((self.M, self.width), float("nan"), dtype=self.dtype, device="cuda")
        kw = dict(y=self.y, ranks=self.ranks, scaling=self.scaling, epilogue=EPI[self.epilogue])
        if self.epilogue == "gate":
            kw.update(residual=self.residual, gate=self.gate, gate_rows=self.gate_rows)
        kw.update(more)
        x, ids = kw.pop("x", self.x), kw.pop("ids", self.ids)
        a, b = kw.pop("a", self.a), kw.pop("b", self.b)
        return ql.qlinear_adapters(x, a, b, ids, self.M, self.N, self.K, out, **kw)

    def reference(self):
        """t in 64 bits and the bound of its fp32 error."""
        x, a, b, ids = f64(self.x), f64(self.a), f64(self.b), self.ids.cpu().numpy()
        ranks = None if self.ranks is None else self.ranks.cpu().numpy()
        scaling = None if self.scaling is None else f64(self.scaling)
        d = oracle.adapter_delta(x, a, b, ids, ranks, scaling)
        e = np.zeros_like(d)
        for i in range(self.n):
            rows = np.flatnonzero(ids == i)
            r = self.rank if ranks is None else min(max(int(ranks[i]), 0), self.rank)
            if not len(rows) or r == 0:
                continue
            s = 1.0 if scaling is None else abs(scaling[i])
            ev = (2 * self.K + 32) * U * (np.abs(x[rows]) @ np.abs(a[i, :r]).T)
            v = np.abs(x[rows] @ a[i, :r].T)
            e[rows] = s * ((ev + (6 * r + 8) * U * v) @ np.abs(b[i, :, :r]).T)
        t = d if self.y is None else f64(self.y) + d
        return t, e + U * np.abs(t)

    def check(self, out):
        t, e = self.reference()
        if self.epilogue == "swiglu":
            F = self.width
            g, u, eg, eu = t[:, :F], t[:, F:], e[:, :F], e[:, F:]
            want = oracle.swiglu(t, F)
            s = np.abs(oracle.silu(g))
            # |silu'| <= 1.1
            e = 1.1 * eg * (np.abs(u) + eu) + (s + 1.1 * eg) * eu + 8 * U * (1 + np.abs(g)) * np.abs(want)
        elif self.epilogue == "gate":
            want = oracle.gate_residual(t, f64(self.residual), f64(self.gate), self.gate_rows)
            gate = np.abs(f64(self.gate))[np.arange(self.M) // self.gate_rows]
            e = gate * e + U * np.abs(want)
        else:
            want = t
        got = f64(out)
        assert got.shape == want.shape and np.all(np.isfinite(got))
        bound = e + HALF_STEP[self.out_type] * (np.abs(want) + e) + 1e-37
        worst = np.max(np.abs(got - want) / bound) if want.size else 0.0
        assert worst <= 1.0, worst
        if self.out_type == "f32" and want.size:
            # beside the worst case, the usual error of fp32 sums: the exact mode's design bar
            assert np.linalg.norm(got - want) <= 2e-5 * np.linalg.norm(want)


SIZES = [
    # M, N, K, rank, adapters
    (1, 64, 64, 8, 1), (1, 1, 64, 8, 1), (2, 3, 128, 16, 2), (1, 4608, 4608, 16, 3), (15, 100, 192, 24, 4),
    (16, 256, 320, 32, 20), (17, 257, 512, 40, 5), (63, 255, 64, 64, 7), (64, 512, 640, 72, 64), (65, 1003, 448, 128, 3),
    (130, 64, 1024, 256, 9), (255, 36, 2048, 16, 1), (256, 260, 128, 8, 40), (257, 300, 576, 16, 6), (300, 1001, 64, 48, 2),
    (321, 130, 4608, 136, 5), (640, 512, 832, 64, 11), (1000, 96, 256, 32, 3), (33, 8, 12288, 16, 2),
    # more than 1024 rows of few columns
    (1025, 64, 64, 8, 1), (1030, 260, 192, 64, 5), (1100, 67, 320, 136, 9), (1500, 128, 128, 16, 70), (1091, 512, 704, 24, 3),
    (2100, 36, 1024, 256, 2), (1200, 300, 2048, 48, 4), (1063, 1000, 320, 32, 12),
]


@pytest.mark.parametrize("ids", ["mixed", "sorted", "distinct"])
@pytest.mark.parametrize("M,N,K,rank,n", SIZES)
def test_sizes(torch, M, N, K, rank, n, ids):
    i = SIZES.index((M, N, K, rank, n))
    p = Problem(torch, M, N, K, rank, n, ids=ids, y=["f32", "bf16"][i % 2], out=["f32", "f32", "bf16"][i % 3],
                table=["bf16", "f16"][(i // 2) % 2], scaling=i % 4 != 3)
    p.check(p.call())


LARGE = [
    # 64-row tiles (more than 1024 rows, many columns), every rank class, whole and odd widths
    (1030, 16132, 128, 16, 3, "sorted", "none"), (1100, 15617, 192, 24, 2, "sorted", "none"),
    (1100, 15620, 320, 64, 3, "mixed", "gate"), (1090, 15700, 64, 136, 70, "mixed", "none"),
    (2048, 8200, 128, 256, 2, "sorted", "gate"), (1100, 16390, 64, 128, 4, "sorted", "swiglu"),
    (1031, 16404, 704, 8, 5, "mixed", "swiglu"), (1100, 15617, 64, 104, 2, "sorted", "none"),
    (1100, 15750, 64, 48, 2, "sorted", "swiglu"),
]


@pytest.mark.parametrize("table", ["bf16", "f16"])
@pytest.mark.parametrize("M,N,K,rank,n,ids,epilogue", LARGE)
def test_large_tiles(torch, M, N, K, rank, n, ids, epilogue, table):
    i = LARGE.index((M, N, K, rank, n, ids, epilogue))
    ranks = [max(1, rank - 3 * j) for j in range(n)] if i % 2 else None
    p = Problem(torch, M, N, K, rank, n, ids=ids, y=["f32", "bf16"][i % 2], out=["f32", "bf16", "bf16"][i % 3],
                table=table, epilogue=epilogue, ranks=ranks)
    out = p.call()
    assert "rows64" in ql.qlinear_last_path()
    p.check(out)
    if table == "bf16":
        # rows in another order: the same bits at their new places
        perm = torch.randperm(M, generator=torch.Generator().manual_seed(i)).cuda()
        if epilogue != "gate":
            again = p.call(x=p.x[perm].contiguous(), ids=p.ids[perm].contiguous(), y=p.y[perm].contiguous())
            assert torch.equal(again, out[perm])
        # what others hold
        mine = (p.ids >= 0) & (p.ids < n) & (p.ids != 1)
        q = {k: getattr(p, k).clone() for k in ("x", "a", "b", "y")}
        q["x"][~mine] = float("nan")
        q["a"][1] = float("inf")
        q["b"][1] = float("nan")
        assert torch.equal(p.call(**q)[mine], out[mine])


def test_large_tiles_in_a_graph(torch):
    """The largest LDS request (rank 256) and 64-row tiles, captured."""
    p = Problem(torch, 2048, 8200, 128, 256, 2, ids="sorted")
    want = p.call()
    out = torch.empty_like(want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        p.call(out)
    for _ in range(4):
        out.zero_()
        torch.cuda.synchronize()
        graph.replay()
        eager = p.call()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(eager, want)


def test_one_gate_row_for_all(torch):
    """gate_rows beyond M, also beyond 32 bits: one row of the gate."""
    p = Problem(torch, 40, 260, 128, 16, 3, epilogue="gate")
    p.gate = p.gate[:1].contiguous()
    p.gate_rows = 40
    want = p.call()
    p.check(want)
    for rows in (41, 2 ** 32, 2 ** 33 + 5, 2 ** 62):
        assert torch.equal(p.call(gate_rows=rows), want)


def test_gate_rows_of_every_size(torch):
    """Samples that begin anywhere among the 16 rows of a step."""
    for rows in (1, 3, 7, 15, 16, 17, 33):
        p = Problem(torch, 50, 132, 64, 8, 2, epilogue="gate", seed=rows)
        p.gate_rows = rows
        p.gate = torch.tanh(torch.randn(-(-50 // rows), 132, generator=torch.Generator().manual_seed(rows))).cuda()
        p.check(p.call())


@pytest.mark.parametrize("epilogue", ["none", "swiglu", "gate"])
@pytest.mark.parametrize("table", ["bf16", "f16"])
@pytest.mark.parametrize("y", ["f32", "bf16", None])
@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("M,N", [(21, 264), (300, 262), (9, 130), (1061, 264), (1030, 130)])
def test_types_and_epilogues(torch, epilogue, table, y, out, M, N):
    p = Problem(torch, M, N, 192, 40, 5, ids="mixed", y=y, out=out, table=table, epilogue=epilogue)
    p.check(p.call())


@pytest.mark.parametrize("M", [5, 40, 400, 1100])
def test_ranks_of_their_own(torch, M):
    """Odd ranks, a rank of zero, ranks below and beyond the table's (clamped); what the table holds past an
    adapter's rank does not matter."""
    ranks = [1, 7, 0, 40, 17, -3, 999, 33]
    for table in ("bf16", "f16"):
        p = Problem(torch, M, 130, 256, 40, len(ranks), ids="distinct", ranks=ranks, table=table)
        first = p.call()
        p.check(first)
        for i, r in enumerate(ranks):
            r = min(max(r, 0), 40)
            p.a[i, r:] = float("nan")
            p.b[i, :, r:] = float("inf")
        assert torch.equal(p.call(), first)


@pytest.mark.parametrize("M", [1, 16, 300, 1033])
def test_no_adapter_at_all(torch, M):
    for ids in (-1, 3, 2 ** 31 - 1, -2 ** 31):
        p = Problem(torch, M, 70, 64, 8, 3, ids=[ids] * M)
        assert torch.equal(p.call(), p.y)
        out = p.y.clone()
        p.y = out
        p.call(out)
        assert torch.equal(p.call(out), out)
    # without a base the product of no adapter is zero
    p = Problem(torch, M, 70, 64, 8, 3, ids=[-1] * M, y=None)
    assert bool((p.call() == 0).all())
    # an empty table
    p = Problem(torch, M, 70, 64, 8, 0, ids=[0] * M, epilogue="gate")
    p.check(p.call())


def test_k_of_zero(torch):
    p = Problem(torch, 20, 64, 0, 16, 2, ids="sorted")
    assert torch.equal(p.call(), p.y)


@pytest.mark.parametrize("M", [16, 37, 300, 1033])
def test_rows_without_an_adapter_stay_in_place(torch, M):
    p = Problem(torch, M, 200, 128, 16, 4, ids="mixed")
    ids = p.ids.cpu()
    none = ((ids < 0) | (ids >= 4)).cuda()
    apart = p.call()
    out = p.y.clone()
    out[none] = float("nan")      # neither read nor written
    marked = out.clone()
    p.call(out, y=out)
    assert torch.equal(out[~none], apart[~none])
    assert torch.equal(out[none].view(torch.int32), marked[none].view(torch.int32))


@pytest.mark.parametrize("epilogue", ["none", "gate"])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("M", [90, 1210])
def test_in_place(torch, epilogue, dt, M):
    p = Problem(torch, M, 260, 320, 24, 6, y=dt, out=dt, epilogue=epilogue)
    apart = p.call()
    out = p.y.clone()
    assert torch.equal(p.call(out, y=out), apart)
    if epilogue == "gate":
        stream = p.residual.clone()
        assert torch.equal(p.call(stream, residual=stream), apart)


@pytest.mark.parametrize("M", [14, 200, 300, 1100])
def test_what_others_hold_never_reaches_a_row(torch, M):
    """NaN and infinities in the rows of one request, in its adapter's tables, and in rows without an adapter."""
    p = Problem(torch, M, 132, 320, 24, 5, ids="mixed")
    clean = p.call()
    ids = p.ids
    mine = (ids >= 0) & (ids < 5) & (ids != 2)
    for bad in (float("nan"), float("inf")):
        q = {k: getattr(p, k).clone() for k in ("x", "a", "b", "y")}
        q["x"][~mine] = bad
        q["a"][2] = bad
        q["b"][2] = bad
        q["y"][~mine] = bad
        out = p.call(**q)
        assert torch.equal(out[mine], clean[mine])
        other = (ids == 2)
        if bool(other.any()):
            assert not bool(torch.isfinite(out[other]).any())


@pytest.mark.parametrize("M", [16, 150, 320, 1090])
def test_a_row_does_not_depend_on_its_place(torch, M):
    """The same rows in another order give the same bits, each at its new place."""
    p = Problem(torch, M, 260, 960, 40, 6, ids="mixed")
    first = p.call()
    for seed in (0, 1):
        perm = torch.randperm(M, generator=torch.Generator().manual_seed(seed)).cuda()
        again = p.call(x=p.x[perm].contiguous(), ids=p.ids[perm].contiguous(), y=p.y[perm].contiguous())
        assert torch.equal(again, first[perm])


@pytest.mark.parametrize("N", [256, 257, 260])
def test_unaligned_outputs(torch, N):
    p = Problem(torch, 40, N, 128, 16, 3)
    want = p.call()
    for shift in (1, 2, 4):
        flat = torch.full((40 * N + 8,), 9.0, device="cuda")
        out = flat[shift:shift + 40 * N].view(40, N)
        assert torch.equal(p.call(out), want)
        assert bool((flat[:shift] == 9.0).all()) and bool((flat[shift + 40 * N:] == 9.0).all())


def test_large_table_offsets(torch):
    """An adapter whose table entries lie past 2^31 elements."""
    K, rank, n = 12288, 64, 2800     # 2.2e9 elements of a
    a = torch.empty((n, rank, K), dtype=torch.bfloat16, device="cuda")
    p = Problem(torch, 6, 64, K, rank, 2, ids=[0, 1, 0, 1, 1, 0])
    b = torch.empty((n, 64, rank), dtype=torch.bfloat16, device="cuda")
    for i, j in ((0, 0), (1, n - 1)):
        a[j], b[j] = p.a[i], p.b[i]
    scaling = torch.ones(n, device="cuda")
    scaling[0], scaling[n - 1] = p.scaling[0], p.scaling[1]
    ids = torch.where(p.ids == 1, n - 1, 0).to(torch.int32)
    out = torch.empty((6, 64), device="cuda")
    ql.qlinear_adapters(p.x, a, b, ids, 6, 64, K, out, y=p.y, scaling=scaling)
    p.check(out)


def test_large_output_offsets(torch):
    """Rows whose outputs lie past 2^31 elements of out: one adapter's rows at both ends."""
    M, N, K = 90000, 24000, 64
    x = torch.zeros((M, K), dtype=torch.bfloat16, device="cuda")
    ids = torch.full((M,), -1, dtype=torch.int32, device="cuda")
    p = Problem(torch, 40, N, K, 8, 1, ids=[0] * 40, y=None)
    x[:20], x[-20:] = p.x[:20], p.x[20:]
    ids[:20], ids[-20:] = 0, 0
    out = torch.zeros((M, N), dtype=torch.float32, device="cuda")
    ql.qlinear_adapters(x, p.a, p.b, ids, M, N, K, out, y=out, scaling=p.scaling)
    p.check(torch.cat([out[:20], out[-20:]]))
    assert float(out[20:-20].abs().max()) == 0.0


def test_graph_serves_other_requests(torch):
    """Captured once; replays follow the adapter of each row, the ranks and the inputs as they are at the replay."""
    ps = [Problem(torch, 48, 260, 640, 24, 6, ids="mixed", seed=s, ranks=[24, 5, 24, 1, 0, 9]) for s in range(3)]
    live = ps[0]
    want = [p.call() for p in ps]
    cur = {k: getattr(live, k).clone() for k in ("x", "a", "b", "ids", "y", "scaling", "ranks")}
    out = torch.empty_like(want[0])
    ws = torch.empty(ql.qlinear_adapters_workspace_bytes(48, 260, 640, 24, 6), dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        live.call(out, workspace=ws, **cur)
    for i in (0, 1, 2, 1, 0):
        for k, t in cur.items():
            t.copy_(getattr(ps[i], k))
        out.fill_(3.0)
        ws.fill_(255)
        torch.cuda.synchronize()
        graph.replay()
        eager = ps[i].call()
        torch.cuda.synchronize()
        assert torch.equal(out, want[i]) and torch.equal(eager, want[i]), i


def test_two_graphs_share_a_workspace(torch):
    """Replayed one after the other on one stream, two graphs may use one workspace."""
    ps = [Problem(torch, 70, 300, 512, 32, 4, seed=1), Problem(torch, 20, 900, 1024, 16, 9, seed=2)]
    want = [p.call() for p in ps]
    ws = torch.empty(max(ql.qlinear_adapters_workspace_bytes(p.M, p.N, p.K, p.rank, p.n) for p in ps), dtype=torch.uint8,
                     device="cuda")
    outs, graphs = [torch.empty_like(w) for w in want], []
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for p, o in zip(ps, outs):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1], stream=side):
            p.call(o, workspace=ws)
    for _ in range(4):
        for o in outs:
            o.zero_()
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o, w) for o, w in zip(outs, want))


def test_two_streams(torch):
    ps = [Problem(torch, 1500, 1024, 1024, 32, 4, seed=s) for s in (1, 2)]
    want = [p.call() for p in ps]
    streams = [torch.cuda.Stream() for _ in ps]
    outs = [torch.empty_like(w) for w in want]
    torch.cuda.synchronize()
    for _ in range(3):
        for p, s, o in zip(ps, streams, outs):
            p.call(o, stream=s)
            p.call(o, stream=s.cuda_stream)
    torch.cuda.synchronize()
    ps[0].call(outs[0], stream=0)
    torch.cuda.synchronize()
    assert all(torch.equal(o, w) for o, w in zip(outs, want))


def test_refused_tensors(torch):
    p = Problem(torch, 6, 64, 128, 16, 2)
    wrong = [
        dict(x=p.x[:, :64]), dict(x=p.x.float()), dict(x=p.x.cpu()), dict(a=p.a[0]), dict(a=p.a.float()),
        dict(a=p.a[:, :12].contiguous(), b=p.b[:, :, :12].contiguous()), dict(b=p.b.half()), dict(b=p.b[:1]),
        dict(b=p.b.transpose(1, 2).contiguous().transpose(1, 2)), dict(ids=p.ids.long()), dict(ids=p.ids[:5]),
        dict(scaling=p.scaling[:1]), dict(scaling=p.scaling.double()), dict(ranks=p.ids), dict(y=p.y.half()),
        dict(y=p.y[:, :32]), dict(workspace=None), dict(workspace=torch.empty(16, dtype=torch.uint8, device="cuda")),
        dict(workspace="other"), dict(epilogue=ql.QL_EPI_SWIGLU), dict(epilogue=ql.QL_EPI_GATE_RESIDUAL),
        dict(epilogue=7),
    ]
    for kw in wrong:
        with pytest.raises((ValueError, TypeError, ql.QLinearError)):
            p.call(**kw)
    torch.cuda.synchronize()


@pytest.mark.parametrize("table", ["bf16", "f16"])
@pytest.mark.parametrize("M,N,rank,epilogue,out", [
    (5, 64, 8, "none", "f32"), (40, 67, 40, "none", "bf16"), (40, 132, 72, "gate", "f32"), (41, 131, 48, "gate", "bf16"),
    (33, 130, 8, "swiglu", "f32"), (34, 264, 48, "swiglu", "f32"), (300, 260, 136, "none", "bf16"),
    (1100, 16384, 8, "gate", "bf16"), (1100, 16385, 104, "none", "f32"), (1100, 16392, 72, "swiglu", "f32")])
def test_infinities_give_what_the_definition_gives(torch, table, M, N, rank, epilogue, out):
    """Infinities and NaN in x, A and B of the row's own adapter: an infinity where the definition's sums are
    infinite, NaN where they are none. All finite values are small integers, so that every product and sum is exact
    and has zeros in its lower bits, where a value that is split into terms has zero terms."""
    K, ranks = 64, [1, 1, 2, rank, 1, 3]
    n = len(ranks)
    g = torch.Generator().manual_seed(M + N + rank)
    whole = lambda lo, hi, *s: torch.randint(lo, hi + 1, s, generator=g).float()  # noqa: E731
    p = Problem(torch, M, N, K, rank, n, ids="mixed", out=out, epilogue=epilogue, ranks=ranks, table=table)
    nonzero = lambda t: torch.where(t == 0, torch.ones_like(t), t)  # noqa: E731
    x, a, b = whole(-3, 3, M, K), nonzero(whole(-2, 2, n, rank, K)), whole(-2, 2, n, N, rank)
    a[2, 0, 5] = 0.0
    inf, nan = float("inf"), float("nan")
    x[0::5, 5], x[1::5, 9], x[1::10, 40] = inf, -inf, inf
    x[3::20, 7] = nan
    a[3, rank - 1, 2], a[4, 0, 1], a[4, 0, 60] = -inf, inf, inf
    b[1, 0::3, 0], b[1, 1::6, 0], b[5, ::4, 1], b[0, ::7, 0] = inf, -inf, inf, nan
    p.x, p.a, p.b = x.to(torch.bfloat16).cuda(), a.to(p.a.dtype).cuda(), b.to(p.b.dtype).cuda()
    p.y = whole(-3, 3, M, N).cuda()
    p.scaling = torch.tensor([1.0, 2.0, 0.5, 1.0, -1.0, 4.0]).cuda()
    if epilogue == "gate":
        p.residual, p.gate = whole(-3, 3, M, N).to(p.dtype).cuda(), nonzero(whole(-2, 2, p.gate.shape[0], N)).cuda()
    got = f64(p.call())
    x, a, b, s, ids = f64(p.x), f64(p.a), f64(p.b), f64(p.scaling), p.ids.cpu().numpy()
    cols = np.r_[0:min(N, 400), max(0, N - 400):N] if epilogue == "none" else np.arange(N)
    with np.errstate(invalid="ignore", over="ignore"):
        t = f64(p.y)[:, cols]
        for m in np.flatnonzero((ids >= 0) & (ids < n)):
            i = ids[m]
            v = (a[i, :ranks[i]] * x[m]).sum(axis=1)
            t[m] = t[m] + s[i] * (b[i][cols, :ranks[i]] * v).sum(axis=1)
        if epilogue == "gate":
            want = f64(p.residual) + f64(p.gate)[np.arange(M) // p.gate_rows] * t
        elif epilogue == "swiglu":
            F = N // 2
            want = t[:, :F] / (1.0 + np.exp(-t[:, :F])) * t[:, F:]
        else:
            got, want = got[:, cols], t
        # the five rows of the smallest case do not meet every adapter
        assert M < 30 or (np.isposinf(want).any() and np.isneginf(want).any() and np.isnan(want).any())
        if epilogue == "swiglu":
            # silu of a finite value is rounded: the last digits of what is finite, and tiny ones, may differ
            odd = ~np.isfinite(want)
            assert np.array_equal(got[odd], want[odd], equal_nan=True)
            assert np.allclose(got[~odd], want[~odd], rtol=1e-4, atol=1e-30)
        else:
            want = f64(torch.from_numpy(want).float().to(p.dtype))  # exact in fp32, rounded once
            assert np.array_equal(got, want, equal_nan=True)


# Widths that end in an odd number of 256-column pieces, the last of them short of two waves' columns.
PIECES = [("none", 15944), ("none", 15943), ("gate", 15944), ("gate", 15943), ("swiglu", 16528), ("swiglu", 16526)]


@pytest.mark.parametrize("rank", [16, 64, 104, 136])
@pytest.mark.parametrize("epilogue,N", PIECES)
def test_blocks_of_two_pieces(torch, epilogue, N, rank):
    """Enough blocks that each takes two 256-column pieces (2048 blocks of one): every epilogue and rank class, rows
    of whole fours and by elements. Checked at the first columns, at those around the pieces' ends, and at the last."""
    M, i = 2100, PIECES.index((epilogue, N)) + [16, 64, 104, 136].index(rank)
    assert -(-M // 64) * -(-N // 256) >= 2048
    y, out = [("f32", "f32"), ("bf16", "bf16"), ("f32", "bf16"), ("bf16", "f32")][i % 4 if rank != 104 else i % 2]
    n = 4
    p = Problem(torch, M, N, 128, rank, n, ids=["mixed", "sorted"][i // 2 % 2], y=y, out=out, table=["bf16", "f16"][i // 3 % 2],
                epilogue=epilogue, ranks=[rank, max(1, rank - 5), 1, rank])
    got = p.call()
    assert "rows64" in ql.qlinear_last_path()
    assert bool(torch.isfinite(got).all())
    w = p.width
    ends = [c for e in range(256, w, 256 * 7) for c in range(e - 5, e + 5)]
    cols = torch.tensor(sorted(set(list(range(0, 200)) + ends + list(range(256 * (w // 256 - 1) - 8, w)))))
    part = copy.copy(p)
    both = torch.cat([cols, w + cols]) if epilogue == "swiglu" else cols
    part.N, part.width = len(both), len(cols)
    part.b, part.y = p.b[:, both.cuda()], p.y[:, both.cuda()]
    if epilogue == "gate":
        part.residual, part.gate = p.residual[:, cols.cuda()], p.gate[:, cols.cuda()]
    part.check(got[:, cols.cuda()])


@pytest.mark.parametrize("table", ["bf16", "f16"])
@pytest.mark.parametrize("M,N,rank", [(3, 64, 8), (30, 67, 40), (300, 132, 72), (1100, 16000, 16), (1100, 16001, 104)])
def test_every_bit_of_the_first_product_counts(torch, table, M, N, rank):
    """Whole numbers whose A x needs up to 24 bits, and tables B that pick one or two of them: every product and
    sum is exact, so that out has the very bits; a second product that took A x to 16 bits would be off by 2^-9
    of what it dropped."""
    K, n = 128, 3
    g = torch.Generator().manual_seed(N + rank)
    p = Problem(torch, M, N, K, rank, n, ids="mixed", y=None, table=table)
    x = torch.randint(128, 256, (M, K), generator=g).float()
    a = torch.randint(128, 256, (n, rank, K), generator=g).float() * torch.where(
        torch.rand((n, rank, 1), generator=g) < 0.5, -1.0, 1.0)
    b = torch.zeros((n, N, rank))
    pick = torch.randint(0, rank, (n, N, 1), generator=g)
    b.scatter_(2, pick, 1.0)
    b.scatter_(2, (pick + 1) % rank, -1.0 * (torch.rand((n, N, 1), generator=g) < 0.5))
    p.x, p.a, p.b = x.to(torch.bfloat16).cuda(), a.to(p.a.dtype).cuda(), b.to(p.b.dtype).cuda()
    p.scaling = torch.tensor([1.0, -2.0, 0.5]).cuda()
    got = f64(p.call())
    ids = p.ids.cpu().numpy()
    want = np.zeros((M, N))
    for i in range(n):
        rows = np.flatnonzero(ids == i)
        if not len(rows):
            continue
        v = x.double().numpy()[rows] @ a[i].double().numpy().T
        # exact in fp32, and beyond the 16 bits of two terms
        assert np.abs(v).max() < 2 ** 23 and (v % 256 != 0).any()
        want[rows] = float(p.scaling[i]) * (v @ b[i].double().numpy().T)
    assert np.array_equal(got, want)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("M,N,epilogue", [(90, 260, "none"), (90, 259, "gate"), (1210, 16000, "gate"), (1210, 16001, "none")])
def test_infinities_in_place_and_in_a_graph(torch, M, N, epilogue, dt):
    """Steps with infinite sums are stored last, from inputs that the call may be about to overwrite, by arguments that
    the kernel reads a second time."""
    p = Problem(torch, M, N, 128, 24, 6, y=dt, out=dt, epilogue=epilogue, ranks=[1, 24, 1, 7, 24, 2])
    p.x[::7, 3] = float("inf")
    p.b[2, ::5, 0] = float("-inf")
    p.a[4, 2, 9] = float("nan")
    bits = torch.int32 if dt == "f32" else torch.int16

    def same(got, want):  # NaN at the same places, the same bits elsewhere
        nan = torch.isnan(want)
        return torch.equal(torch.isnan(got), nan) and torch.equal(got.view(bits)[~nan], want.view(bits)[~nan])

    apart = p.call()
    assert bool(torch.isinf(apart).any()) and bool(torch.isnan(apart).any())
    out = p.y.clone()
    assert same(p.call(out, y=out), apart)
    if epilogue == "gate":
        stream = p.residual.clone()
        assert same(p.call(stream, residual=stream), apart)
    out = torch.empty_like(apart)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        p.call(out)
    for _ in range(4):
        out.zero_()
        torch.cuda.synchronize()
        graph.replay()
        eager = p.call()
        torch.cuda.synchronize()
        assert same(out, apart) and same(eager, apart)
