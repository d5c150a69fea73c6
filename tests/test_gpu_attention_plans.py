"""GPU tests of qlinear_attention where it divides its work in every way: whole tiles in front of cut ones, kernels of
256 rows of every width, masked and not, over many stages of keys, cut and not; and where offsets that are read on the
device change, or break, the division.

Tolerance: that of test_gpu_attention.py, with the mean deviation sum p |v - out| / sum p of the values bounded by the
root of their variance, sqrt(sum p v^2 / sum p - out^2) (Jensen), which two products give for many rows. All of it is
computed in 64 bits on the device.
"""
import numpy as np
import pytest

from group_wise_affine_qlinear_amd import qlinear as ql

from gpu_helpers import torch_or_skip

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.fixture(scope="module")
def torch():
    t = torch_or_skip()
    ql.load_library()
    return t


def edges(lengths, first=0):
    return [int(i) for i in np.cumsum([first] + list(lengths))]


def make(torch, nq, nk, hq, hkv, D, seed, spread=2.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    q = (rand(nq, hq, D) * spread).to(torch.bfloat16)
    k = (rand(nk, hkv, D) + 0.5 * rand(1, hkv, D)).to(torch.bfloat16)
    v = (rand(nk, hkv, D) + 0.5 * rand(1, hkv, D)).to(torch.bfloat16)
    return q, k, v


def compare(torch, out, before, q, k, v, scale, q_at, k_at, mask):
    """Every row of `out` against the definition; rows of no sample against `before`."""
    group = q.shape[1] // k.shape[1]
    D = q.shape[2]
    live = torch.zeros(q.shape[0], dtype=torch.bool, device="cuda")
    for q0, q1, k0, k1 in zip(q_at[:-1], q_at[1:], k_at[:-1], k_at[1:]):
        live[q0:q1] = True
        if q1 == q0:
            continue
        keys = torch.arange(k0, k1, device="cuda")
        if mask is not None:
            keys = keys[mask[k0:k1]]
        n = len(keys)
        if n == 0:
            assert (out[q0:q1] == 0).all()
            continue
        for h in range(q.shape[1]):
            kk, vv = k[keys, h // group].double(), v[keys, h // group].double()
            kt, ka = kk.T.contiguous(), kk.abs().T.contiguous()
            for a in range(q0, q1, 4096):
                b = min(a + 4096, q1)
                x = q[a:b, h].double()
                s = torch.mm(x, kt).mul_(scale)
                size = scale * torch.mm(x.abs(), ka).amax(dim=1, keepdim=True)
                p = s.sub_(s.amax(dim=1, keepdim=True)).exp_()
                p /= p.sum(dim=1, keepdim=True)
                want = torch.mm(p, vv)
                spread = (torch.mm(p, vv * vv) - want * want).clamp(min=0).sqrt()
                d = 2.0 ** -8 + 2 * ((D + 16) * U * size + 4 * U)
                e = d / (1 - d) * spread + (n + n / 32 + 16) * U * torch.mm(p, vv.abs())
                err = (out[a:b, h].double() - want).abs()
                assert (err <= e + 2.0 ** -8 * (want.abs() + e)).all(), (q0, h, a, (err - e).max().item(), err.max().item())
    assert torch.equal(out[~live], before[~live])


def check(torch, q, k, v, q_len=None, k_len=None, mask=None, scale=None, workspace=ql.TORCH_WORKSPACE, path=None, out=None):
    """Runs the call twice, the second time into `out`, and compares it. Samples begin behind two rows and one key."""
    inputs = q.clone(), k, v
    out = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device="cuda") if out is None else out
    before = out.clone()
    kw, at = {}, ([0, q.shape[0]], [0, k.shape[0]])
    if q_len is not None:
        at = edges(q_len, 2), edges(k_len, 1)
        kw = {"q_offsets": torch.tensor(at[0], dtype=torch.int32, device="cuda"),
              "k_offsets": torch.tensor(at[1], dtype=torch.int32, device="cuda")}
    scale = q.shape[2] ** -0.5 if scale is None else scale
    first = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
    for o in (first, out):
        ql.qlinear_attention(q, k, v, o, scale=scale, key_mask=mask, workspace=workspace, **kw)
        if path is not None:
            assert ql.qlinear_last_path() == "attention_" + path
    live = slice(at[0][0], at[0][-1])
    assert torch.equal(first[live], out[live])
    compare(torch, out, before, *inputs, scale, *at, mask)
    return out


def hide(torch, k, v, seed, q_len=None, k_len=None):
    """A mask with runs longer than a stage, short holes and, of several samples, one without any key; what is hidden is
    not finite."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    n = k.shape[0]
    mask = torch.rand(n, generator=g, device="cuda") < 0.8
    mask[n // 3:n // 3 + 200] = False
    mask[:70] = False
    mask[-90:-30] = False
    if k_len is not None:
        at = edges(k_len, 1)
        mask[at[1]:at[2]] = False
    k[~mask], v[~mask] = float("nan"), float("inf")
    return mask


# queries, keys, query heads, key heads, D, with a workspace, path. One sample: whole tiles, and behind them tiles that
# are cut, that go 32 rows to a block, or that are not cut.
ONE = [
    (33000, 1100, 2, 2, 128, True, "rows128_slots512"),        # 512 whole, 4 cut
    (8237, 1100, 8, 2, 88, True, "rows128_slots512"),          # shared key heads, odd width: 516 tiles
    (33000, 700, 2, 2, 40, True, "rows128_slots512"),
    (8300, 2200, 8, 8, 256, True, "rows256_slots256"),         # 256 whole, 8 cut
    (8300, 2200, 8, 8, 256, False, "rows256_slots0"),
    (8300, 700, 8, 8, 256, True, "rows256_slots0_rest32"),     # 256 whole, 8 of 32 rows to a block over several stages
    (8300, 700, 8, 8, 192, True, "rows256_slots256"),
    (8300, 700, 8, 8, 184, False, "rows256_slots0"),
    (4000, 9000, 4, 4, 248, True, "rows256_slots256"),         # all cut
    (2100, 9000, 4, 2, 144, True, "rows256_slots256"),
    (32850, 4100, 4, 1, 64, True, "rows256_slots512"),         # 512 whole, 2 cut
    (32850, 4100, 4, 1, 64, False, "rows256_slots0"),
    (33024, 4100, 1, 1, 56, True, "rows256_slots512"),         # all cut
]


@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("nq,nk,hq,hkv,D,workspace,path", ONE)
def test_one_sample(torch, nq, nk, hq, hkv, D, workspace, path, masked):
    q, k, v = make(torch, nq, nk, hq, hkv, D, nq + D)
    mask = hide(torch, k, v, D) if masked else None
    check(torch, q, k, v, mask=mask, workspace=ql.TORCH_WORKSPACE if workspace else None, path=path)


# queries and keys of each sample, heads, D, rows of a tile, tiles that are whole (of as many as there are)
SEVERAL = [
    ([33000], [1100], 2, 2, 128, 128, 512),                    # one sample between offsets
    ([20000, 1, 0, 13200], [700, 900, 5, 1900], 2, 2, 128, 128, 512),
    ([9, 4200, 4099], [600, 1500, 1900], 8, 8, 256, 256, 256),
    ([9, 4200, 4099], [600, 1500, 1900], 8, 8, 192, 256, 256),
    ([16000, 17, 500, 16400], [3100, 5000, 4400, 5000], 4, 1, 64, 256, 512),
    ([130] * 70, [1400 - 9 * i for i in range(70)], 4, 4, 72, 128, 512),    # more samples than a wave has lanes
    ([300] * 9 + [40], [2000] * 10, 2, 2, 256, 128, 0),        # 56 tiles, all cut
]


@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("q_len,k_len,hq,hkv,D,rows,whole", SEVERAL)
def test_several_samples(torch, q_len, k_len, hq, hkv, D, rows, whole, masked):
    q, k, v = make(torch, sum(q_len) + 5, sum(k_len) + 4, hq, hkv, D, len(q_len) + D)
    mask = hide(torch, k, v, D, q_len, k_len) if masked and len(k_len) > 1 else hide(torch, k, v, D) if masked else None
    slots = 256 if D > 128 else 512
    tiles = sum(-(-n * (hq // hkv) // rows) for n in q_len) * hkv
    assert tiles // slots * slots == whole and tiles % slots > 0  # some are cut
    for workspace, cut in ((ql.TORCH_WORKSPACE, slots), (None, 0)):
        check(torch, q, k, v, q_len, k_len, mask, workspace=workspace, path=f"rows{rows}_slots{cut}")


@pytest.mark.parametrize("nq,nk,hq,hkv,D,path", [(33000, 1100, 2, 2, 128, "rows128_slots512"),
                                                 (8300, 2200, 8, 8, 256, "rows256_slots256"),
                                                 (8300, 700, 8, 8, 192, "rows256_slots256"),
                                                 (32850, 4100, 4, 1, 64, "rows256_slots512"),
                                                 (8300, 700, 8, 8, 256, "rows256_slots0_rest32")])
def test_scores_that_grow_along_the_keys(torch, nq, nk, hq, hkv, D, path):
    """The maximum is followed again and again, by each query at keys of its own; the same from the last key on."""
    q, k, v = make(torch, nq, nk, hq, hkv, D, 17)
    ramp = torch.linspace(-4, 4, nk, device="cuda")[:, None, None]
    k = (k.float() * 0.3 + ramp * q[:1, ::hq // hkv].float() * 0.2).to(torch.bfloat16)
    check(torch, q, k, v, path=path)
    check(torch, q, k.flip(0).contiguous(), v, path=path, scale=0.1)


@pytest.mark.parametrize("nq,nk,hq,D,path", [(8300, 2200, 8, 256, "rows256_slots256"), (8300, 700, 8, 192, "rows256_slots256"),
                                             (33024, 4100, 1, 64, "rows256_slots512"), (33000, 1100, 2, 128, "rows128_slots512")])
def test_values_that_are_not_finite_stay_with_their_query(torch, nq, nk, hq, D, path):
    q, k, v = make(torch, nq, nk, hq, hq, D, 23)
    clean = check(torch, q, k, v, path=path)
    rows = torch.tensor([1, 40, 255, 256, nq - 1], device="cuda")
    q[rows, 0, 3] = torch.tensor([float("nan"), float("inf"), -float("inf"), float("nan"), float("nan")], device="cuda",
                                 dtype=torch.bfloat16)
    out = torch.empty_like(clean)
    ql.qlinear_attention(q, k, v, out)
    assert torch.isnan(out[rows, 0]).all()  # an infinite query has scores of both infinities
    out[rows, 0] = clean[rows, 0]
    assert torch.equal(out, clean)


@pytest.mark.parametrize("nq,nk,D,path", [(3, 500, 64, "rows32_slots0"), (3, 4000, 256, "rows32_slots512"),
                                          (100, 500, 128, "rows128_slots0"), (100, 1500, 192, "rows128_slots256"),
                                          (2000, 9000, 256, "rows256_slots256"), (33024, 4100, 64, "rows256_slots512")])
def test_large_scores_and_values(torch, nq, nk, D, path):
    """One key is far ahead of the others, so its values are what every query gives, bit for bit: the other weights vanish,
    and a bf16 value times a bf16 weight is exact in fp32 and so divided by the weight again. With scores beyond those
    that are served a query may be NaN, but is never zeros."""
    g = torch.Generator(device="cuda").manual_seed(D)
    base = torch.randn((1, 1, D), generator=g, device="cuda").to(torch.bfloat16)
    q = base.repeat(nq, 1, 1)
    k = (0.2 * torch.randn((nk, 1, D), generator=g, device="cuda")).to(torch.bfloat16)
    best = nk * 2 // 3
    k[best] = base[0]
    v = torch.randn((nk, 1, D), generator=g, device="cuda").to(torch.bfloat16)
    square = (base.double() ** 2).sum().item()
    out = torch.empty_like(q)
    for sign in (1.0, -1.0):
        # all scores far below zero: the best key's, at -2^lg, is the least of them
        if sign < 0:
            k = (base * 4).expand(nk, 1, D).contiguous()
            k[best] = base[0]
            q = -q
        for lg in (10, 20, 25.5, 26, 28, 30, 31, 32, 33, 34, 50):
            ql.qlinear_attention(q, k, v, out, scale=0.97 * 2.0 ** lg / square)
            assert ql.qlinear_last_path() == "attention_" + path
            right = (out == v[best]).all(dim=2)
            served = lg <= (28 if sign > 0 else 26)  # the other keys' scores are four times as far below
            assert right.all() if served else (right | ~torch.isfinite(out).all(dim=2)).all(), lg
    out.fill_(7.0)
    ql.qlinear_attention(q, k, v, out, key_mask=torch.zeros(nk, dtype=torch.bool, device="cuda"), scale=1e9)
    assert (out == 0).all()
    v = (v.abs() + 1) * 2.0 ** 80  # 9000 of them below 2^100
    ql.qlinear_attention(q, k, v, out, scale=0.97 * 2.0 ** 26 / square)
    assert (out == v[best]).all()
    ql.qlinear_attention(q, k, v, out, scale=1e-30)
    mean = v.double().mean(dim=0)
    assert ((out.double() - mean).abs() <= 2.0 ** -7 * mean).all()  # the weights' rounding and the output's, 2^-8 each


@pytest.mark.parametrize("nq,nk,hq,hkv,D,path", [(8237, 1100, 8, 2, 88, "rows128_slots512"), (8300, 2200, 8, 8, 256, "rows256_slots256"),
                                                 (8300, 700, 8, 8, 256, "rows256_slots0_rest32"),
                                                 (32850, 4100, 4, 1, 64, "rows256_slots512")])
def test_in_place(torch, nq, nk, hq, hkv, D, path):
    q, k, v = make(torch, nq, nk, hq, hkv, D, 53)
    want = ql.qlinear_attention(q, k, v, torch.empty_like(q))
    again = q.clone()
    ql.qlinear_attention(again, k, v, again)
    assert ql.qlinear_last_path() == "attention_" + path
    assert torch.equal(again, want)


@pytest.mark.parametrize("nq,nk,D", [(20, 700, 64), (300, 600, 128), (300, 8100, 256)])
@pytest.mark.parametrize("far", ["q", "k", "v", "out"])
def test_largest_pitches(torch, nq, nk, D, far):
    """One of the arrays with the longest rows that are served: byte offsets pass 31 bits within queries and 32 within keys,
    29 within 64 rows."""
    q, k, v = make(torch, nq, nk, 2, 2, D, 19)
    want = check(torch, q, k, v)
    t = {"q": q, "k": k, "v": v, "out": torch.empty_like(q)}
    long = torch.full((t[far].shape[0], 1 << 22), 7.0, dtype=torch.bfloat16, device="cuda")
    t[far] = long[:, 8:8 + 2 * D].unflatten(1, (2, D)).copy_(t[far])
    ql.qlinear_attention(t["q"], t["k"], t["v"], t["out"])
    assert torch.equal(t["out"], want)
    assert (long[:, :8] == 7.0).all() and (long[:, 8 + 2 * D:] == 7.0).all()


# queries, keys, samples, query heads, key heads, D
DEVICE = [(40, 20000, 4, 2, 2, 64), (700, 20000, 4, 2, 2, 128), (900, 20000, 4, 2, 2, 256), (3000, 9000, 4, 2, 1, 192)]


# the last two ask for more tiles than there are blocks to join, and for more pieces than there is room for
@pytest.mark.parametrize("nq,nk,samples,hq,hkv,D", DEVICE + [(896, 140000, 64, 1, 1, 64), (2560, 60000, 16, 3, 3, 128)])
def test_offsets_out_of_order_stay_within_their_arrays(torch, nq, nk, samples, hq, hkv, D):
    """Offsets under which several samples have all queries and all keys. The values of out are unspecified, but neither
    rows beside it nor bytes behind the workspace are touched, and the next call is none the worse."""
    need = ql.qlinear_attention_workspace_bytes(nq, nk, samples, hq, hkv, D)
    assert need > 0
    q, k, v = make(torch, nq, nk, hq, hkv, D, 47)
    space = torch.full((nq + 2, hq, D), 7.0, dtype=torch.bfloat16, device="cuda")
    ws = torch.full((need + (1 << 20),), 77, dtype=torch.uint8, device="cuda")
    big, low = 2147483647, -2147483648
    turns = lambda x: torch.tensor([x[i % len(x)] for i in range(samples + 1)], dtype=torch.int32, device="cuda")  # noqa: E731
    for a, b in (((nq, 0), (nk // 50, 0, nk, 0)), ((0, nq), (0, nk)), ((low, big), (low, big)), ((0, big), (nk // 2, nk))):
        ql.qlinear_attention(q, k, v, space[1:-1], q_offsets=turns(a), k_offsets=turns(b), workspace=ws[:need])
        torch.cuda.synchronize()
        assert not ql.qlinear_last_path().endswith("slots0")
        assert (space[0] == 7.0).all() and (space[-1] == 7.0).all() and (ws[need:] == 77).all()
    even = [nq // samples - 1] * samples, [nk // samples - 1] * samples
    check(torch, q, k, v, *even, workspace=ws)


@pytest.mark.parametrize("nq,nk,samples,hq,hkv,D", DEVICE)
def test_a_graph_follows_offsets_that_move_what_is_cut(torch, nq, nk, samples, hq, hkv, D):
    """One captured call over lengths that give the long sample to each place in turn, that cut nothing, that cut
    everything, and that leave samples empty: each replay against 64 bits and against the eager call."""
    q, k, v = make(torch, nq, nk, hq, hkv, D, 31)
    qo = torch.zeros(samples + 1, dtype=torch.int32, device="cuda")
    ko, mask = torch.zeros_like(qo), torch.ones(nk, dtype=torch.bool, device="cuda")
    ws = torch.empty(ql.qlinear_attention_workspace_bytes(nq, nk, samples, hq, hkv, D), dtype=torch.uint8, device="cuda")
    assert ws.numel() > 0
    out = torch.zeros_like(q)

    def call(o, w):
        ql.qlinear_attention(q, k, v, o, q_offsets=qo, k_offsets=ko, key_mask=mask, workspace=w)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        call(out, ws)
    assert not ql.qlinear_last_path().endswith("slots0")
    most, some = nk - 300, 100
    lengths = [([nq // 4] * 4, [nk // 4] * 4),
               ([nq - 3, 1, 1, 1], [most, some, some, some]), ([1, nq - 3, 1, 1], [some, most, some, some]),
               ([1, 1, 1, nq - 3], [some, some, some, most]), ([nq // 4] * 4, [some] * 4),
               ([0, nq, 0, 0], [nk // 2, nk // 2, 0, 0]), ([0, 0, 0, 0], [0, 0, 0, nk]), ([5, 0, 7, 9], [0, nk, 0, 0]),
               ([nq // 4] * 4, [nk // 4] * 4)]
    for i, (a, b) in enumerate(lengths):
        at = edges(a), edges(b)
        qo.copy_(torch.tensor(at[0]))
        ko.copy_(torch.tensor(at[1]))
        mask.copy_(torch.arange(nk) % (3 + i) != 0)
        eager = torch.zeros_like(q)
        torch.cuda.synchronize()
        call(eager, ql.TORCH_WORKSPACE)
        out.zero_()
        ws.fill_(255)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, eager)
        compare(torch, out, torch.zeros_like(q), q, k, v, D ** -0.5, *at, mask)
