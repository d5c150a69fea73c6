"""CPU tests of qlinear_qk_norm_rope and qlinear_attention: the oracle's
definitions against hand values, workspace sizing, the table of rotations, and
every refusal (each failing call is rejected before any HIP call)."""
import ctypes

import numpy as np
import pytest

import oracle
from group_wise_affine_qlinear_amd import qlinear as ql
from test_binding_streams import SIDE, STREAMS, Stream, Tensor, taken, torch  # noqa: F401


@pytest.fixture(scope="module")
def lib():
    return ql.load_library()


def test_oracle_rotation_by_hand():
    u = np.array([[[1.0, 2.0, 3.0, 4.0, 9.0]]])
    quarter = np.float64(np.pi / 2)
    # pair 0 by a quarter turn, pair 1 by a half turn; the last value is not turned
    assert np.allclose(oracle.rotate_heads(u, [[1], [2]], [quarter, quarter], [0, 1]), [[[-3.0, -2.0, 1.0, -4.0, 9.0]]])
    assert np.allclose(oracle.rotate_heads(u, [[1], [2]], [quarter, quarter], [0, 1], "pairs"), [[[-2.0, 1.0, -3.0, -4.0, 9.0]]])
    assert np.allclose(oracle.rotate_heads(u, [[1], [2]], [quarter, quarter], [0, 2]), [[[-3.0, 2.0, 1.0, 4.0, 9.0]]])
    v = np.array([[[3.0, 4.0]]])
    got = oracle.qk_norm_rope(v, [2.0, 1.0], "rms", 1e-30, [[1]], [quarter])
    assert np.allclose(got, np.array([[[-4.0, 6.0]]]) / np.sqrt(12.5))


def test_oracle_attention_by_hand():
    q = np.array([[[1.0, 0.0]], [[0.0, 1.0]], [[5.0, 5.0]]])
    k = np.array([[[np.log(3.0), 0.0]], [[0.0, 0.0]], [[0.0, 2 * np.log(2.0)]]])
    v = np.array([[[1.0, 0.0]], [[0.0, 1.0]], [[8.0, 8.0]]])
    out, live = oracle.attention(q, k, v, 1.0, [0, 1, 2], [0, 2, 3])
    assert np.allclose(out[:2, 0], [[0.75, 0.25], [8.0, 8.0]]) and live.tolist() == [True, True, False]
    out, _ = oracle.attention(q, k, v, 0.5, key_mask=[0, 1, 1])
    # weights 1 and 2
    assert np.allclose(out[1, 0], [16 / 3, 17 / 3])
    assert (oracle.attention(q, k, v, 1.0, key_mask=[0, 0, 0])[0] == 0).all()
    # heads 0 and 1 share the first key head
    out, _ = oracle.attention(np.ones((1, 4, 2)), np.ones((1, 2, 2)), np.array([[[1.0, 2.0], [3.0, 4.0]]]), 1.0)
    assert out[0].tolist() == [[1, 2], [1, 2], [3, 4], [3, 4]]


@pytest.mark.parametrize("order", [ql.QL_ROPE_AXES_OWN, ql.QL_ROPE_AXES_SHARED, ql.QL_ROPE_AXES_TURNS])
def test_rope_table(order):
    f, a = ql.qlinear_rope_table_host(100.0, [3, 1, 2], order)
    if order == ql.QL_ROPE_AXES_OWN:
        want, axis = [1, 100 ** (-1 / 3), 100 ** (-2 / 3), 1, 1, 0.1], [0, 0, 0, 1, 2, 2]
    else:
        want = [100 ** (-i / 6) for i in range(6)]
        axis = [0, 0, 0, 1, 2, 2] if order == ql.QL_ROPE_AXES_SHARED else [0, 1, 2, 0, 2, 0]
    assert np.array_equal(f, np.float32(want)) and a.tolist() == axis
    with pytest.raises(ql.QLinearError):
        ql.qlinear_rope_table_host(100.0, [3], 3)
    with pytest.raises(ql.QLinearError):
        ql.qlinear_rope_table_host(100.0, [])


@pytest.mark.parametrize("pairs", [[65537], [1 << 45], [65536, 1], [1 << 62, 1 << 62], [1 << 45, -(1 << 45)], [4, -1]])
def test_rope_table_refuses_sizes(pairs):
    """More pairs than a table has are refused by the library, before memory is taken for them."""
    with pytest.raises(ql.QLinearError):
        ql.qlinear_rope_table_host(100.0, pairs)


def _qk(**kw):
    a = ql.ql_qk_args()
    base = dict(M=4, head_dim=64, q_heads=4, kv_heads=2, q=0x1000, k=0x2000, v=0x3000, q_ld=256, k_ld=128, v_ld=128, in_dtype=0,
                q_out=0x4000, k_out=0x5000, v_out=0x6000, q_out_ld=256, k_out_ld=128, v_out_ld=128, norm=1, eps=1e-6,
                q_weight=0x7000, k_weight=0x7100, rope=0, pairs=32, freqs=0x8000, pair_axis=0x8100, axes=3, positions=0x9000)
    base.update(kw)
    for k, v in base.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("kw,status", [
    (dict(M=-1), ql.QL_EINVAL),
    (dict(M=1 << 24), ql.QL_EUNSUPPORTED),
    (dict(head_dim=0), ql.QL_EINVAL),
    (dict(head_dim=60), ql.QL_EUNSUPPORTED),
    (dict(head_dim=264), ql.QL_EUNSUPPORTED),
    (dict(q_heads=-1), ql.QL_EINVAL),
    (dict(q_heads=0), ql.QL_EINVAL),
    (dict(kv_heads=0), ql.QL_EINVAL),
    (dict(q_heads=65537), ql.QL_EUNSUPPORTED),
    (dict(kv_heads=1 << 40), ql.QL_EUNSUPPORTED),
    (dict(q=0, k=0, v=0, q_out=0, k_out=0, v_out=0, q_weight=0, k_weight=0), ql.QL_EINVAL),
    (dict(q=0), ql.QL_EINVAL),
    (dict(k_out=0), ql.QL_EINVAL),
    (dict(v=0), ql.QL_EINVAL),
    (dict(q=0, q_out=0), ql.QL_EINVAL),                               # a weight for queries that are not there
    (dict(k=0, k_out=0), ql.QL_EINVAL),
    (dict(q_ld=255), ql.QL_EINVAL),
    (dict(v_ld=127), ql.QL_EINVAL),
    (dict(k_out_ld=0), ql.QL_EINVAL),
    (dict(in_dtype=2), ql.QL_EINVAL),
    (dict(q_out=0x1000), ql.QL_EINVAL),                               # fp32 in place
    (dict(in_dtype=1, q_out=0x1000, q_out_ld=264), ql.QL_EINVAL),     # in place with another pitch
    (dict(norm=3), ql.QL_EINVAL),
    (dict(eps=0.0), ql.QL_EINVAL),
    (dict(norm=2, eps=float("nan")), ql.QL_EINVAL),
    (dict(rope=2), ql.QL_EINVAL),
    (dict(pairs=-4), ql.QL_EINVAL),
    (dict(pairs=30), ql.QL_EUNSUPPORTED),
    (dict(pairs=36), ql.QL_EINVAL),
    (dict(freqs=0), ql.QL_EINVAL),
    (dict(positions=0), ql.QL_EINVAL),
    (dict(axes=0), ql.QL_EINVAL),
    (dict(axes=65537), ql.QL_EUNSUPPORTED),
    (dict(q=0x1002), ql.QL_EALIGN),
    (dict(v_out=0x6001), ql.QL_EALIGN),
    (dict(q_weight=0x7002), ql.QL_EALIGN),
    (dict(freqs=0x8002), ql.QL_EALIGN),
    (dict(pair_axis=0x8101), ql.QL_EALIGN),
    (dict(positions=0x9002), ql.QL_EALIGN),
    (dict(rows_end=0xa002), ql.QL_EALIGN),
])
def test_qk_refusals(lib, kw, status):
    assert lib.qlinear_qk_norm_rope(ctypes.byref(_qk(**kw)), None) == status


def test_qk_null_and_empty(lib):
    assert lib.qlinear_qk_norm_rope(None, None) == ql.QL_EINVAL
    assert lib.qlinear_qk_norm_rope(ctypes.byref(_qk(M=0)), None) == ql.QL_OK


@pytest.mark.parametrize("kw", [dict(q=0, k=0, v=0, q_out=0, k_out=0, v_out=0, positions=0), dict(q=0, k=0, v=0),
                                dict(q=0, q_out=0), dict(k_out=0, v_out=0)])
def test_qk_without_rows_has_null_arrays(lib, kw):
    """Tensors without elements give null pointers, beside weights and outputs that are there."""
    assert lib.qlinear_qk_norm_rope(ctypes.byref(_qk(M=0, **kw)), None) == ql.QL_OK
    for bad, status in ((dict(head_dim=60), ql.QL_EUNSUPPORTED), (dict(norm=3), ql.QL_EINVAL), (dict(pairs=36), ql.QL_EINVAL)):
        assert lib.qlinear_qk_norm_rope(ctypes.byref(_qk(M=0, **kw, **bad)), None) == status


def _att(**kw):
    a = ql.ql_attention_args()
    base = dict(q=0x1000, k=0x2000, v=0x3000, out=0x4000, q_ld=512, k_ld=128, v_ld=128, out_ld=512, Mq=16, Mk=5000, q_heads=8,
                kv_heads=2, head_dim=64, scale=0.125, samples=3, q_offsets=0x5000, k_offsets=0x6000, key_mask=0x7001,
                workspace=0x10000, workspace_bytes=16)
    base.update(kw)
    for k, v in base.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("kw,status", [
    (dict(), ql.QL_EWORKSPACE),
    (dict(Mq=-1), ql.QL_EINVAL),
    (dict(Mk=-1), ql.QL_EINVAL),
    (dict(q_heads=0), ql.QL_EINVAL),
    (dict(kv_heads=0), ql.QL_EINVAL),
    (dict(kv_heads=3), ql.QL_EINVAL),
    (dict(q_heads=65544), ql.QL_EUNSUPPORTED),
    (dict(Mq=(1 << 28) + 1), ql.QL_EUNSUPPORTED),
    (dict(Mk=(1 << 30) + 1), ql.QL_EUNSUPPORTED),
    (dict(head_dim=0), ql.QL_EINVAL),
    (dict(head_dim=68), ql.QL_EUNSUPPORTED),
    (dict(head_dim=264), ql.QL_EUNSUPPORTED),
    (dict(samples=-1), ql.QL_EINVAL),
    (dict(samples=(1 << 20) + 1), ql.QL_EUNSUPPORTED),
    (dict(samples=1 << 20, kv_heads=65536, q_heads=65536, Mq=1), ql.QL_EUNSUPPORTED),  # more blocks than a grid holds
    (dict(scale=0.0), ql.QL_EINVAL),
    (dict(scale=-1.0), ql.QL_EINVAL),
    (dict(scale=float("nan")), ql.QL_EINVAL),
    (dict(scale=float("inf")), ql.QL_EINVAL),
    (dict(scale=1.1e30), ql.QL_EINVAL),
    (dict(scale=0.9e-30), ql.QL_EINVAL),
    (dict(q_offsets=0), ql.QL_EINVAL),
    (dict(k_offsets=0), ql.QL_EINVAL),
    (dict(q=0), ql.QL_EINVAL),
    (dict(k=0), ql.QL_EINVAL),
    (dict(v=0), ql.QL_EINVAL),
    (dict(out=0), ql.QL_EINVAL),
    (dict(q_ld=504), ql.QL_EINVAL),
    (dict(out_ld=0), ql.QL_EINVAL),
    (dict(k_ld=120), ql.QL_EINVAL),
    (dict(v_ld=120), ql.QL_EINVAL),
    (dict(q_ld=516), ql.QL_EALIGN),
    (dict(v_ld=132), ql.QL_EALIGN),
    (dict(k_ld=(1 << 22) + 8), ql.QL_EUNSUPPORTED),
    (dict(out_ld=(1 << 22) + 8), ql.QL_EUNSUPPORTED),
    (dict(q=0x1008), ql.QL_EALIGN),
    (dict(k=0x2008), ql.QL_EALIGN),
    (dict(v=0x3002), ql.QL_EALIGN),
    (dict(out=0x4008), ql.QL_EALIGN),
    (dict(workspace=0x10008), ql.QL_EALIGN),
    (dict(q_offsets=0x5002), ql.QL_EALIGN),
    (dict(k_offsets=0x6001), ql.QL_EALIGN),
])
def test_attention_refusals(lib, kw, status):
    assert lib.qlinear_attention(ctypes.byref(_att(**kw)), None) == status


def test_attention_in_place_has_one_pitch(lib):
    """Rows of out that do not lie on those of q would be overwritten before other blocks read them."""
    kw = dict(out=0x1000, out_ld=520, workspace_bytes=0)
    assert lib.qlinear_attention(ctypes.byref(_att(**kw)), None) == ql.QL_EINVAL
    # the same pitch, or one row, goes on to the next check
    for more in (dict(out_ld=512), dict(Mq=1)):
        assert lib.qlinear_attention(ctypes.byref(_att(**{**kw, **more})), None) == ql.QL_EWORKSPACE


def test_attention_null_and_empty(lib):
    assert lib.qlinear_attention(None, None) == ql.QL_EINVAL
    assert lib.qlinear_attention(ctypes.byref(_att(Mq=0)), None) == ql.QL_OK
    assert lib.qlinear_attention(ctypes.byref(_att(samples=0)), None) == ql.QL_OK


@pytest.mark.parametrize("Mq,samples,group,heads,tile", [
    (1 << 20, 1 << 20, 1, 15, 32), (1 << 20, 1 << 20, 1, 16, 32), (1 << 20, 1 << 18, 8, 32, 32), (1 << 20, 1 << 18, 8, 31, 32),
    (1 << 27, 1, 8, 8, 128), (1 << 23, 1, 8, 64, 128), (1 << 27, 100, 1, 15, 128), (1 << 27, 100, 1, 16, 128),
    (1 << 30, 1 << 20, 1, 1, 128), (1 << 30, 1 << 20, 1, 2, 128)])
def test_attention_limit_of_tiles(lib, Mq, samples, group, heads, tile):
    """What the header says is served and what is refused; an address that is not aligned is looked at behind the sizes."""
    kw = dict(Mq=Mq, samples=samples, q_heads=group * heads, kv_heads=heads, head_dim=128, q=0x1008, q_ld=group * heads * 128,
              out_ld=group * heads * 128, k_ld=heads * 128, v_ld=heads * 128)
    tiles = (-(-Mq * group // tile) + samples) * heads
    assert tiles < 2 ** 24 - 2048 or tiles >= 2 ** 24
    status = ql.QL_EALIGN if tiles < 2 ** 24 else ql.QL_EUNSUPPORTED
    assert lib.qlinear_attention(ctypes.byref(_att(**kw)), None) == status


def test_attention_keys_of_one_sum(lib):
    """Keys that nothing cuts are refused where fp32 sums lose too much, but for samples, whose lengths the host does not see."""
    one = dict(samples=0, q_offsets=0, k_offsets=0)
    # whole tiles of many rows; rows that four waves share; keys that are cut
    for kw, most in ((dict(Mq=4608, q_heads=18, kv_heads=18, head_dim=256, q_ld=4608, k_ld=4608, v_ld=4608, out_ld=4608), 1 << 22),
                     (dict(Mq=300000, q_heads=2, kv_heads=2), 1 << 22)):
        assert lib.qlinear_attention(ctypes.byref(_att(Mk=most, **one, **kw)), None) == ql.QL_EWORKSPACE
        assert lib.qlinear_attention(ctypes.byref(_att(Mk=most + 1, **one, **kw)), None) == ql.QL_EUNSUPPORTED
        assert lib.qlinear_attention(ctypes.byref(_att(Mk=most + 1, **{**one, **kw, "workspace": 0})), None) == ql.QL_EUNSUPPORTED
        assert lib.qlinear_attention(ctypes.byref(_att(Mk=1 << 30, **kw)), None) == ql.QL_EWORKSPACE
    assert lib.qlinear_attention(ctypes.byref(_att(Mk=(1 << 24) + 1, Mq=4, workspace=0, **one)), None) == ql.QL_EUNSUPPORTED
    assert lib.qlinear_attention(ctypes.byref(_att(Mk=1 << 30, Mq=4, **one)), None) == ql.QL_EWORKSPACE


def test_attention_workspace(lib):
    for case in ((16, 5000, 3, 8, 2, 64), (1, 65536, 1, 18, 18, 256), (77, 16896, 1, 24, 24, 128), (4608, 4608, 1, 18, 18, 256)):
        need = ql.qlinear_attention_workspace_bytes(*case)
        assert 0 < need < 600 << 20 and need % 16 == 0, (case, need)
        Mq, Mk, S, hq, hkv, D = case
        a = _att(Mq=Mq, Mk=Mk, samples=S, q_heads=hq, kv_heads=hkv, head_dim=D, q_ld=hq * D, out_ld=hq * D, k_ld=hkv * D,
                 v_ld=hkv * D, workspace_bytes=need - 1)
        assert lib.qlinear_attention(ctypes.byref(a), None) == ql.QL_EWORKSPACE
    for none in ((0, 100, 1, 1, 1, 64), (8, 0, 1, 1, 1, 64), (8, 10, 1, 1, 1, 64), (8, 9000, 1, 3, 2, 64), (8, 9000, 1, 2, 2, 60),
                 (-1, 9000, 1, 2, 2, 64), (8, 9000, 0, 2, 2, 64)):
        assert ql.qlinear_attention_workspace_bytes(*none) == 0, none


# ------------------------------------------------------------------ binding (stand-ins of test_binding_streams)

REAL = ql.load_library()


@pytest.fixture
def made(taken):  # noqa: F811
    ql._torch().bool = torch.bool
    # sizes as the library gives them: the stand-in answers every other call with 0
    ql.load_library().qlinear_attention_workspace_bytes = REAL.qlinear_attention_workspace_bytes
    return taken


class Heads(Tensor):
    def stride(self):
        return (self.shape[1] * self.shape[2], self.shape[2], 1)


def _call_attention(stream=None, **kw):
    bf16, i32 = torch.bfloat16, torch.int32
    args = dict(q=Heads((8, 4, 64), bf16), k=Heads((9000, 2, 64), bf16), v=Heads((9000, 2, 64), bf16), out=Heads((8, 4, 64), bf16),
                q_offsets=Tensor((3,), i32), k_offsets=Tensor((3,), i32), key_mask=Tensor((9000,), torch.bool))
    args.update(kw)
    return ql.qlinear_attention(args.pop("q"), args.pop("k"), args.pop("v"), args.pop("out"), stream=stream, **args)


def _call_qk(stream=None, **kw):
    f32, bf16, i32 = torch.float32, torch.bfloat16, torch.int32
    args = dict(q=Heads((8, 4, 64), f32), k=Heads((8, 2, 64), f32), v=Heads((8, 2, 64), f32), q_out=Heads((8, 4, 64), bf16),
                k_out=Heads((8, 2, 64), bf16), v_out=Heads((8, 2, 64), bf16), q_weight=Tensor((64,), f32),
                k_weight=Tensor((64,), f32), freqs=Tensor((32,), f32), pair_axis=Tensor((32,), i32),
                positions=Tensor((3, 8), i32), rows_end=Tensor((1,), i32))
    args.update(kw)
    ql.qlinear_qk_norm_rope(8, 64, stream=stream, **args)


@pytest.mark.parametrize("stream,handle", STREAMS)
def test_scratch_is_taken_on_the_stream_of_the_call(made, stream, handle):
    _call_attention(stream)
    assert [t.taken_on for t in made] == [handle]


def test_scratch_of_the_caller_is_used(made):
    _call_attention(Stream(SIDE), workspace=Tensor((4096,), torch.uint8))
    _call_attention(workspace=None)
    _call_attention(k=Heads((9, 2, 64), torch.bfloat16), v=Heads((9, 2, 64), torch.bfloat16), key_mask=None)  # nothing to cut
    _call_qk()
    assert made == []


@pytest.mark.parametrize("name", ["q", "k", "v", "out", "q_offsets", "k_offsets", "key_mask", "workspace"])
def test_attention_takes_tensors(made, name):
    for bad in ([1.0], 3.0, np.zeros((8, 4, 64), np.float32), "out"):
        with pytest.raises(ValueError if name == "workspace" and isinstance(bad, str) else TypeError):
            _call_attention(**{name: bad})


@pytest.mark.parametrize("name", ["q", "k", "v", "q_out", "k_out", "v_out", "q_weight", "k_weight", "freqs", "pair_axis", "positions",
                                  "rows_end"])
def test_qk_takes_tensors(made, name):
    for bad in ([1.0], 3.0, np.zeros((8, 4, 64), np.float32), "q"):
        with pytest.raises(TypeError):
            _call_qk(**{name: bad})


def test_shapes_and_types_are_checked(made):
    f32, bf16, i32 = torch.float32, torch.bfloat16, torch.int32
    for kw, error in ((dict(k=Heads((9000, 3, 64), bf16)), ValueError), (dict(v=Heads((8999, 2, 64), bf16)), ValueError),
                      (dict(out=Heads((8, 3, 64), bf16)), ValueError), (dict(q=Heads((8, 4, 64), f32)), TypeError),
                      (dict(out=Heads((8, 4, 64), f32)), TypeError), (dict(k_offsets=Tensor((4,), i32)), ValueError),
                      (dict(k_offsets=None), ValueError), (dict(q_offsets=None), ValueError),
                      (dict(key_mask=Tensor((8999,), torch.bool)), ValueError), (dict(key_mask=Tensor((9000,), i32)), TypeError),
                      (dict(workspace="device"), ValueError)):
        with pytest.raises(error):
            _call_attention(**kw)
    for kw, error in ((dict(k=Heads((8, 4, 64), f32)), ValueError), (dict(v=Heads((8, 2, 64), bf16)), TypeError),
                      (dict(q_out=None), TypeError), (dict(q=None), ValueError), (dict(v=None), ValueError),
                      (dict(q_out=Heads((8, 4, 64), f32)), TypeError), (dict(positions=Tensor((3, 9), i32)), ValueError),
                      (dict(freqs=None), ValueError), (dict(positions=None), TypeError),
                      (dict(pair_axis=Tensor((31,), i32)), ValueError), (dict(rows_end=Tensor((2,), i32)), ValueError)):
        with pytest.raises(error):
            _call_qk(**kw)


def test_rows_must_not_overlap():
    import torch as real
    t = real.zeros((8, 4, 64), dtype=real.bfloat16)
    ok = ql._heads(real, t[:, :2], "q", real.bfloat16, 8, 64, t.device)
    assert ok == (t.data_ptr(), 256, 2)
    for bad in (t.transpose(0, 1)[:, :4].transpose(0, 1)[:, ::2], t[:, :, ::2].repeat(1, 1, 2)[:, ::2], t[:1].expand(8, 4, 64)):
        with pytest.raises(ValueError):
            ql._heads(real, bad, "q", real.bfloat16, 8, 64, t.device)


def test_bindings_take_device_tensors_only():
    import torch as real
    q = real.zeros((4, 2, 64), dtype=real.bfloat16)
    with pytest.raises(ValueError):
        ql.qlinear_attention(q, q, q, q.clone())
    with pytest.raises(ValueError):
        ql.qlinear_qk_norm_rope(4, 64, q=q, q_out=q.clone())


@pytest.fixture(scope="module")
def assembly(tmp_path_factory):
    """The attention's kernels as the library's flags compile them."""
    import os
    import subprocess

    from test_isa_hazards import _hipcc

    from group_wise_affine_qlinear_amd import build as qb
    if _hipcc() is None:
        pytest.skip("hipcc not available")
    flags = [f for f in qb.COMMON_FLAGS if f not in ("-fPIC", "-fvisibility=hidden")]
    out = tmp_path_factory.mktemp("asm") / "attention.s"
    res = subprocess.run([_hipcc(), *flags, "--cuda-device-only", "-S", os.path.join(qb.CSRC, "attention.hip"), "-o", str(out)],
                         capture_output=True, text=True)
    assert res.returncode == 0, res.stderr[-2000:]
    return out.read_text()


def test_mfma_operands_have_two_wait_states(assembly):
    """The attention's products keep the wait states between a VALU write and an MFMA read (see test_isa_hazards)."""
    from test_isa_hazards import scan
    n, bad = scan(assembly)
    assert n > 0 and not bad, bad[:5]


def test_accumulators_are_the_kernels_own(assembly):
    """attention_kernel names its accumulators in instructions of its own: no instruction that the compiler made touches
    an AGPR there, and no accumulator is read or written by them before the wait that a product needs."""
    import re
    kernels, name, own, since = 0, None, False, None
    for raw in assembly.splitlines():
        line = raw.split(";")[0].strip()
        m = re.match(r"(_Z\w*attention_kernel\w*):", raw)
        if m:
            name, since = m.group(1), None
            kernels += 1
        elif raw.startswith(".Lfunc_end"):
            name = None
        if name is None:
            continue
        if "#ASMSTART" in raw or "#ASMEND" in raw:
            own = "#ASMSTART" in raw
            continue
        if not line or line.startswith(".") or line.endswith(":"):
            continue
        agpr = re.search(r"\ba(\d+|\[)", line)
        assert own or not agpr, (name, line)
        op = line.split()[0]
        # instructions since the last product of each block of straight code; s_nop n counts n + 1
        if op.startswith("v_mfma") and agpr:
            since = 0
        elif op.startswith("v_accvgpr") and since is not None:
            assert since >= 19, (name, line, since)
        elif since is not None:
            since += int(line.split()[1]) + 1 if op == "s_nop" else 1
    assert kernels == 16  # heads of 64, 96, 128, 192 and 256, with and without a mask, 128 and (64, 192 and 256) 256 rows to a tile


def test_host_code_under_asan_and_ubsan(tmp_path):
    """The validation and sizing code of the entry points under the sanitizers (host side only; no call reaches a
    device): host.cpp as in test_host_asan, with a driver of its own."""
    import os
    import shutil
    import subprocess

    from test_host_asan import HERE, SAN, _run

    from group_wise_affine_qlinear_amd import build as qb
    others = [os.path.join(qb.BUILD_DIR, os.path.splitext(s)[0] + ".o") for s in qb.SOURCES if s != "host.cpp"]
    gxx = shutil.which("g++")
    if not gxx or not all(os.path.exists(o) for o in others):
        pytest.skip("library objects or g++ missing: run the library build first")
    host_san = []
    for f in SAN:
        host_san += ["-Xarch_host", f]
    flags = [f for f in qb.COMMON_FLAGS if f != "-O3"]
    host_obj, drv_obj, exe = (str(tmp_path / n) for n in ("host.o", "driver.o", "driver"))
    _run([qb.hipcc(), "-x", "hip", *flags, "-O1", "-g", *host_san, "-c", os.path.join(qb.CSRC, "host.cpp"), "-o", host_obj])
    _run([gxx, "-std=c++17", "-O1", "-g", *SAN, "-I", os.path.join(qb.ROOT, "include"), "-c",
          os.path.join(HERE, "host_asan", "driver_attention.cpp"), "-o", drv_obj])
    _run([gxx, *SAN, drv_obj, host_obj, *others, "-L", "/opt/rocm/lib", "-lamdhip64", "-Wl,-rpath,/opt/rocm/lib", "-o", exe])
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:halt_on_error=1", UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1",
               HIP_VISIBLE_DEVICES="")
    res = subprocess.run([exe], capture_output=True, text=True, env=env, timeout=300)
    report = res.stdout + res.stderr
    assert "AddressSanitizer" not in report and "runtime error" not in report, report
    assert res.returncode == 0 and "host checks passed" in res.stdout, report
