"""CPU tests of qlinear_block_norm and qlinear_adapters: the oracle's
definitions against hand values, workspace sizing, and every refusal (each
failing call is rejected before any HIP call)."""
import ctypes

import numpy as np
import pytest

import oracle
from group_wise_affine_qlinear_amd import qlinear as ql

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def lib():
    return ql.load_library()


def test_oracle_norms_by_hand():
    v = np.array([[3.0, 4.0]])
    assert np.allclose(oracle.norm_rows(v, "rms", 1e-30), v / np.sqrt(12.5), rtol=1e-15)
    assert np.allclose(oracle.norm_rows(v, "layer", 1e-30), [[-1.0, 1.0]], rtol=1e-15)
    assert np.allclose(oracle.norm_rows(v, "rms", 12.5), v / 5.0, rtol=1e-7)
    assert np.array_equal(oracle.norm_rows(v, "none", 1.0), v)


def test_oracle_block_norm_by_hand():
    r, h = oracle.block_norm(np.array([[1.0, 2.0]]), np.array([[3.0, 4.0]]), residual_scale=0.5, post="layer",
                             post_eps=1e-30, post_weight=np.array([2.0, 3.0]), post_bias=np.array([1.0, 0.0]),
                             gate=np.array([[0.5, -1.0]]), pre="rms", pre_eps=1e-30, pre_bias=np.array([1.0, 1.0]),
                             scale=np.array([[1.0, 0.0]]), shift=np.array([[0.0, 10.0]]))
    # z = (-1 * 2 + 1, 1 * 3) = (-1, 3); r = (0.5 - 0.5, 1 - 3) = (0, -2); rms sqrt(2)
    assert np.allclose(r, [[0.0, -2.0]])
    assert np.allclose(h, [[2.0, 11.0 - np.sqrt(2.0)]])


def test_oracle_adapter_delta_by_hand():
    x = np.array([[1.0, 2.0], [3.0, 4.0], [5.0, 6.0]])
    a = np.array([[[1.0, 0.0], [0.0, 1.0]], [[1.0, 1.0], [1.0, -1.0]]])
    b = np.array([[[1.0, 2.0]], [[3.0, 4.0]]])
    d = oracle.adapter_delta(x, a, b, [0, 1, 7], scaling=[2.0, 1.0])
    # row 0: v = (1, 2), 2 * (1 + 4); row 1: v = (7, -1), 21 - 4; row 2: none
    assert d.tolist() == [[10.0], [17.0], [0.0]]
    assert oracle.adapter_delta(x, a, b, [0, 1, -1], ranks=[1, 9]).tolist() == [[1.0], [17.0], [0.0]]


def _norm(**kw):
    a = ql.ql_block_norm_args()
    base = dict(M=4, D=64, residual=0x1000, residual_dtype=1, residual_scale=1.0, y=0x2000, y_dtype=0, post_norm=1,
                post_eps=1e-6, gate=0x3000, gate_ld=64, residual_out=0x1000, pre_norm=2, pre_eps=1e-6, scale=0x4000,
                scale_ld=64, shift=0x5000, shift_ld=64, mod_rows=2, h=0x6000)
    base.update(kw)
    for k, v in base.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("kw,status", [
    (dict(M=-1), ql.QL_EINVAL),
    (dict(D=0), ql.QL_EINVAL),
    (dict(D=65537, gate_ld=1 << 20, scale_ld=1 << 20, shift_ld=1 << 20), ql.QL_EUNSUPPORTED),
    (dict(M=1 << 40), ql.QL_EUNSUPPORTED),
    (dict(residual=0), ql.QL_EINVAL),
    (dict(residual_dtype=2), ql.QL_EINVAL),
    (dict(y_dtype=-1), ql.QL_EINVAL),
    (dict(residual_scale=float("nan")), ql.QL_EINVAL),
    (dict(residual_scale=float("inf")), ql.QL_EINVAL),
    (dict(post_norm=3), ql.QL_EINVAL),
    (dict(post_eps=0.0), ql.QL_EINVAL),
    (dict(pre_eps=-1e-6), ql.QL_EINVAL),
    (dict(pre_eps=float("nan")), ql.QL_EINVAL),
    (dict(pre_eps=float("inf")), ql.QL_EINVAL),
    (dict(h=0, residual_out=0), ql.QL_EINVAL),                       # no output
    (dict(h=0), ql.QL_EINVAL),                                       # a norm before, and nothing to put it in
    (dict(h=0, pre_norm=0), ql.QL_EINVAL),
    (dict(h=0, pre_norm=0, scale=0), ql.QL_EINVAL),
    (dict(x16=0x7000), ql.QL_EINVAL),                                # without rowscale
    (dict(rowscale=0x7000), ql.QL_EINVAL),
    (dict(y=0), ql.QL_EINVAL),                                       # an update without y
    (dict(y=0, residual_out=0), ql.QL_EINVAL),
    (dict(y=0, residual_out=0, gate=0), ql.QL_EINVAL),
    (dict(y=0, residual_out=0, gate=0, post_norm=0, post_weight=0x8000), ql.QL_EINVAL),
    (dict(gate_ld=63), ql.QL_EINVAL),
    (dict(scale_ld=0), ql.QL_EINVAL),
    (dict(shift_ld=-64), ql.QL_EINVAL),
    (dict(mod_rows=-1), ql.QL_EINVAL),
    (dict(row_sample=0x9000, samples=-1), ql.QL_EINVAL),
    (dict(residual=0x1001, residual_out=0x1000), ql.QL_EALIGN),
    (dict(residual_out=0x1001), ql.QL_EALIGN),
    (dict(y=0x2002), ql.QL_EALIGN),
    (dict(h=0x6001), ql.QL_EALIGN),
    (dict(x16=0x7001, rowscale=0x8000), ql.QL_EALIGN),
    (dict(x16=0x7000, rowscale=0x8002), ql.QL_EALIGN),
    (dict(gate=0x3002), ql.QL_EALIGN),
    (dict(scale=0x4001), ql.QL_EALIGN),
    (dict(pre_weight=0x4002), ql.QL_EALIGN),
    (dict(row_sample=0x9002, samples=2), ql.QL_EALIGN),
])
def test_block_norm_refusals(lib, kw, status):
    assert lib.qlinear_block_norm(ctypes.byref(_norm(**kw)), None) == status


def test_block_norm_null_and_empty(lib):
    assert lib.qlinear_block_norm(None, None) == ql.QL_EINVAL
    assert lib.qlinear_block_norm(ctypes.byref(_norm(M=0)), None) == ql.QL_OK


def _adapters(**kw):
    a = ql.ql_adapter_args()
    base = dict(x=0x1000, a=0x2000, b=0x3000, ab_dtype=0, M=8, N=64, K=128, adapters=2, rank=16, row_adapter=0x4000,
                y=0x5000, y_dtype=0, out=0x6000, out_dtype=0, workspace=0x10000, workspace_bytes=1 << 30)
    base.update(kw)
    for k, v in base.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("kw,status", [
    (dict(M=-1), ql.QL_EINVAL),
    (dict(N=-1), ql.QL_EINVAL),
    (dict(K=100), ql.QL_EINVAL),
    (dict(K=-64), ql.QL_EINVAL),
    (dict(M=1 << 31), ql.QL_EINVAL),
    (dict(K=1 << 31), ql.QL_EINVAL),
    (dict(adapters=-1), ql.QL_EINVAL),
    (dict(rank=0), ql.QL_EUNSUPPORTED),
    (dict(rank=12), ql.QL_EUNSUPPORTED),
    (dict(rank=264), ql.QL_EUNSUPPORTED),
    (dict(rank=-8), ql.QL_EUNSUPPORTED),
    (dict(M=1 << 30, N=1 << 20), ql.QL_EUNSUPPORTED),                # more blocks than a grid holds
    (dict(ab_dtype=2), ql.QL_EINVAL),
    (dict(out_dtype=5), ql.QL_EINVAL),
    (dict(y_dtype=5), ql.QL_EINVAL),
    (dict(epilogue=3), ql.QL_EINVAL),
    (dict(epilogue=1, N=63), ql.QL_EINVAL),
    (dict(epilogue=1, y=0x6000), ql.QL_EINVAL),                      # SwiGLU in place
    (dict(y=0x6000, y_dtype=1), ql.QL_EINVAL),                       # in place across types
    (dict(epilogue=2), ql.QL_EINVAL),
    (dict(epilogue=2, residual=0x7000, gate=0x8000), ql.QL_EINVAL),
    (dict(epilogue=2, residual=0x7000, gate_rows=1), ql.QL_EINVAL),
    (dict(x=0), ql.QL_EINVAL),
    (dict(a=0), ql.QL_EINVAL),
    (dict(b=0), ql.QL_EINVAL),
    (dict(out=0), ql.QL_EINVAL),
    (dict(row_adapter=0), ql.QL_EINVAL),
    (dict(x=0x1008), ql.QL_EALIGN),
    (dict(a=0x2002), ql.QL_EALIGN),
    (dict(b=0x3008), ql.QL_EALIGN),
    (dict(workspace=0x10004), ql.QL_EALIGN),
    (dict(out=0x6002), ql.QL_EALIGN),
    (dict(y=0x5002), ql.QL_EALIGN),
    (dict(row_adapter=0x4002), ql.QL_EALIGN),
    (dict(ranks=0x4001), ql.QL_EALIGN),
    (dict(scaling=0x4002), ql.QL_EALIGN),
    (dict(epilogue=2, residual=0x7002, gate=0x8000, gate_rows=1), ql.QL_EALIGN),
    (dict(epilogue=2, residual=0x7000, gate=0x8002, gate_rows=1), ql.QL_EALIGN),
    (dict(workspace=0), ql.QL_EWORKSPACE),
    (dict(workspace_bytes=16), ql.QL_EWORKSPACE),
])
def test_adapters_refusals(lib, kw, status):
    assert lib.qlinear_adapters(ctypes.byref(_adapters(**kw)), None) == status


def test_adapters_null_and_empty(lib):
    assert lib.qlinear_adapters(None, None) == ql.QL_EINVAL
    assert lib.qlinear_adapters(ctypes.byref(_adapters(M=0)), None) == ql.QL_OK
    assert lib.qlinear_adapters(ctypes.byref(_adapters(N=0)), None) == ql.QL_OK


def test_adapters_workspace_sizes(lib):
    for M, N, K, r, n in ((1, 64, 64, 8, 1), (16, 4608, 4608, 16, 32), (4096, 4608, 12288, 64, 8), (300, 7, 0, 256, 3)):
        need = ql.qlinear_adapters_workspace_bytes(M, N, K, r, n)
        assert need > 0 and need % (M * r * 4) == 0, (M, N, K, r, n, need)
        a = _adapters(M=M, N=N, K=K, rank=r, adapters=n, workspace_bytes=need - 1)
        assert lib.qlinear_adapters(ctypes.byref(a), None) == ql.QL_EWORKSPACE
    assert ql.qlinear_adapters_workspace_bytes(8, 64, 128, 16, 0) == 0
    for bad in ((-1, 64, 64, 8, 1), (8, 64, 65, 8, 1), (8, 64, 64, 9, 1), (8, 64, 64, 8, -1), (0, 64, 64, 8, 1)):
        assert ql.qlinear_adapters_workspace_bytes(*bad) == 0, bad


def test_bindings_take_device_tensors_only():
    r = torch.zeros((4, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        ql.qlinear_block_norm(r, 4, 64, h=torch.zeros_like(r), pre_norm=ql.QL_NORM_RMS)
    x, a, b = (torch.zeros(s, dtype=torch.bfloat16) for s in ((4, 64), (1, 8, 64), (1, 32, 8)))
    with pytest.raises(ValueError):
        ql.qlinear_adapters(x, a, b, torch.zeros(4, dtype=torch.int32), 4, 32, 64, torch.zeros((4, 32)))


def test_adapter_mfma_operands_have_two_wait_states(tmp_path):
    """The adapters' products keep the wait states between a VALU write and an MFMA read (see test_isa_hazards)."""
    import os
    import subprocess

    from test_isa_hazards import _hipcc, scan

    from group_wise_affine_qlinear_amd import build as qb
    if _hipcc() is None:
        pytest.skip("hipcc not available")
    flags = [f for f in qb.COMMON_FLAGS if f not in ("-fPIC", "-fvisibility=hidden")]
    out = tmp_path / "adapters.s"
    res = subprocess.run([_hipcc(), *flags, "--cuda-device-only", "-S", os.path.join(qb.CSRC, "adapters.hip"), "-o", str(out)],
                         capture_output=True, text=True)
    assert res.returncode == 0, res.stderr[-2000:]
    n, bad = scan(out.read_text())
    assert n > 0 and not bad, bad[:5]


def test_host_code_under_asan_and_ubsan(tmp_path):
    """The validation and sizing code of both entry points under the sanitizers (host side only; no call
    reaches a device): host.cpp as in test_host_asan, with a driver of its own."""
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
          os.path.join(HERE, "host_asan", "driver_block.cpp"), "-o", drv_obj])
    _run([gxx, *SAN, drv_obj, host_obj, *others, "-L", "/opt/rocm/lib", "-lamdhip64", "-Wl,-rpath,/opt/rocm/lib", "-o", exe])
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:halt_on_error=1", UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1",
               HIP_VISIBLE_DEVICES="")
    res = subprocess.run([exe], capture_output=True, text=True, env=env, timeout=300)
    report = res.stdout + res.stderr
    assert "AddressSanitizer" not in report and "runtime error" not in report, report
    assert res.returncode == 0 and "host checks passed" in res.stdout, report


def test_adapters_piece_limit(lib):
    """2^24 - 1 pieces of 64 rows by 256 columns of out are served, one more is refused."""
    rows = 64 * ((1 << 24) - 1)
    none, swiglu = ql.QL_EPI_NONE, ql.QL_EPI_SWIGLU
    for M, N, epilogue, served in ((rows, 256, none, True), (rows, 512, swiglu, True), (rows + 1, 256, none, False),
                                   (rows + 1, 255, none, False), (rows, 257, none, False), (rows + 1, 512, swiglu, False),
                                   (rows, 514, swiglu, False), (1 << 30, 1 << 20, none, False)):
        need = ql.qlinear_adapters_workspace_bytes(M, N, 64, 8, 2)
        assert need >= M * 8 * 4
        a = _adapters(M=M, N=N, K=64, rank=8, workspace_bytes=need - 1, epilogue=epilogue)
        want = ql.QL_EWORKSPACE if served else ql.QL_EUNSUPPORTED
        assert lib.qlinear_adapters(ctypes.byref(a), None) == want, (M, N, epilogue)


def test_block_norm_row_limit(lib):
    assert lib.qlinear_block_norm(ctypes.byref(_norm(M=4194304)), None) == ql.QL_EUNSUPPORTED
    assert "limits" in ql.qlinear_status_string(ql.QL_EUNSUPPORTED)
