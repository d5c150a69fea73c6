"""CPU tests of where the binding takes device memory for a call on another stream.

torch's caching allocator hands a freed block out again at once to the stream
it was taken on, for work that is queued behind the block's last use there. A
block that is written by a call on another stream has to be taken under that
stream, or work that is still pending on the first one shares the memory. The
library and torch's device side are stand-ins here: what is checked is the
stream that is current at each allocation.
"""
import contextlib
import types

import pytest

from group_wise_affine_qlinear_amd import qlinear as ql

torch = pytest.importorskip("torch")

DEVICE = torch.device("cuda", 0)


class Stream:
    def __init__(self, handle):
        self.cuda_stream, self.device = handle, DEVICE


class Tensor:
    """A contiguous device tensor as the binding sees one."""

    is_cuda, device = True, DEVICE

    def __init__(self, shape, dtype, taken_on=None):
        self.shape, self.dtype, self.taken_on, self.recorded = tuple(shape), dtype, taken_on, []

    def data_ptr(self):
        return 0x1000

    def is_contiguous(self):
        return True

    def dim(self):
        return len(self.shape)

    def numel(self):
        n = 1
        for d in self.shape:
            n *= d
        return n

    def element_size(self):
        return torch.empty(0, dtype=self.dtype).element_size()

    def record_stream(self, stream):
        self.recorded.append(stream.cuda_stream)


CURRENT, SIDE = 0x10, 0x20


@pytest.fixture
def taken(monkeypatch):
    """The tensors that calls took, each with the handle of the stream that was current then."""
    made, current = [], [CURRENT]

    def empty(shape, dtype, device):
        assert device == DEVICE
        made.append(Tensor((shape,) if isinstance(shape, int) else shape, dtype, current[-1]))
        return made[-1]

    @contextlib.contextmanager
    def under(stream):
        current.append(stream.cuda_stream)
        yield
        current.pop()

    cuda = types.SimpleNamespace(stream=under, current_stream=lambda device=None: Stream(current[-1]),
                                 ExternalStream=lambda handle, device=None: Stream(handle),
                                 default_stream=lambda device=None: Stream(0), current_device=lambda: 0)
    fake = types.SimpleNamespace(Tensor=Tensor, empty=empty, cuda=cuda, _C=types.SimpleNamespace(),
                                 **{n: getattr(torch, n) for n in ("uint8", "int16", "uint16", "int32", "uint32", "float16",
                                                                   "bfloat16", "float32")})
    real = ql.load_library()

    class Library:
        """Launches nothing; sizes come from the library, and every call asks for scratch."""

        def __getattr__(self, name):
            if name in ("qlinear_forward_workspace_bytes", "qlinear_adapters_workspace_bytes"):
                return lambda *args: 4096
            if name.endswith(("_words", "_ld")):
                return getattr(real, name)
            return lambda *args: ql.QL_OK

    library = Library()
    monkeypatch.setattr(ql, "_torch", lambda: fake)
    monkeypatch.setattr(ql, "load_library", lambda: library)
    return made


STREAMS = [(None, CURRENT), (Stream(SIDE), SIDE), (SIDE, SIDE), (0, 0)]


def _adapters(stream, **kw):
    M, N, K, rank, n = 8, 64, 128, 16, 2
    bf16 = torch.bfloat16
    ql.qlinear_adapters(Tensor((M, K), bf16), Tensor((n, rank, K), bf16), Tensor((n, N, rank), bf16),
                        Tensor((M,), torch.int32), M, N, K, Tensor((M, N), torch.float32), stream=stream, **kw)


def _forward(stream, **kw):
    M, N, K = 8, 64, 128
    u16 = torch.int16
    ql.qlinear_forward_ex(Tensor((M, K), u16), Tensor((N, K // 8), torch.int32), Tensor((N, K // 64), u16),
                          Tensor((N, K // 64), u16), 4, M, N, K, Tensor((M, N), torch.float32), stream=stream, **kw)


@pytest.mark.parametrize("call", [_adapters, _forward])
@pytest.mark.parametrize("stream,handle", STREAMS)
def test_scratch_is_taken_on_the_stream_of_the_call(taken, call, stream, handle):
    call(stream)
    assert [t.taken_on for t in taken] == [handle]


@pytest.mark.parametrize("call", [_adapters, _forward])
def test_scratch_of_the_caller_is_used(taken, call):
    call(Stream(SIDE), workspace=Tensor((4096,), torch.uint8))
    assert taken == []


def _results(name, stream):
    M, N, K = 8, 64, 128
    u16 = torch.int16
    x = Tensor((M, K), u16)
    if name == "qlinear_group_sums":
        return [ql.qlinear_group_sums(x, M, K, stream=stream)]
    if name == "qlinear_fast_activations":
        return ql.qlinear_fast_activations(x, M, K, stream=stream)
    if name == "qlinear_fast_activations_adaln":
        return ql.qlinear_fast_activations_adaln(x, Tensor((1, K), torch.float32), M, M, K, stream=stream)
    weight = Tensor((N, K // 8), torch.int32), Tensor((N, K // 64), u16), Tensor((N, K // 64), u16)
    return getattr(ql, name)(*weight, 4, 64, N, K, stream=stream)


@pytest.mark.parametrize("name", ["qlinear_group_sums", "qlinear_fast_activations", "qlinear_fast_activations_adaln",
                                  "qlinear_repack", "qlinear_repack_glu"])
@pytest.mark.parametrize("stream,handle", STREAMS)
def test_results_are_taken_on_the_stream_of_the_call(taken, name, stream, handle):
    """Results also outlive what the current stream does with them."""
    results = list(_results(name, stream))
    assert results == taken and all(t.taken_on == handle for t in results)
    assert all(t.recorded == ([] if stream is None else [CURRENT]) for t in results)
