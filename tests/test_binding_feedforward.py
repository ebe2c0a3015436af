"""CPU checks of the feed-forward binding's rules for devices, with stand-ins
for CUDA tensors and a library that must not be called."""
import pytest
import torch

from moe_grouped_gemm_fp8_gb300 import _lib, api, feedforward

FP8, I32, BF16, F32 = torch.float8_e4m3fn, torch.int32, torch.bfloat16, torch.float32


class On(torch.Tensor):
    """A host tensor that says it lives on CUDA device `at`."""
    __torch_function__ = torch._C._disabled_torch_function_impl
    at = 0
    is_cuda = True
    device = property(lambda t: torch.device("cuda", t.at))

    def get_device(self):
        return self.at


def on(at, dtype, *shape):
    t = torch.zeros(*shape, dtype=torch.uint8 if dtype is FP8 else dtype)
    t = (t.view(FP8) if dtype is FP8 else t).as_subclass(On)
    t.at = at
    return t


def words(at, rows, cols, groups=None):
    return on(at, I32, *api.sf_packed_shape(rows, cols, groups))


@pytest.fixture
def calls(monkeypatch):
    """The library's entry points that were reached; cuda:0 is current."""
    seen = []

    class Lib:
        def __getattr__(self, name):
            return lambda *a: seen.append(name) or 0

    monkeypatch.setattr(_lib, "lib", Lib)
    monkeypatch.setattr(feedforward, "_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(api, "_raw_stream", lambda dev: 0)
    monkeypatch.setattr(feedforward, "_raw_stream", lambda dev: 0)
    real = torch.empty
    monkeypatch.setattr(torch, "empty", lambda *a, device=None, **kw: real(*a, **kw).as_subclass(On))
    return seen


M, K, F, G = 128, 256, 128, 2


def contiguous(at):
    index = on(at, I32, M)
    return lambda: feedforward.m_grouped_fp8_gated_gemm_nt_contiguous(
        on(0, FP8, M, K), words(0, M, K), on(0, FP8, G, 2 * F, K), words(0, 2 * F, K, G), index)


def masked(at):
    counts = on(at, I32, G)
    return lambda: feedforward.m_grouped_fp8_gated_gemm_nt_masked(
        on(0, FP8, G, M, K), words(0, M, K, G), on(0, FP8, G, 2 * F, K), words(0, 2 * F, K, G), counts)


def backward(at):
    index = on(at, I32, M)
    return lambda: feedforward.fp8_gated_backward(on(0, BF16, M, F), on(0, FP8, M, 2 * F), words(0, M, 2 * F),
                                                  m_indices=index)


def requantise(at):
    index = on(at, I32, M)
    return lambda: feedforward.requantize_fp8_cols(on(0, FP8, M, K), words(0, M, K), m_indices=index)


@pytest.mark.parametrize("make", [contiguous, masked, backward, requantise])
def test_an_index_tensor_of_another_device_is_refused(make, calls):
    make(0)()
    assert len(calls) == 1
    with pytest.raises(ValueError, match="current CUDA device is cuda:0"):
        make(1)()
    assert len(calls) == 1  # nothing reached the library


class Side:
    """A stand-in for a CUDA stream."""
    device = torch.device("cuda", 0)

    def __init__(self, handle):
        self.cuda_stream = handle


@pytest.fixture
def current(calls, monkeypatch):
    """The current stream, last; raw handle 7 stands for a side stream."""
    stack = [Side(0)]
    monkeypatch.setattr(torch.cuda, "set_stream", lambda s: stack.__setitem__(-1, s))
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: stack[-1])
    monkeypatch.setattr(torch.cuda, "default_stream", lambda: stack[0])
    monkeypatch.setattr(torch.cuda, "ExternalStream", Side)
    monkeypatch.setattr(api, "_raw_stream", lambda dev: stack[-1].cuda_stream)
    monkeypatch.setattr(feedforward, "_raw_stream", lambda dev: stack[-1].cuda_stream)
    return stack


class Copied(On):
    """A tensor of unusual strides whose copy notes the stream it is made on."""
    def is_contiguous(self):
        return False

    def contiguous(self):
        self.log.append(torch.cuda.current_stream().cuda_stream)
        return self


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("handle", [7, 0])
def test_a_copy_of_the_input_is_made_on_the_calls_stream(dtype, handle, calls, current, monkeypatch):
    used = []
    monkeypatch.setattr(On, "record_stream", lambda t, s: used.append(s.cuda_stream), raising=False)
    current.append(Side(3))  # the caller's own stream
    x = on(0, dtype, 4, 128).as_subclass(Copied)
    x.log = []
    api.quantize_fp8(x, 1, stream=handle)
    if dtype is F32:
        api.quantize_fp8_cols(x, stream=handle)
        api.transform_sf_into_required_layout(x, 4, 512, 1, stream=handle)
    assert x.log == [handle] * (3 if dtype is F32 else 1)
    # the results are not handed out again before the caller's stream is past their release
    assert used == [3] * (5 if dtype is F32 else 2)
    assert current[-1].cuda_stream == 3


def _tensors():
    """One call of every operator, on ordinary arguments."""
    x, w = on(0, BF16, M, K), on(0, F32, K)
    q, sf = on(0, FP8, M, K), words(0, M, K)
    b, sfb = on(0, FP8, 2 * F, K), words(0, 2 * F, K)
    bg, sfg = on(0, FP8, G, 2 * F, K), words(0, 2 * F, K, G)
    gu, gu_sf = on(0, FP8, M, 2 * F), words(0, M, 2 * F)
    r = on(0, F32, M)
    f = feedforward
    return {
        "quantize_fp8": lambda s: api.quantize_fp8(x, 1, stream=s),
        "dequantize_fp8": lambda s: f.dequantize_fp8(q, sf, stream=s),
        "requantize_fp8_cols": lambda s: f.requantize_fp8_cols(q, sf, stream=s),
        "fp8_gated_gemm_nt": lambda s: f.fp8_gated_gemm_nt(q, sf, b, sfb, out_format="fp8", checkpoint=True, stream=s),
        "contiguous": lambda s: f.m_grouped_fp8_gated_gemm_nt_contiguous(q, sf, bg, sfg, on(0, I32, M), stream=s),
        "masked": lambda s: f.m_grouped_fp8_gated_gemm_nt_masked(
            on(0, FP8, G, M, K), words(0, M, K, G), bg, sfg, on(0, I32, G), stream=s),
        "fp8_gated_backward": lambda s: f.fp8_gated_backward(on(0, BF16, M, F), gu, gu_sf, stream=s),
        "layer_norm": lambda s: f.layer_norm(x, w, w, stream=s),
        "layer_norm_backward": lambda s: f.layer_norm_backward(x, x, w, r, r, stream=s),
    }


@pytest.mark.parametrize("name", _tensors())
def test_results_and_workspaces_are_allocated_on_the_calls_stream(name, calls, current, monkeypatch):
    """What a call writes comes from its stream's memory: memory of the
    current stream may still be in use there."""
    where, inner = [], torch.empty
    monkeypatch.setattr(torch, "empty", lambda *a, **kw: where.append(torch.cuda.current_stream().cuda_stream) or
                        inner(*a, **kw))
    monkeypatch.setattr(On, "record_stream", lambda t, s: None, raising=False)
    monkeypatch.setattr(feedforward, "_backward_workspace", lambda cols, sms: 64)
    current.append(Side(3))
    _tensors()[name](7)
    assert where and set(where) == {7} and len(calls) >= 1


def _products():
    """One call of every product, on ordinary arguments; without a result it allocates its own."""
    q, sf = on(0, FP8, M, K), words(0, M, K)
    bg, sfg = on(0, FP8, G, 2 * F, K), words(0, 2 * F, K, G)
    b, sfb = on(0, FP8, 2 * F, K), words(0, 2 * F, K)
    square = on(0, FP8, M, M), words(0, M, M)
    return {
        "fp8_gemm_nt": lambda s, **kw: api.fp8_gemm_nt(q, sf, b, sfb, stream=s, **kw),
        "fp8_gemm_nt, no workspace": lambda s, **kw: api.fp8_gemm_nt(q, sf, b, sfb, stream=s, workspace=False, **kw),
        "fp8_gemm_nt_fp32_sf": lambda s, **kw: api.fp8_gemm_nt_fp32_sf(
            q, on(0, F32, K // 128, M), b, on(0, F32, 2 * F // 128, K // 128), stream=s, **kw),
        "fp8_gemm_nn": lambda s, **kw: api.fp8_gemm_nn(*square, *square, stream=s, **kw),
        "contiguous": lambda s, **kw: api.m_grouped_fp8_gemm_nt_contiguous(q, sf, bg, sfg, on(0, I32, M), stream=s, **kw),
        "masked": lambda s, **kw: api.m_grouped_fp8_gemm_nt_masked(
            on(0, FP8, G, M, K), words(0, M, K, G), bg, sfg, on(0, I32, G), stream=s, **kw),
        "k_grouped": lambda s, **kw: api.k_grouped_fp8_gemm_tn_contiguous(
            on(0, FP8, K, M), words(0, M, K), on(0, FP8, K, M), words(0, M, K), on(0, I32, G), stream=s, **kw),
    }


@pytest.fixture
def allocations(calls, current, monkeypatch):
    """The current stream at every allocation."""
    where, inner = [], torch.empty
    monkeypatch.setattr(torch, "empty", lambda *a, **kw: where.append(torch.cuda.current_stream().cuda_stream) or
                        inner(*a, **kw))
    monkeypatch.setattr(On, "record_stream", lambda t, s: None, raising=False)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    monkeypatch.setattr(api, "get_num_sms", lambda: 1)
    monkeypatch.setattr(api, "get_tma_aligned_size", lambda x, size: (x + 3) // 4 * 4)
    monkeypatch.setattr(api, "_WORKSPACES", {})
    current.append(Side(3))
    return where


@pytest.mark.parametrize("name", _products())
def test_the_products_results_are_allocated_on_the_calls_stream(name, allocations, calls):
    _products()[name](7)
    assert allocations and set(allocations) == {7} and len(calls) == 1


def test_a_workspace_is_made_on_the_stream_that_uses_it(allocations, calls):
    """With a given result only the binding's workspace (and its zeros) is left."""
    d = on(0, BF16, M, 2 * F)
    _products()["fp8_gemm_nt"](7, d=d)
    assert allocations == [7] and len(calls) == 1
    _products()["fp8_gemm_nt"](7, d=d)
    assert len(allocations) == 1 and len(calls) == 2  # kept
