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
