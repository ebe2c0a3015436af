"""CPU checks of the serving binding: refusals, devices and explicit streams,
with stand-ins for CUDA tensors and a library that must not be called."""
import pytest
import torch

from moe_grouped_gemm_fp8_gb300 import _lib, api, feedforward, serving
from test_binding_feedforward import On, on, words

BF16, F32, I8, I32, FP8 = torch.bfloat16, torch.float32, torch.int8, torch.int32, torch.float8_e4m3fn
T, D, F, E, K = 3, 256, 128, 4, 2


def view(t):
    """A view of a stand-in as one itself."""
    return t.as_subclass(On)


@pytest.fixture
def calls(monkeypatch):
    """The library's entry points that were reached; cuda:0 is current."""
    seen = []

    class Lib:
        def __getattr__(self, name):
            return lambda *a: seen.append((name, a)) or 0

    monkeypatch.setattr(_lib, "lib", Lib)
    for module in (feedforward, serving):
        monkeypatch.setattr(module, "_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(api, "_raw_stream", lambda dev: 0)
    monkeypatch.setattr(feedforward, "_raw_stream", lambda dev: 0)
    monkeypatch.setattr(serving, "_moe_workspace", lambda *a: 16)
    real = torch.empty
    monkeypatch.setattr(torch, "empty", lambda *a, device=None, **kw: real(*a, **kw).as_subclass(On))
    return seen


def args(**kw):
    a = dict(x=on(0, BF16, T, D), router=on(0, F32, E, D), up=on(0, FP8, E, 2 * F, D), up_sf=words(0, 2 * F, D, E),
             down=on(0, FP8, E, D, F), down_sf=words(0, D, F, E), top_k=K)
    a.update(kw)
    return a


def test_the_usual_call_reaches_the_library(calls):
    r = serving.fp8_moe_few_tokens(**args())
    assert [n for n, _ in calls] == ["dg_fp8_moe_few_tokens"]
    assert r.y.shape == (T, D) and r.experts.shape == (T, K) and r.weights.dtype == F32


@pytest.mark.parametrize("kw,error", [
    (dict(x=on(0, F32, T, D)), TypeError),
    (dict(x=on(0, BF16, T, 2 * D)), ValueError),
    (dict(router=on(0, torch.float16, E, D)), TypeError),
    (dict(router=on(0, F32, E + 1, D)), ValueError),
    (dict(up=on(0, FP8, E, 2 * F + 1, D)), ValueError),
    (dict(down=on(0, FP8, E, F, D)), ValueError),
    (dict(up_sf=words(0, F, D, E)), ValueError),
    (dict(down_sf=on(0, F32, E, 1, D)), TypeError),
    (dict(router_bias=on(0, F32, E)), ValueError),                       # with softmax
    (dict(router_bias=on(0, F32, E + 1), score="sigmoid"), ValueError),
    (dict(score="max"), ValueError),
    (dict(activation="relu"), ValueError),
    (dict(c=on(0, BF16, T, D + 1)), ValueError),
    (dict(d=on(0, F32, T, D)), TypeError),
    (dict(num_tokens=on(0, torch.int64, 1)), TypeError),
    (dict(num_tokens=on(0, I32, 2)), ValueError),
    (dict(x=on(0, BF16, 65, D)), ValueError),
])
def test_moe_refusals(calls, kw, error):
    with pytest.raises(error):
        serving.fp8_moe_few_tokens(**args(**kw))
    assert not calls


@pytest.mark.parametrize("name,make", [
    ("x", lambda: on(1, BF16, T, D)), ("router", lambda: on(1, F32, E, D)), ("up", lambda: on(1, FP8, E, 2 * F, D)),
    ("up_sf", lambda: words(1, 2 * F, D, E)), ("down", lambda: on(1, FP8, E, D, F)), ("down_sf", lambda: words(1, D, F, E)),
    ("c", lambda: on(1, BF16, T, D)), ("d", lambda: on(1, BF16, T, D)), ("num_tokens", lambda: on(1, I32, 1)),
])
def test_a_tensor_of_another_device_is_refused(calls, name, make):
    with pytest.raises(ValueError, match="current CUDA device is cuda:0"):
        serving.fp8_moe_few_tokens(**args(**{name: make()}))
    assert not calls


def gemm(**kw):
    a = dict(a=on(0, I8, 5, 32), sa=on(0, F32, 5), b=on(0, I8, 7, 32), sb=on(0, F32, 7))
    a.update(kw)
    return serving.int8_gemm_nt(**a)


def test_int8_refusals(calls):
    assert gemm().shape == (5, 7) and gemm(out_dtype=torch.float16).dtype == torch.float16
    n = len(calls)
    for kw, error in [(dict(a=on(0, torch.uint8, 5, 32)), TypeError), (dict(b=on(0, I8, 7, 48)), ValueError),
                      (dict(sa=on(0, F32, 4)), ValueError), (dict(sb=on(0, BF16, 7)), TypeError),
                      (dict(out_dtype=F32), TypeError), (dict(c=on(0, torch.float16, 5, 7)), TypeError),
                      (dict(c=on(0, BF16, 5, 8)), ValueError), (dict(d=on(0, BF16, 7, 5)), ValueError),
                      (dict(a=view(on(0, I8, 32, 5).t())), ValueError), (dict(b=on(1, I8, 7, 32)), ValueError),
                      (dict(sa=on(1, F32, 5)), ValueError)]:
        with pytest.raises(error):
            gemm(**kw)
    assert len(calls) == n


def test_quantise_refusals(calls):
    q, s = serving.quantize_int8(on(0, BF16, 4, 10))
    assert q.dtype == I8 and q.shape == (4, 10) and s.shape == (4,)
    n = len(calls)
    good = (on(0, I8, 4, 10), on(0, F32, 4))
    for x, out, error in [(on(0, torch.float64, 4, 10), None, TypeError), (on(0, BF16, 4, 10, 2), None, ValueError),
                          (on(0, BF16, 4, 0), None, ValueError), (view(on(0, BF16, 10, 4).t()), None, ValueError),
                          (on(1, BF16, 4, 10), None, ValueError), (on(0, BF16, 4, 10), (good[0], on(0, F32, 5)), ValueError),
                          (on(0, BF16, 4, 10), (on(0, torch.uint8, 4, 10), good[1]), TypeError),
                          (on(0, BF16, 4, 10), (on(1, I8, 4, 10), good[1]), ValueError)]:
        with pytest.raises(error):
            serving.quantize_int8(x, out=out)
    assert len(calls) == n


def test_rows_that_overlap_are_refused(calls):
    x = view(on(0, BF16, 4, 10).as_strided((4, 10), (5, 1)))
    with pytest.raises(ValueError, match="overlap"):
        serving.quantize_int8(x)
    assert not calls


@pytest.mark.parametrize("call", [lambda s: serving.fp8_moe_few_tokens(**args(), stream=s), lambda s: gemm(stream=s),
                                  lambda s: serving.quantize_int8(on(0, BF16, 4, 10), stream=s)])
def test_an_explicit_stream_is_current_while_memory_is_made(calls, monkeypatch, call):
    class Side:
        device = torch.device("cuda", 0)

    side, here, current = Side(), object(), []
    monkeypatch.setattr(torch.cuda, "Stream", Side)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: here)
    monkeypatch.setattr(torch.cuda, "set_stream", lambda s: current.append(s))
    made = []
    inner = torch.empty
    monkeypatch.setattr(torch, "empty", lambda *a, **kw: made.append(current[-1]) or inner(*a, **kw))
    kept = []
    monkeypatch.setattr(On, "record_stream", lambda t, s: kept.append(s), raising=False)
    call(side)
    assert made and all(s is side for s in made)
    assert current[-1] is here and kept and all(s is here for s in kept)
