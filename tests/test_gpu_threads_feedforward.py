"""Several host threads in the feed-forward operators at once, each on its own
CUDA stream, with calls of one kernel that need different amounts of shared
memory: the limit belongs to the kernel, and no thread's call may lower it
under another's launch.  Every result equals the same call made alone."""
import threading

import pytest
import torch

import moe_grouped_gemm_fp8_gb300 as dg

pytestmark = pytest.mark.gpu


def _gated(k, out_format):
    """One token: the kernel's shared memory follows K."""
    g = torch.Generator().manual_seed(k)
    q, sf = dg.quantize_fp8(torch.randn(1, k, generator=g).cuda(), 1)
    qw, sw = dg.quantize_fp8(torch.randn(512, k, generator=g).cuda(), 128)
    return lambda: [t for t in dg.fp8_gated_gemm_nt(q, sf, qw, sw, out_format=out_format) if t is not None]


def _norm(rows, cols, dtype, out_format):
    """The ring's shared memory follows the rows a CTA takes and their width."""
    g = torch.Generator().manual_seed(rows + cols)
    x = torch.randn(rows, cols, generator=g).to(dtype).cuda()
    w, b = torch.randn(2, cols, generator=g).cuda()
    return lambda: [t for t in dg.layer_norm(x, w, b, out_format=out_format) if t is not None]


def _backward(rows, cols, dtype):
    g = torch.Generator().manual_seed(rows * cols)
    x, dy = (torch.randn(rows, cols, generator=g).to(dtype).cuda() for _ in range(2))
    w, b = torch.randn(2, cols, generator=g).cuda()
    r = dg.layer_norm(x, w, b)
    return lambda: list(dg.layer_norm_backward(dy, x, w, r.mean, r.rstd))


# calls of one kernel each, by the shared memory they need
CASES = {
    "one token to BF16": lambda: [_gated(k, "bf16") for k in (128, 1024, 7168, 28672)],
    "one token to 8 bits": lambda: [_gated(k, "fp8") for k in (128, 1024, 7168, 28672)],
    "norm to 8 bits": lambda: [_norm(r, c, torch.bfloat16, "fp8") for r, c in ((160, 5120), (310, 6144), (500, 7168), (160, 16384))],
    "norm": lambda: [_norm(r, c, torch.float32, "same") for r, c in ((160, 5120), (310, 4096), (500, 2048), (160, 8192))],
    "norm's backward pass": lambda: [_backward(r, c, torch.float32) for r, c in ((160, 1024), (310, 2048), (500, 1024), (160, 4096))],
}


@pytest.mark.parametrize("case", CASES)
def test_concurrent_host_threads(case):
    calls = CASES[case]()
    want = [call() for call in calls]
    torch.cuda.synchronize()
    errors = []

    def worker(t):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                for it in range(300):
                    at = (t + it) % len(calls)
                    got = calls[at]()
                    if it % 50 == 49:
                        stream.synchronize()
                        if not all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(got, want[at])):
                            errors.append("thread %d iteration %d differs" % (t, it))
        except Exception as e:  # reported below, on the test's thread
            errors.append("thread %d: %r" % (t, e))

    threads = [threading.Thread(target=worker, args=(t,)) for t in range(6)]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    assert not errors, errors
    assert dg.get_device_error()[0] == 0
