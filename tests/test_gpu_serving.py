"""The serving operators together, as a decode step runs them: norm, an 8-bit
integer projection, a mixture-of-experts layer on its result; in graphs, by
programmatic launch, from several threads, under the debug library."""
import os
import subprocess
import sys
import threading

import pytest
import torch

import moe_grouped_gemm_fp8_gb300 as dg
from moe_grouped_gemm_fp8_gb300 import block

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


class Step:
    """x + W8 norm(x), then the experts on its norm with the residual."""

    def __init__(self, t, d=512, f=256, e=6, k=2, seed=0):
        g = torch.Generator().manual_seed(seed + t)
        r = lambda *s: torch.randn(*s, generator=g).cuda()  # noqa: E731
        self.k, self.x = k, r(t, d).to(BF16)
        self.weight = r(d, d) * d ** -0.5
        self.w8, self.s8 = dg.quantize_int8(self.weight)
        self.norm, self.bias = 1 + 0.1 * r(d), 0.1 * r(d)
        self.up, self.down = r(e, 2 * f, d) * d ** -0.5, r(e, d, f) * f ** -0.5
        self.experts = block.GatedExperts(self.up, self.down)
        self.router = r(e, d) * d ** -0.5

    def __call__(self):
        n = dg.layer_norm(self.x, self.norm, self.bias)
        q, s = dg.quantize_int8(n.y)
        a = dg.int8_gemm_nt(q, s, self.w8, self.s8, c=self.x)
        n2 = dg.layer_norm(a, self.norm, self.bias)
        r = self.experts.few_tokens(n2.y, self.router, self.k, c=a)
        return [n.y, q, s, a, n2.y, *r]

    def plain(self):
        """The same in 64 bits, from the products' real weights and codes' definition; the choice of experts as made."""
        n, q, s, a, n2, y, chosen, weights = self()
        ln = torch.nn.functional.layer_norm
        d = self.x.shape[1]
        w = self.norm.double(), self.bias.double()
        a64 = self.x.double() + ln(self.x.double(), (d,), *w) @ self.weight.double().t()
        n64 = ln(a64, (d,), *w)
        up, down = (dg.dequantize_fp8(v.q, v.sf, torch.float32).double() for v in (self.experts.up, self.experts.down))
        y64 = a64.clone()
        for t in range(len(a64)):
            for j in range(self.k):
                e = int(chosen[t, j])
                gu = up[e] @ n64[t]
                f = len(gu) // 2
                y64[t] += weights[t, j].double() * (down[e] @ (gu[:f] * torch.sigmoid(gu[:f]) * gu[f:]))
        return a, a64, y, y64


@pytest.mark.parametrize("t", [1, 7, 64])
def test_step_is_near_the_formulas(t):
    a, a64, y, y64 = Step(t).plain()
    # roundings of the step: BF16 at the norm, the projection and y, 8 bits (half of 1/127 of the largest) at both
    # operands of the projection: of the order of 2^-8 to 2^-7 of the results, far below a wrong term
    for got, want in ((a, a64), (y, y64)):
        assert float((got.double() - want).norm() / want.norm()) <= 2.0 ** -5
    assert dg.get_device_error()[0] == 0


@pytest.mark.parametrize("graph", [False, True])
@pytest.mark.parametrize("t", [1, 9, 40])
def test_programmatic_launch_gives_the_same_bits(t, graph):
    step = Step(t)
    dg.set_pdl(False)
    want = [v.clone() for v in step()]
    torch.cuda.synchronize()
    try:
        dg.set_pdl(True)
        if graph:
            s = torch.cuda.Stream()
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                step()
            torch.cuda.current_stream().wait_stream(s)
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                got = step()
        for _ in range(8):
            if graph:
                for v in got:
                    v.zero_()
                g.replay()
            else:
                got = step()
            torch.cuda.synchronize()
            for i, (a, b) in enumerate(zip(got, want)):
                assert torch.equal(a, b), i
        assert dg.get_device_error()[0] == 0
    finally:
        dg.set_pdl(False)


def test_concurrent_host_threads():
    """Calls of one kernel that need different amounts of shared memory and registers, and cooperative launches, from
    several threads on streams of their own: each result equals the same call made alone."""
    steps = [Step(t, d=d, f=f, seed=s) for s, (t, d, f) in enumerate([(1, 512, 256), (12, 1024, 512), (30, 256, 128), (64, 512, 128)])]
    want = [[v.clone() for v in s()] for s in steps]
    torch.cuda.synchronize()
    errors = []

    def worker(i):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                for it in range(60):
                    at = (i + it) % len(steps)
                    got = steps[at]()
                    if it % 10 == 9:
                        stream.synchronize()
                        if not all(torch.equal(a, b) for a, b in zip(got, want[at])):
                            errors.append("thread %d iteration %d differs" % (i, it))
        except Exception as e:  # reported below, on the test's thread
            errors.append("thread %d: %r" % (i, e))

    threads = [threading.Thread(target=worker, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    assert dg.get_device_error()[0] == 0


def test_padded_graph_follows_its_count():
    """A captured step whose token count changes between replays."""
    t, d, f, e, k = 16, 384, 256, 5, 2
    g = torch.Generator().manual_seed(3)
    r = lambda *s: torch.randn(*s, generator=g).cuda()  # noqa: E731
    net = block.GatedExperts(r(e, 2 * f, d) * d ** -0.5, r(e, d, f) * f ** -0.5)
    x, router, n = r(t, d).to(BF16), r(e, d), torch.tensor([t], dtype=torch.int32, device="cuda")
    y = torch.zeros(t, d, dtype=BF16, device="cuda")
    net.few_tokens(x, router, k, c=x, num_tokens=n, d=y)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = net.few_tokens(x, router, k, c=x, num_tokens=n, d=y)
    for live in (16, 3, 0, 9, 1):
        x.copy_(r(t, d))
        n.fill_(live)
        y.fill_(5.0)
        graph.replay()
        torch.cuda.synchronize()
        assert (y[live:] == 5.0).all() and (out.experts[live:] == -1).all()
        if live:
            alone = net.few_tokens(x[:live].contiguous(), router, k, c=x[:live].contiguous())
            assert torch.equal(out.experts[:live], alone.experts)
            # (another batch size may split the sums elsewhere)
            assert ((y[:live].float() - alone.y.float()).abs() <= 2.0 ** -7 * alone.y.float().abs() + 2.0 ** -8).all()
    assert dg.get_device_error()[0] == 0


SUITES = ["tests/test_gpu_moe_few_tokens.py", "tests/test_gpu_int8.py"]


def test_the_suites_pass_under_the_debug_library():
    if os.environ.get("DG_DEBUG_LIBRARY", "0") not in ("", "0"):
        pytest.skip("already running under the debug library")
    from moe_grouped_gemm_fp8_gb300 import build
    build.build(debug=True)
    env = dict(os.environ, DG_DEBUG_LIBRARY="1")
    r = subprocess.run([sys.executable, "-m", "pytest", *SUITES, "-m", "gpu", "-x", "-q", "-p", "no:cacheprovider"],
                       env=env, cwd=ROOT, timeout=1800, capture_output=True, text=True)
    assert r.returncode == 0, r.stdout[-6000:] + r.stderr[-3000:]
