"""Programmatic dependent launch along the feed-forward block's own chains:
every kernel reads what the one before it wrote, so its reads have to come
after its wait.  Eagerly and in a CUDA graph, the bits of the same chain
without it."""
import pytest
import torch

import moe_grouped_gemm_fp8_gb300 as dg
from moe_grouped_gemm_fp8_gb300 import block

pytestmark = pytest.mark.gpu


def _dense(m, d, f):
    gen = torch.Generator().manual_seed(m + f)
    r = lambda *s: torch.randn(*s, generator=gen).cuda()  # noqa: E731
    net = block.GatedFeedForward(r(2 * f, d) * d ** -0.5, r(d, f) * f ** -0.5, 1 + 0.1 * r(d), 0.1 * r(d))
    x, dy = r(m, d).to(torch.bfloat16), r(m, d).to(torch.bfloat16)

    def chain():
        y, saved = net.forward(x, training=True)
        return [y, *saved[1:], *net.backward(dy, saved)]
    return chain


def _experts(d, f):
    gen = torch.Generator().manual_seed(d + f)
    r = lambda *s: torch.randn(*s, generator=gen).cuda()  # noqa: E731
    net = block.GatedExperts(r(2, 2 * f, d) * d ** -0.5, r(2, d, f) * f ** -0.5)
    m = 512
    x, dy = r(m, d), r(m, d).to(torch.bfloat16)
    index = torch.tensor([0] * 256 + [1] * 256, dtype=torch.int32).cuda()
    ks = torch.tensor([256, 256], dtype=torch.int32).cuda()
    counts = torch.tensor([200, 33], dtype=torch.int32).cuda()

    def chain():
        q, sf = dg.quantize_fp8(x, 1)
        y, kept = net.forward(q, sf, index, training=True)
        qm, sfm = dg.quantize_fp8(x.view(2, 256, d), 1)
        decoded = net.decode(qm, sfm, counts)
        return [y, decoded[0, :200], decoded[1, :33], *net.backward(dy, q, sf, kept, index, ks)]
    return chain


@pytest.mark.parametrize("graph", [False, True])
@pytest.mark.parametrize("make", [lambda: _dense(1, 512, 256), lambda: _dense(3, 1024, 2048), lambda: _dense(64, 512, 640),
                                  lambda: _dense(700, 1024, 1152), lambda: _experts(512, 384)],
                         ids=["one token", "three tokens", "few tokens", "many tokens", "experts"])
def test_chain_matches_serial(make, graph):
    chain = make()
    dg.set_pdl(False)
    want = [t.clone() for t in chain()]
    torch.cuda.synchronize()
    try:
        dg.set_pdl(True)
        if graph:
            s = torch.cuda.Stream()
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                chain()
            torch.cuda.current_stream().wait_stream(s)
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                got = chain()
        for _ in range(5):
            if graph:
                for t in got:
                    t.view(torch.uint8).zero_()
                g.replay()
            else:
                got = chain()
            torch.cuda.synchronize()
            for i, (a, b) in enumerate(zip(got, want)):
                assert torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8)), i
        assert dg.get_device_error()[0] == 0
    finally:
        dg.set_pdl(False)
