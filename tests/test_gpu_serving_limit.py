"""A limit of the SMs to use is kept by the products of the serving operators. The profiler that reads the launches' grids
runs in a process of its own."""
import json
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.mark.parametrize("sms", [1, 9, 40, 151])
def test_a_limit_of_the_sms_is_kept(sms, tmp_path):
    r = subprocess.run([sys.executable, os.path.abspath(__file__), str(sms), str(tmp_path)], cwd=os.path.dirname(HERE),
                       timeout=300, capture_output=True, text=True)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-4000:]
    if "no kernels" in r.stdout:
        pytest.skip("the profiler shows no kernels here")


def main(sms, folder):
    sys.path[:0] = [os.path.dirname(HERE), HERE]
    import torch
    from torch.profiler import ProfilerActivity, profile

    import moe_grouped_gemm_fp8_gb300 as dg
    import test_gpu_int8 as I
    import test_gpu_moe_few_tokens as M

    def grids(call):
        """(kernel's name, CTAs) of a call's launches."""
        with profile(activities=[ProfilerActivity.CUDA]) as p:
            call()
            torch.cuda.synchronize()
        path = os.path.join(folder, "trace.json")
        p.export_chrome_trace(path)
        events = [e for e in json.load(open(path))["traceEvents"] if e.get("cat") == "kernel"]
        return [(e["name"], e["args"]["grid"][0] * e["args"]["grid"][1] * e["args"]["grid"][2]) for e in events]

    calls = []
    for m, n, k in [(1, 4096, 1024), (30, 4096, 1024), (64, 4096, 1024), (64, 200, 2048), (100, 300, 2048), (300, 1000, 512),
                    (2000, 3000, 512)]:
        a, b, sa, sb = I.codes(m, k), I.codes(n, k, 1), I.scales(m), I.scales(n, 1)
        calls.append(("int8", lambda a=a, b=b, sa=sa, sb=sb: dg.int8_gemm_nt(a, sa, b, sb)))
    for t in (1, 12, 20, 64):
        w, x, r = M.weights(6, 1024, 512), M.tokens(t, 1024), M.gate(6, 1024)
        calls.append(("moe_layer", lambda x=x, r=r, w=w: dg.fp8_moe_few_tokens(x, r, *w, 2).y))
    want = [c() for _, c in calls]
    grids(calls[0][1])  # (a process's first profile may show nothing)
    if not grids(calls[0][1]):
        print("no kernels")
        return
    dg.set_num_sms(sms)
    for (name, call), y in zip(calls, want):
        launched = [(k, n) for k, n in grids(call) if name in k]
        assert len(launched) == 1 and launched[0][1] <= sms, launched
        # (sums may be split elsewhere)
        assert (call().float() - y.float()).norm() <= 2.0 ** -7 * y.float().norm()
    assert dg.get_device_error()[0] == 0


if __name__ == "__main__":
    main(int(sys.argv[1]), sys.argv[2])
