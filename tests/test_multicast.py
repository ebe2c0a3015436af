"""TMA multicast belongs to processes with one GPU and no other ranks."""
import os
import re

import pytest

import moe_grouped_gemm_fp8_gb300 as dg
from moe_grouped_gemm_fp8_gb300 import workloads

SHAPE = (4096, 7168, 16384, False, 152)  # 256-row tiles, in clusters on one GPU
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(autouse=True)
def plain(monkeypatch):
    for k in ("DG_BLOCK_M", "DG_BLOCK_N", "DG_SPLIT_K", "DG_CTA_PAIR", "DG_STREAM_K", "DG_MULTICAST", "DG_TALL_EPI8",
              "WORLD_SIZE"):
        monkeypatch.delenv(k, raising=False)
    from moe_grouped_gemm_fp8_gb300 import build
    build.build()


def test_a_rank_of_several_never_plans_multicast(monkeypatch):
    alone = {}
    for cfg in workloads.PREFILL + workloads.DECODE:
        for has_c in (False, True):
            alone[cfg["m"], cfg["n"], cfg["k"], has_c] = dg.plan_fp8_gemm_nt_ws(cfg["m"], cfg["n"], cfg["k"], has_c, 152)
    assert any(p["multicast"] for p in alone.values())
    for world in ("2", "8"):
        monkeypatch.setenv("WORLD_SIZE", world)
        for forced in (None, "1"):
            if forced:
                monkeypatch.setenv("DG_MULTICAST", forced)
            for (m, n, k, has_c), p in alone.items():
                assert dg.plan_fp8_gemm_nt_ws(m, n, k, has_c, 152) == dict(p, multicast=False)
        monkeypatch.delenv("DG_MULTICAST")
    monkeypatch.setenv("WORLD_SIZE", "1")
    assert dg.plan_fp8_gemm_nt_ws(*SHAPE)["multicast"]


def test_every_choice_of_multicast_asks_the_same_question():
    """DG_MULTICAST is read in one place, which also counts ranks and devices;
    the two launches that can use clusters ask there."""
    host = open(os.path.join(ROOT, "moe_grouped_gemm_fp8_gb300", "csrc", "host.cu")).read()
    assert len(re.findall(r"env\(\)\.multicast", host)) == 1
    body = host[host.index("bool multicast_on()"):]
    body = body[:body.index("\n}")]
    assert "world_size" in body and "g_visible_devices" in body
    assert re.search(r"p\.multicast = [^;]*multicast_on\(\)", host)
    assert re.search(r"args\.mc = [^;]*multicast_on\(\)", host)


@pytest.mark.gpu
def test_launches_of_a_rank_take_one_cta_a_tile(monkeypatch, capfd):
    """The launches themselves, by their printed configuration; the same bits."""
    import torch
    monkeypatch.setenv("DG_PRINT_CONFIGS", "1")
    g = torch.Generator().manual_seed(0)
    q, sf = dg.quantize_fp8(torch.randn(4096, 512, generator=g).cuda(), 1)
    qb, sfb = dg.quantize_fp8(torch.randn(7168, 512, generator=g).cuda(), 128)
    qa, sfa = dg.quantize_fp8_cols(torch.randn(256, 512, generator=g).cuda())
    ks = torch.tensor([256], dtype=torch.int32).cuda()
    monkeypatch.setenv("DG_BLOCK_M", "256")
    out = {}
    for world in ("1", "2"):
        monkeypatch.setenv("WORLD_SIZE", world)
        capfd.readouterr()
        d = dg.fp8_gemm_nt(q, sf, qb, sfb)
        monkeypatch.delenv("DG_BLOCK_M")
        monkeypatch.setenv("DG_BLOCK_N", "256")
        w = dg.k_grouped_fp8_gemm_tn_contiguous(qa, sfa, qa, sfa, ks)
        monkeypatch.delenv("DG_BLOCK_N")
        monkeypatch.setenv("DG_BLOCK_M", "256")
        printed = [line for line in capfd.readouterr().err.splitlines() if "fp8_gemm" in line]
        assert len(printed) == 2, printed
        assert all(("multicast" in line) == (world == "1") for line in printed), printed
        out[world] = d, w
    assert torch.equal(out["1"][0], out["2"][0]) and torch.equal(out["1"][1], out["2"][1])
