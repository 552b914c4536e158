"""What the MXFP4 x MXFP4 and NVFP4 products find when they are given no workspace: it is in the device's own
error word, after the call, on any stream and from a captured graph."""
import pytest
import torch

import mixture_experts_layer_21_b200 as m
from tests.test_mxfp4 import _case

pytestmark = pytest.mark.gpu
DEVICE, TIMEOUT = 6, 7


def _operands(lens, K=320, bad=True):
    ac, asc, wc, wsc, idx, _, cu, M = _case(lens, 128, K, True, seed=4, T=30)
    if bad:
        idx[1] = 30
    w = m.moe_prepare_weights(m.Weight("mxfp4", wc.cuda(), wsc.cuda()))
    return ac.cuda(), asc.cuda(), w, cu.cuda(), idx.cuda()


@pytest.mark.parametrize("lens", [[9, 20], [140, 250]])
@pytest.mark.parametrize("side", [False, True])
def test_a_bad_row_index_is_seen(lens, side):
    a = _operands(lens)
    torch.cuda.synchronize()
    m.moe_get_device_error()
    st = torch.cuda.Stream() if side else None
    got = m.moe_grouped_gemm_mxfp4(*a, stream=st)
    junk = [torch.zeros(256, dtype=torch.uint8, device="cuda") for _ in range(64)]  # blocks freed by the call, if any
    assert m.moe_get_device_error(stream=st) == DEVICE
    assert m.moe_get_device_error(stream=st) == 0      # read once
    torch.cuda.synchronize()
    assert not bool(got[1].any()) and not any(bool(j.any()) for j in junk)
    a[4][1] = 3
    m.moe_grouped_gemm_mxfp4(*a)
    assert m.moe_get_device_error() == 0


def test_from_a_captured_graph():
    a = _operands([9, 20], bad=False)
    m.moe_grouped_gemm_mxfp4(*a)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        m.moe_grouped_gemm_mxfp4(*a)
    for bad, want in ((2, 0), (30, DEVICE), (5, 0)):
        a[4][1] = bad
        g.replay()
        assert m.moe_get_device_error() == want


def test_a_wait_that_ran_out_is_seen(monkeypatch):
    a = _operands([200, 90], K=32768, bad=False)
    monkeypatch.setenv("MOE_WAIT_LIMIT_CYCLES", "1")
    m.moe_grouped_gemm_mxfp4(*a)
    assert m.moe_get_device_error() == TIMEOUT


def test_nvfp4_product():
    g = torch.Generator().manual_seed(2)
    w = m.moe_prepare_weights(m.Weight("nvfp4", torch.randint(0, 256, (2, 64, 128), generator=g, dtype=torch.uint8).cuda(),
                                       torch.full((2, 64, 16), 0x38, dtype=torch.uint8, device="cuda"),
                                       torch.ones(2, device="cuda")))
    q, sb, s, _ = m.moe_quantize_nvfp4(torch.randn(20, 256, device="cuda").bfloat16(), deq=False)
    m.moe_grouped_gemm_nvfp4(q, sb, s, w, torch.tensor([15, 99], dtype=torch.int32, device="cuda"))
    assert m.moe_get_device_error() == DEVICE
    m.moe_grouped_gemm_nvfp4(q, sb, s, w, torch.tensor([15, 20], dtype=torch.int32, device="cuda"))
    assert m.moe_get_device_error() == 0
