"""Segment ends that fall, leave [0, M_alloc] or repeat, in every grouped product: a segment whose end lies
before an earlier one is empty, the next begins where the longest so far ended, the error word says so, and
rows behind the last segment are zero.

The tolerance of the MXFP4 x MXFP4 product is that of tests/test_mxfp4.py. For bf16 weights the products are
exact in fp32 and the sum of K = 64 terms is within 64 * 2^-22 of the magnitudes added, before the bf16
rounding (2^-8).
"""
import numpy as np
import pytest
import torch

import mixture_experts_layer_21_b200 as m
from tests.test_mxfp4 import _case, _reference

DEVICE = 6
# ends given for 60 rows: a short step after a fall, a fall at the end, ends outside [0, 60], a fall over many
ENDS = {"step after a fall": [50, 1, 52, 60], "last falls": [10, 5, 8, 2], "outside": [-7, 20, 61, 2 ** 31 - 1],
        "all negative": [-1, -2, -3, -2 ** 31], "falls twice": [40, 3, 41, 7], "in order": [10, 10, 33, 60]}


def _clamped(ends, M):
    return np.maximum.accumulate(np.clip(ends, 0, M))


def _expected_error(ends, M):
    c = np.clip(ends, 0, M)
    return DEVICE if np.any(c != ends) or np.any(np.diff(c) < 0) else 0


def test_the_clamped_ends_never_fall():
    for ends in ENDS.values():
        c = _clamped(np.array(ends, np.int64), 60)
        assert np.all(np.diff(c) >= 0) and c.min() >= 0 and c.max() <= 60
    assert _clamped(np.array([50, 1, 52, 60]), 60).tolist() == [50, 50, 52, 60]


@pytest.mark.gpu
@pytest.mark.parametrize("ends", sorted(ENDS))
@pytest.mark.parametrize("tile", ["16", "32", "64", "128", "pairs"])
@pytest.mark.parametrize("gather", [False, True])
def test_mxfp4_product(ends, tile, gather, monkeypatch):
    monkeypatch.setenv("MOE_GEMM_PAIRS", "1" if tile == "pairs" else "0")
    if tile != "pairs":
        monkeypatch.setenv("MOE_TOKEN_TILE", tile)
    given = np.array(ENDS[ends], np.int64)
    case = list(_case([15] * 4, 136, 96, gather, seed=3))
    ac, asc, wc, wsc, idx, _, _, M = case
    w = m.moe_prepare_weights(m.Weight("mxfp4", wc.cuda(), wsc.cuda()))
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    got = m.moe_grouped_gemm_mxfp4(ac.cuda(), asc.cuda(), w, torch.from_numpy(given).int().cuda(),
                                   None if idx is None else idx.cuda(), ws=ws)
    torch.cuda.synchronize()
    assert m.moe_get_device_error(ws) == _expected_error(given, M)
    case[6] = torch.from_numpy(_clamped(given, M)).int()
    ref, slack = _reference(tuple(case))
    assert np.all(np.abs(got.double().cpu().numpy() - ref) <= slack + (np.abs(ref) + slack) * 2.0 ** -8)
    assert not bool(got[int(case[6][-1]):].any())


@pytest.mark.gpu
@pytest.mark.parametrize("ends", sorted(ENDS))
@pytest.mark.parametrize("pairs", ["0", "1"])
def test_bf16_product(ends, pairs, monkeypatch):
    monkeypatch.setenv("MOE_GEMM_PAIRS", pairs)
    given = np.array(ENDS[ends], np.int64)
    g = torch.Generator().manual_seed(4)
    a, wt = torch.randn(60, 64, generator=g).bfloat16(), torch.randn(4, 136, 64, generator=g).bfloat16()
    w = m.Weight("bf16", wt.cuda())
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    got = m.moe_grouped_gemm(a.cuda(), w, torch.from_numpy(given).int().cuda(), ws=ws)
    torch.cuda.synchronize()
    assert m.moe_get_device_error(ws) == _expected_error(given, 60)
    ref, slack = np.zeros((60, 136)), np.zeros((60, 136))
    lo = 0
    for e, hi in enumerate(_clamped(given, 60)):
        x, y = a[lo:hi].double().numpy(), wt[e].double().numpy()
        ref[lo:hi], slack[lo:hi] = x @ y.T, 64 * 2.0 ** -22 * (np.abs(x) @ np.abs(y).T)
        lo = hi
    assert np.all(np.abs(got.double().cpu().numpy() - ref) <= slack + (np.abs(ref) + slack) * 2.0 ** -8)


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("ends", sorted(ENDS))
def test_fp4_weights_on_bf16_rows_and_on_nvfp4_rows(ends, fmt):
    """The given ends and the clamped ones give the same bits."""
    given = np.array(ENDS[ends], np.int64)
    clamped = torch.from_numpy(_clamped(given, 60)).int().cuda()
    g = torch.Generator().manual_seed(5)
    N, K = 136, 256
    codes = torch.randint(0, 256, (4, N, K // 2), generator=g, dtype=torch.uint8).cuda()
    lo, hi, per = (118, 126, 32) if fmt == "mxfp4" else (0x30, 0x48, 16)
    scale = torch.randint(lo, hi, (4, N, K // per), generator=g, dtype=torch.uint8).cuda()
    w = m.moe_prepare_weights(m.Weight(fmt, codes, scale, torch.ones(4, device="cuda") if fmt == "nvfp4" else None))
    a = torch.randn(60, K, generator=g).bfloat16().cuda()
    n = m._lib.moe_grouped_gemm_workspace_size(60, w.desc_ref)
    calls = [lambda cu, ws: m.moe_grouped_gemm(a, w, cu, ws=ws)]
    if fmt == "nvfp4":
        q, sb, s, _ = m.moe_quantize_nvfp4(a, deq=False)
        calls.append(lambda cu, ws: m.moe_grouped_gemm_nvfp4(q, sb, s, w, cu, ws=ws))
    for call in calls:
        ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
        want = call(clamped, ws)
        assert m.moe_get_device_error(ws) == 0
        got = call(torch.from_numpy(given).int().cuda(), ws)
        assert m.moe_get_device_error(ws) == _expected_error(given, 60)
        assert torch.equal(got, want) and not bool(got[int(clamped[-1]):].any())


@pytest.mark.gpu
@pytest.mark.parametrize("tile", ["16", "64", "pairs"])
def test_many_segments_with_falls(tile, monkeypatch):
    """More segments than a warp has lanes, ends that fall inside and across its chunks of 32."""
    monkeypatch.setenv("MOE_GEMM_PAIRS", "1" if tile == "pairs" else "0")
    monkeypatch.setenv("MOE_TOKEN_TILE", "16" if tile == "pairs" else tile)
    lens = [5, 0, 7] * 26
    case = list(_case(lens, 72, 64, False, seed=6))
    M = case[-1]
    given = np.cumsum(lens)
    given[[3, 31, 32, 40, 63, 64, 76]] = [0, 2, 200, 1, -4, 30, M + 9]
    ac, asc, wc, wsc, M = case[0], case[1], case[2], case[3], case[7]
    w = m.moe_prepare_weights(m.Weight("mxfp4", wc.cuda(), wsc.cuda()))
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    got = m.moe_grouped_gemm_mxfp4(ac.cuda(), asc.cuda(), w, torch.from_numpy(given).int().cuda(), ws=ws)
    torch.cuda.synchronize()
    assert m.moe_get_device_error(ws) == DEVICE
    case[6] = torch.from_numpy(_clamped(given, M)).int()
    ref, slack = _reference(tuple(case))
    assert np.all(np.abs(got.double().cpu().numpy() - ref) <= slack + (np.abs(ref) + slack) * 2.0 ** -8)
