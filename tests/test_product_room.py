"""Memory for the rows that the MXFP4 x MXFP4 product gathers first: its size is checked by the launch that
uses it, and a pointer without a size is refused."""
import ctypes

import pytest
import torch

import mixture_experts_layer_21_b200 as m
from tests.test_mxfp4 import _case, _product, _w

L = m.lib()
INVALID, ALIGN, WS_SMALL = 1, 3, 4


def _room(w, rows, nbytes, M=7, idx=16, a_rows=8):
    return L.moe_grouped_gemm_mxfp4_room(16, 1, a_rows, idx, M, ctypes.byref(w), 16, 16, rows, nbytes, 16, 256, None)


@pytest.mark.parametrize("env", [("MOE_GEMM_PAIRS", "1"), ("MOE_TOKEN_TILE", "64")])
def test_room_one_byte_short_is_refused(env, monkeypatch):
    monkeypatch.setenv("MOE_GEMM_PAIRS", "0")
    monkeypatch.setenv(*env)
    w = _w(K=96)
    need = L.moe_grouped_gemm_mxfp4_rows_size(7, ctypes.byref(w))
    assert need == 7 * 51
    assert _room(w, 16, need - 1) == WS_SMALL and _room(w, 16, 0) == WS_SMALL
    assert _room(w, 8, need) == ALIGN
    # sized for fewer rows, and before the environment asked for more
    assert _room(w, 16, L.moe_grouped_gemm_mxfp4_rows_size(6, ctypes.byref(w))) == WS_SMALL
    monkeypatch.setenv("MOE_GEMM_PAIRS", "0")
    monkeypatch.delenv("MOE_TOKEN_TILE", raising=False)
    before = L.moe_grouped_gemm_mxfp4_rows_size(7, ctypes.byref(w))
    monkeypatch.setenv(*env)
    assert before == 0 and _room(w, 16, before) == WS_SMALL


def test_room_without_a_size_is_refused():
    w = _w(K=96)
    call = lambda rows: L.moe_grouped_gemm_mxfp4(16, 1, 8, 16, 7, ctypes.byref(w), 16, 16, rows, 16, 256, None)
    assert call(16) == INVALID and call(8) == ALIGN


@pytest.mark.gpu
@pytest.mark.parametrize("pairs", ["0", "1"])
def test_room_of_the_size_asked_for_is_not_passed(pairs, monkeypatch):
    """The bytes behind it stay, and one byte fewer is refused with nothing written."""
    monkeypatch.setenv("MOE_GEMM_PAIRS", pairs)
    monkeypatch.setenv("MOE_TOKEN_TILE", "128")
    case = _case([150, 0, 61], 264, 352, True, seed=17, T=90, pad=2)
    want, _ = _product(case)
    ac, asc, wc, wsc, idx, al, cu, M = [t.cuda() if torch.is_tensor(t) else t for t in case]
    w = m.moe_prepare_weights(m.Weight("mxfp4", wc, wsc))
    n = L.moe_grouped_gemm_mxfp4_rows_size(M, w.desc_ref)
    assert n == M * (352 // 2 + 352 // 32)
    room = torch.full((n + 64,), 77, dtype=torch.uint8, device="cuda")
    out = torch.full((M, 264), 5.0, dtype=torch.bfloat16, device="cuda")
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    call = lambda size: L.moe_grouped_gemm_mxfp4_room(ac.data_ptr(), asc.data_ptr(), 90, idx.data_ptr(), M, w.desc_ref,
                                                      cu.data_ptr(), out.data_ptr(), room.data_ptr(), size, ws.data_ptr(),
                                                      256, torch.cuda.current_stream().cuda_stream)
    assert call(n - 1) == WS_SMALL
    torch.cuda.synchronize()
    assert bool((out == 5).all()) and bool((room == 77).all())
    assert call(n) == 0
    torch.cuda.synchronize()
    assert torch.equal(out, want) and bool((room[n:] == 77).all()) and m.moe_get_device_error(ws) == 0
