"""Workspaces and index arrays at addresses that their kernels could not use are refused on the host."""
import ctypes

import pytest

import mixture_experts_layer_21_b200 as m
from tests.test_abi import _fwd

L = m.lib()
ALIGN = 3


def _w(fmt, K=256):
    w = m.moe_weight_t(fmt, 2, 64, K, 16, 16, None)
    w.kdata, w.kscale, w.kalpha = 16, 16, 16
    return w


@pytest.mark.parametrize("kw", [dict(ws=17), dict(ws=18), dict(cu=18), dict(idx=17)])
def test_mxfp4_product(kw):
    d = dict(ws=16, cu=16, idx=16)
    d.update(kw)
    w = _w(1)
    assert L.moe_grouped_gemm_mxfp4(16, 1, 8, d["idx"], 8, ctypes.byref(w), d["cu"], 16, None, d["ws"], 256, None) == ALIGN
    assert L.moe_grouped_gemm_mxfp4_room(16, 1, 8, d["idx"], 8, ctypes.byref(w), d["cu"], 16, None, 0, d["ws"], 256,
                                         None) == ALIGN


@pytest.mark.parametrize("fmt,ws,cu", [(0, 18, 16), (0, 16, 17), (1, 20, 16), (1, 24, 16), (2, 20, 16), (2, 16, 18)])
def test_grouped_product(fmt, ws, cu):
    w = _w(fmt)
    assert L.moe_grouped_gemm(16, 8, ctypes.byref(w), cu, 16, ws, 1 << 20, None) == ALIGN


@pytest.mark.parametrize("ws,cu", [(18, 16), (16, 17)])
def test_nvfp4_product(ws, cu):
    w = _w(2)
    assert L.moe_grouped_gemm_nvfp4(16, 16, 16, 8, ctypes.byref(w), cu, 16, ws, 256, None) == ALIGN


def test_permutation_and_layer():
    assert L.moe_permute(16, 16, 4, 2, 8, 0, None, None, 0, 16, 16, 16, 16, None, 0, 18, 1 << 20, None) == ALIGN
    p, nws = _fwd()
    assert L.moe_forward(ctypes.byref(p), 24, nws, None) == ALIGN
