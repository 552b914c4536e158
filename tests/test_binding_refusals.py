"""What the binding refuses of tensors on the GPU, by the message that names the reason: types, shapes, strides,
devices and sizes, for the routing, the norm, the quantiser and the MXFP4 product."""
import pytest
import torch

import mixture_experts_layer_21_b200 as m

pytestmark = pytest.mark.gpu
u8, i32, f32, bf16 = torch.uint8, torch.int32, torch.float32, torch.bfloat16


def _z(*shape, dtype=f32, device="cuda"):
    return torch.zeros(*shape, dtype=dtype, device=device)


@pytest.mark.parametrize("kw,message", [
    (dict(logits=_z(4, 8, device="cpu")), "current CUDA device"),
    (dict(logits=lambda: _z(4, 8, dtype=torch.float16)), "logits: need bf16 or fp32"),
    (dict(logits=lambda: _z(8, 4).t()), "logits: need contiguous rows"),
    (dict(logits=lambda: _z(1, 8).expand(4, 8)), "logits: need contiguous rows"),
    (dict(bias=lambda: _z(7)), "bias: need"), (dict(bias=lambda: _z(8, dtype=bf16)), "bias: need"),
    (dict(bias=lambda: _z(16)[::2]), "bias: need a contiguous"), (dict(bias=_z(8, device="cpu")), "bias: need"),
    (dict(ids=lambda: _z(4, 2, dtype=torch.int64)), "ids: need"), (dict(ids=lambda: _z(4, 3, dtype=i32)), "ids: need"),
    (dict(ids=lambda: _z(2, 4, dtype=i32).t()), "ids: need a contiguous"), (dict(w=lambda: _z(4, 2, dtype=bf16)), "w: need"),
    (dict(w=lambda: _z(4, 4)[:, ::2]), "w: need a contiguous")])
def test_route_scored(kw, message):
    kw = {k: v() if callable(v) else v for k, v in kw.items()}
    with pytest.raises(ValueError, match=message):
        m.moe_route_scored(kw.pop("logits", _z(4, 8)), 2, **kw)


@pytest.mark.parametrize("kw,status", [(dict(topk=9), "INVALID"), (dict(topk=0), "INVALID"), (dict(n_group=3), "INVALID"),
                                       (dict(n_group=4, topk_group=5), "INVALID"),
                                       (dict(routed_scaling_factor=0.0), "INVALID")])
def test_route_scored_by_the_library(kw, status):
    kw = dict(topk=2) | kw
    with pytest.raises(m.MoEError, match=status):
        m.moe_route_scored(_z(4, 8), kw.pop("topk"), **kw)


@pytest.mark.parametrize("x,out,message", [
    (lambda: _z(4, 64, dtype=torch.float16), {}, "x: need bf16 or fp32"),
    (lambda: _z(64, 4, dtype=bf16).t(), {}, "x: need contiguous rows"),
    (lambda: _z(4, 64, dtype=bf16, device="cpu"), {}, "current CUDA device"),
    (lambda: _z(4, 64, dtype=bf16), dict(codes=lambda: _z(4, 64, dtype=u8)), "codes: need"),
    (lambda: _z(4, 64, dtype=bf16), dict(scales=lambda: _z(4, 1, dtype=u8)), "scales: need"),
    (lambda: _z(4, 64, dtype=bf16), dict(deq=lambda: _z(4, 64)), "deq: need"),
    (lambda: _z(4, 64, dtype=bf16), dict(deq=lambda: _z(64, 4, dtype=bf16).t()), "deq: need a contiguous")])
def test_quantize_mxfp4(x, out, message):
    with pytest.raises(ValueError, match=message):
        m.moe_quantize_mxfp4(x(), deq=True, out={k: v() for k, v in out.items()})


@pytest.mark.parametrize("x", [lambda: _z(4, 48, dtype=bf16), lambda: _z(4, 72, dtype=bf16)[:, 8:].narrow(1, 0, 40),
                               lambda: _z(4, 66, dtype=bf16)[:, :64], lambda: _z(4, 68)[:, 4:]])
def test_quantize_mxfp4_sizes_and_strides(x):
    with pytest.raises(m.MoEError, match="ALIGNMENT"):
        m.moe_quantize_mxfp4(x())


@pytest.mark.parametrize("kw,message", [
    (dict(residual=lambda: _z(4, 64)), "residual: need"), (dict(residual=lambda: _z(4, 32, dtype=bf16)), "residual: need"),
    (dict(weight=lambda: _z(64, dtype=torch.float16)), "weight: need bf16 or fp32"),
    (dict(weight=lambda: _z(128, dtype=bf16)[::2]), "weight: need a contiguous"),
    (dict(out=dict(y=lambda: _z(4, 64))), "y: need"), (dict(quant="mxfp8", out=dict(codes=lambda: _z(4, 32, dtype=u8))), "codes: need"),
    (dict(quant="mxfp4", out=dict(codes=lambda: _z(4, 64, dtype=u8))), "codes: need"), (dict(deq=True), "deq needs quant")])
def test_add_rmsnorm(kw, message):
    kw = {k: {n: t() for n, t in v.items()} if isinstance(v, dict) else v() if callable(v) else v for k, v in kw.items()}
    with pytest.raises(ValueError, match=message):
        m.moe_add_rmsnorm(_z(4, 64, dtype=bf16), **kw)


def _product(**kw):
    w = m.Weight("mxfp4", _z(2, 64, 32, dtype=u8), _z(2, 64, 2, dtype=u8))
    d = dict(a_codes=_z(6, 32, dtype=u8), a_scales=_z(6, 2, dtype=u8), w=w, cu_seqlens=torch.tensor([2, 6], dtype=i32, device="cuda"))
    d.update(kw)
    if d.pop("prepare", True) and d["w"].fmt != "bf16":
        m.moe_prepare_weights(d["w"])
    return m.moe_grouped_gemm_mxfp4(**d)


@pytest.mark.parametrize("kw,message", [
    (dict(a_codes=_z(6, 32, dtype=u8, device="cpu")), "current CUDA device"),
    (dict(a_codes=lambda: _z(6, 64, dtype=u8)), "a_codes: need"), (dict(a_codes=lambda: _z(6, 32, dtype=torch.int8)), "a_codes: need"),
    (dict(a_codes=lambda: _z(6, 64, dtype=u8)[:, :32]), "a_codes: need a contiguous"),
    (dict(a_scales=lambda: _z(5, 2, dtype=u8)), "a_scales: need"), (dict(cu_seqlens=lambda: _z(3, dtype=i32)), "cu_seqlens: need"),
    (dict(cu_seqlens=lambda: _z(2, dtype=torch.int64)), "cu_seqlens: need"),
    (dict(row_idx=lambda: _z(6, dtype=torch.int64)), "row_idx: need"), (dict(row_idx=lambda: _z(12, dtype=i32)[::2]), "row_idx: need a contiguous"),
    (dict(out=lambda: _z(6, 64)), "out: need"), (dict(out=lambda: _z(5, 64, dtype=bf16)), "out: need"),
    (dict(ws=_z(256, dtype=u8, device="cpu")), "ws: need")])
def test_product(kw, message):
    kw = {k: v() if callable(v) else v for k, v in kw.items()}
    with pytest.raises(ValueError, match=message):
        _product(**kw)


def test_product_by_the_library():
    with pytest.raises(m.MoEError, match="NOT_PREPARED"):
        _product(prepare=False)
    with pytest.raises(m.MoEError, match="UNSUPPORTED"):
        _product(w=m.Weight("bf16", _z(2, 64, 64, dtype=bf16)))
    with pytest.raises(m.MoEError, match="WORKSPACE_TOO_SMALL"):
        _product(ws=_z(255, dtype=u8))
    with pytest.raises(m.MoEError, match="ALIGNMENT"):
        _product(ws=_z(300, dtype=u8)[1:])
    assert _product().shape == (6, 64) and m.moe_get_device_error() == 0
