"""Residual addition and RMS norm (moe_add_rmsnorm) against the 64-bit oracle, and its refusals.

Tolerances. r is one fp32 addition and one bf16 rounding: |r| (2^-24 + 2^-8). y before its rounding
carries the fp32 sum of squares (a chain of at most 8 * 4 products and additions per thread, 5 shuffle
steps and 32 partial sums: 69 half-steps, halved by the root), root, division and two products:
at most (35 + 4 + 1) 2^-24 relative, taken as E = 48 * 2^-24; as bf16, E + 2^-8 (1 + E), plus half the
smallest subnormal. A quantised value must be what the rule gives for some y' within E of y: its
scale one of the two that amax (1 +- E) give, its code between those of y (1 - E) and y (1 + E).
"""
import ctypes

import numpy as np
import pytest
import torch

import mixture_experts_layer_21_b200 as m
from oracle import moe_oracle as O

L = m.lib()
INVALID, UNSUP, ALIGN = 1, 2, 3
E = 48 * 2.0 ** -24


def _args(**kw):
    d = dict(x=16, residual=16, weight=16, x_is_f32=0, weight_is_f32=0, T=4, H=64, x_stride=0, residual_stride=0,
             residual_out_stride=0, y_stride=0, eps=1e-6, quant=1, residual_out=16, y=16, codes=16, scales=1, deq=None)
    d.update(kw)
    return m.moe_rmsnorm_args_t(*[d[f[0]] for f in m.moe_rmsnorm_args_t._fields_])


@pytest.mark.parametrize("kw,want", [
    (dict(T=-1), INVALID), (dict(H=0), INVALID), (dict(quant=3), INVALID), (dict(quant=-1), INVALID),
    (dict(eps=0.0), INVALID), (dict(eps=float("nan")), INVALID), (dict(eps=float("inf")), INVALID),
    (dict(x_stride=56), INVALID), (dict(residual_stride=-64), INVALID), (dict(y_stride=8), INVALID),
    (dict(x=None), INVALID), (dict(codes=None), INVALID), (dict(scales=None), INVALID),
    (dict(quant=0), INVALID), (dict(quant=0, codes=None, scales=None, residual_out=None, y=None), INVALID),
    (dict(quant=0, codes=None, scales=None, deq=16), INVALID),
    (dict(H=72), ALIGN), (dict(H=60, quant=0, codes=None, scales=None), ALIGN), (dict(x_stride=68), ALIGN),
    (dict(x=8), ALIGN), (dict(residual=4), ALIGN), (dict(weight=2), ALIGN), (dict(y=24), ALIGN), (dict(codes=1), ALIGN),
    (dict(deq=8), ALIGN), (dict(H=32800), UNSUP)])
def test_refuses(kw, want):
    assert L.moe_add_rmsnorm(ctypes.byref(_args(**kw)), None) == want


def test_no_rows_is_a_no_op_and_null_args_are_refused():
    assert L.moe_add_rmsnorm(ctypes.byref(_args(T=0, x=None)), None) == 0
    assert L.moe_add_rmsnorm(None, None) == INVALID


def test_binding_refuses_cpu_tensors():
    with pytest.raises((ValueError, RuntimeError, AssertionError)):
        m.moe_add_rmsnorm(torch.zeros(2, 64, dtype=torch.bfloat16))


def _check_rows(got, ref, extra):
    got = got.double().cpu().numpy()
    assert np.all(np.abs(got - ref) <= np.abs(ref) * (extra + 2.0 ** -8 * (1 + extra)) + 2.0 ** -134)


def _check_quant(r, y, quant):
    T, H = y.shape
    emax = 8 if quant == "mxfp8" else 2
    enc = O.e4m3_encode if quant == "mxfp8" else O.e2m1_encode
    dec = O.e4m3_decode if quant == "mxfp8" else O.e2m1_decode
    scales = r["scales"].cpu().numpy().astype(np.int64)
    amax = np.abs(y).reshape(T, H // 32, 32).max(axis=2)
    lo, hi = (O.mx_scale_exponent(amax * f, emax) + 127 for f in (1 - E, 1 + E))
    assert np.all((scales >= lo) & (scales <= hi))
    p = np.repeat(np.ldexp(1.0, scales - 127), 32, axis=1)
    codes = r["codes"].cpu().numpy() if quant == "mxfp8" else O.unpack_e2m1(r["codes"].cpu().numpy())
    v = dec(codes)
    a, b = dec(enc(y * (1 - E) / p)), dec(enc(y * (1 + E) / p))
    assert np.all((v >= np.minimum(a, b)) & (v <= np.maximum(a, b)))
    if r["deq"] is not None:
        assert np.array_equal(r["deq"].double().cpu().numpy(), v * p)


def _inputs(T, H, f32, res, wt, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, H, generator=g) * 3
    x = x if f32 else x.bfloat16()
    big = torch.where(torch.rand(H, generator=g) < 0.02, 30.0, 1.0)
    r = (torch.randn(T, H, generator=g) * 2 * big).bfloat16() if res else None
    w = 1 + 0.3 * torch.randn(H, generator=g)
    return x, r, None if wt is None else w if wt == "f32" else w.bfloat16()


def _run(T, H, f32, res, wt, quant, deq=False, seed=1, **kw):
    x, r, w = _inputs(T, H, f32, res, wt, seed)
    c = lambda t: None if t is None else t.cuda()
    got = m.moe_add_rmsnorm(c(x), c(w), c(r), 1e-5, quant, deq=deq, **kw)
    torch.cuda.synchronize()
    n = lambda t: None if t is None else t.double().numpy()
    rr, y = O.add_rmsnorm(n(x), n(r), n(w), 1e-5)
    if res:
        _check_rows(got["residual"], rr, 2.0 ** -24)
    if got["y"] is not None:
        _check_rows(got["y"], y, E)
    if quant:
        _check_quant(got, y, quant)
    return got


@pytest.mark.gpu
@pytest.mark.parametrize("T,H", [(1, 7168), (1, 32), (3, 64), (130, 2880), (37, 4096), (300, 7168), (1111, 256),
                                 (5, 8224), (2, 16384), (3, 32768), (4, 24608)])
@pytest.mark.parametrize("quant", [None, "mxfp8", "mxfp4"])
def test_matches_oracle(T, H, quant):
    _run(T, H, False, True, "bf16", quant, deq=quant is not None)


@pytest.mark.gpu
@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("res", [False, True])
@pytest.mark.parametrize("wt", [None, "bf16", "f32"])
@pytest.mark.parametrize("quant,want_y", [(None, True), ("mxfp8", False), ("mxfp4", True)])
def test_types_and_optional_parts(f32, res, wt, quant, want_y):
    got = _run(67, 1056, f32, res, wt, quant, want_y=want_y)
    assert (got["y"] is None) == (not want_y) and (got["residual"] is None) == (not res) and got["deq"] is None


@pytest.mark.gpu
@pytest.mark.parametrize("H", [8, 40, 1000, 8200])
def test_rows_of_eights_without_quantisation(H):
    _run(9, H, False, True, "f32", None)


@pytest.mark.gpu
@pytest.mark.parametrize("T", [7, 400])
def test_strides_in_place_and_rows_around(T):
    """Strided inputs and outputs, residual and x updated in place; the columns between the rows and
    the rows behind the last stay as they were."""
    H = 320
    x, r, w = _inputs(T, H, False, True, "bf16", 3)
    xs, rs = (torch.full((T + 2, H + 24), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    xs[:T, :H], rs[:T, :H] = x.cuda(), r.cuda()
    codes = torch.full((T + 2, H), 9, dtype=torch.uint8, device="cuda")
    scales = torch.full((T + 2, H // 32), 9, dtype=torch.uint8, device="cuda")
    got = m.moe_add_rmsnorm(xs[:T, :H], w.cuda(), rs[:T, :H], 1e-5, "mxfp8",
                            out=dict(residual=rs[:T, :H], y=xs[:T, :H], codes=codes[:T], scales=scales[:T]))
    torch.cuda.synchronize()
    rr, y = O.add_rmsnorm(x.double().numpy(), r.double().numpy(), w.double().numpy(), 1e-5)
    _check_rows(rs[:T, :H], rr, 2.0 ** -24)
    _check_rows(xs[:T, :H], y, E)
    _check_quant(got, y, "mxfp8")
    for t in (xs, rs):
        assert bool((t[:, H:] == 7).all()) and bool((t[T:] == 7).all())
    assert bool((codes[T:] == 9).all()) and bool((scales[T:] == 9).all())


@pytest.mark.gpu
@pytest.mark.parametrize("quant", ["mxfp8", "mxfp4"])
def test_zero_rows_tiny_rows_and_nan(quant):
    """A zero row gives zeros with the smallest scale; tiny rows are ruled by eps; an infinity or NaN
    poisons its own row alone."""
    H = 256
    x = torch.randn(6, H, generator=torch.Generator().manual_seed(1))
    x[1] = 0
    x[2] *= 1e-30
    x[3, 5] = float("nan")
    x[4, 40] = float("inf")
    got = m.moe_add_rmsnorm(x.cuda(), quant=quant, deq=True)
    torch.cuda.synchronize()
    keep = [0, 1, 2, 5]
    _, y = O.add_rmsnorm(x.double().numpy()[keep])
    sub = {k: None if v is None else v[keep] for k, v in got.items()}
    _check_rows(sub["y"], y, E)
    _check_quant(sub, y, quant)
    assert bool((got["scales"][1] == 0).all()) and bool((got["codes"][1] == 0).all())
    assert bool(got["deq"][3].isnan().all()) and bool((got["scales"][3] == 255).all())
    assert bool(got["y"][4, 40].isnan()) and int(got["scales"][4, 1]) == 255
    assert bool((got["scales"][4, 2:] == 0).all())


@pytest.mark.gpu
def test_binding_refuses_bad_tensors():
    x = torch.zeros(4, 64, dtype=torch.bfloat16, device="cuda")
    for kw in (dict(residual=x[:3]), dict(residual=x.float()), dict(weight=x[0, :32]), dict(deq=True),
               dict(out=dict(y=x.float())), dict(quant="mxfp8", out=dict(codes=torch.empty(4, 63, dtype=torch.uint8)))):
        with pytest.raises(ValueError):
            m.moe_add_rmsnorm(x, **kw)
    with pytest.raises(ValueError):
        m.moe_add_rmsnorm(x[:1].expand(4, 64))         # rows that overlap
    with pytest.raises(ValueError):
        m.moe_add_rmsnorm(torch.zeros(64, 4, dtype=torch.bfloat16, device="cuda").t())
    with pytest.raises(m.MoEError):
        m.moe_add_rmsnorm(torch.zeros(4, 68, dtype=torch.bfloat16, device="cuda")[:, 4:], weight=None)


@pytest.mark.gpu
@pytest.mark.parametrize("H", [32, 96, 512, 544])
@pytest.mark.parametrize("T", [296, 301, 1000])
def test_many_short_rows(T, H):
    """Rows of up to 512 values share a block, a warp each; the last block is not full."""
    _run(T, H, False, True, "bf16", "mxfp4", deq=True)
    _run(T, H, True, False, "f32", "mxfp8")


@pytest.mark.gpu
def test_graph_and_stream():
    """On a side stream, and captured and replayed on new rows."""
    x, r, w = (None if t is None else t.cuda() for t in _inputs(70, 512, False, True, "bf16", 4))
    out = dict(y=torch.empty_like(x), residual=torch.empty_like(x),
               codes=torch.empty(70, 256, dtype=torch.uint8, device="cuda"),
               scales=torch.empty(70, 16, dtype=torch.uint8, device="cuda"))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    m.moe_add_rmsnorm(x, w, r, 1e-5, "mxfp4", out=out, stream=side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        m.moe_add_rmsnorm(x, w, r, 1e-5, "mxfp4", out=out)
    x2 = _inputs(70, 512, False, True, "bf16", 5)[0].cuda()
    x.copy_(x2)
    g.replay()
    torch.cuda.synchronize()
    want = m.moe_add_rmsnorm(x2, w, r, 1e-5, "mxfp4")
    for k in out:
        assert torch.equal(out[k], want[k])
