"""Routing by scores (moe_route_scored): ids bit-exact and weights against the 64-bit oracle, and
the calls it refuses.

Weight tolerance, relative: scores of 32 bits carry the rounding of the exponential's argument
(half a step of |l - max| or |l|, that is |l| 2^-24 relative to the exponential), the exponential's
2 units (2^-22), a sum of at most 1024 positive terms whose longest chain is 32 + 5 additions
(37 * 2^-24) and three more roundings: (D + 44) 2^-24 with D the largest |l - max| or |l| of a row's
chosen experts; twice that where the chosen scores are summed and divided again.
"""
import ctypes

import numpy as np
import pytest
import torch

import mixture_experts_layer_21_b200 as m
from oracle import moe_oracle as O

L = m.lib()
INVALID, UNSUP, ALIGN = 1, 2, 3


def _call(**kw):
    d = dict(logits=16, in_is_bf16=0, row_stride=None, bias=None, T=4, E=16, topk=2, scoring=0, n_group=1, topk_group=1,
             group_score=0, renormalize=1, routed_scaling_factor=1.0, topk_ids=16, topk_w=16)
    d.update(kw)
    if d["row_stride"] is None:
        d["row_stride"] = d["E"]
    return L.moe_route_scored(ctypes.byref(m.moe_route_args_t(**d)), None)


@pytest.mark.parametrize("kw", [dict(T=-1), dict(E=0), dict(topk=0), dict(topk=17), dict(row_stride=15),
                                dict(row_stride=0), dict(row_stride=-16), dict(scoring=2), dict(scoring=-1),
                                dict(n_group=0), dict(n_group=3), dict(n_group=4, topk_group=0),
                                dict(n_group=4, topk_group=5), dict(n_group=8, topk_group=1, topk=3),
                                dict(group_score=2), dict(routed_scaling_factor=0.0),
                                dict(routed_scaling_factor=float("nan")), dict(routed_scaling_factor=float("inf")),
                                dict(logits=None), dict(topk_ids=None), dict(topk_w=None)])
def test_refuses_bad_arguments(kw):
    assert _call(**kw) == INVALID


@pytest.mark.parametrize("kw", [dict(logits=18), dict(logits=17, in_is_bf16=1), dict(bias=2), dict(topk_ids=18),
                                dict(topk_w=17)])
def test_refuses_misaligned_pointers(kw):
    assert _call(**kw) == ALIGN


@pytest.mark.parametrize("kw", [dict(E=1025), dict(E=66, n_group=33, topk_group=33), dict(E=64, topk=33)])
def test_refuses_unsupported_sizes(kw):
    assert _call(**kw) == UNSUP


def test_packed_arguments_have_the_structures_layout():
    for pack, cls in ((m._ROUTE_ARGS, m.moe_route_args_t), (m._RMSNORM_ARGS, m.moe_rmsnorm_args_t)):
        vals = [1000 + i for i in range(len(cls._fields_))]
        a = cls.from_buffer_copy(pack.pack(*vals).ljust(ctypes.sizeof(cls), b"\0"))
        assert [getattr(a, f[0]) for f in cls._fields_] == vals


def test_no_tokens_is_a_no_op():
    assert _call(T=0, logits=None, topk_ids=None, topk_w=None) == 0
    assert L.moe_route_scored(None, None) == INVALID


@pytest.mark.parametrize("bad", ["dtype", "cpu", "bias", "cols"])
def test_binding_refuses(bad):
    x = torch.zeros(4, 8)
    with pytest.raises((ValueError, RuntimeError, AssertionError)):
        m.moe_route_scored(x.half() if bad == "dtype" else x, 2, bias=torch.zeros(7) if bad == "bias" else None)


def test_oracle_agrees_with_the_two_special_forms():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((40, 32)).astype(np.float32)
    b = (0.1 * rng.standard_normal(32)).astype(np.float32)
    for got, want in ((O.route_scored(x, 4), O.route_topk(x, 4)),
                      (O.route_scored(x, 4, "sigmoid", b, 8, 3, "top2", True, 2.5),
                       O.route_topk_grouped(x, 4, 8, 3, b, 2.5))):
        assert np.array_equal(got[0], want[0])
        assert np.allclose(got[1], want[1], rtol=1e-12)


def test_oracle_masks():
    x = np.full((3, 6), -np.inf)
    x[0, 4], x[1, 2], x[1, 5] = 1.0, np.nan, 3.0
    ids, w = O.route_scored(x, 3, "softmax", np.array([0, 9.0, 0, 0, 0, 0]))
    assert ids.tolist() == [[4, 0, 1], [5, 0, 1], [0, 1, 2]]
    assert w.tolist() == [[1, 0, 0], [1, 0, 0], [0, 0, 0]]


def _check(x, k, scoring, bias, ng, tg, gscore, renorm, scale, strided=0):
    xd = x.cuda()
    if strided:
        wide = torch.full((x.shape[0], x.shape[1] + strided), 99.0, dtype=x.dtype, device="cuda")
        wide[:, :x.shape[1]] = xd
        xd = wide[:, :x.shape[1]]
    ids, w = m.moe_route_scored(xd, k, scoring, None if bias is None else bias.cuda(), ng, tg, gscore, renorm, scale)
    torch.cuda.synchronize()
    xn = x.double().numpy()
    rids, rw = O.route_scored(xn, k, scoring, None if bias is None else bias.numpy(), ng, tg, gscore, renorm, scale)
    assert np.array_equal(ids.cpu().numpy(), rids)
    live = np.where(np.isfinite(xn), xn, np.nan)
    chosen = np.take_along_axis(live, rids.astype(np.int64), 1)
    with np.errstate(all="ignore"):
        ref = np.nanmax(np.where(np.isfinite(live), live, -1e30), axis=1, keepdims=True) if scoring == "softmax" else 0.0
        D = np.nan_to_num(np.abs(chosen - ref), nan=0.0, posinf=0.0)
    D = D.max(axis=1, keepdims=True) if x.shape[0] else D
    tol = (2 if renorm else 1) * (D + 44) * 2.0 ** -24 * np.abs(rw)
    assert np.all(np.abs(w.cpu().numpy().astype(np.float64) - rw) <= tol)


CASES = [  # T, E, k, scoring, bias, groups, kept, group score, renorm
    (1, 256, 8, "sigmoid", True, 8, 4, "top2", True),
    (300, 256, 8, "sigmoid", True, 8, 4, "top2", True),
    (129, 128, 4, "softmax", True, 1, 1, "max", False),
    (64, 160, 6, "softmax", False, 8, 3, "max", False),
    (65, 160, 6, "softmax", False, 8, 3, "top2", True),
    (33, 1024, 32, "sigmoid", True, 32, 7, "max", True),
    (31, 1024, 8, "softmax", True, 1, 1, "max", True),
    (7, 1, 1, "softmax", False, 1, 1, "max", True),
    (5, 33, 32, "sigmoid", False, 1, 1, "max", False),
    (17, 12, 3, "sigmoid", True, 12, 3, "top2", True),
    (40, 513, 5, "softmax", True, 27, 26, "top2", False),
    (2000, 64, 6, "sigmoid", True, 4, 2, "max", True),
]


@pytest.mark.gpu
@pytest.mark.parametrize("T,E,k,scoring,bias,ng,tg,gscore,renorm", CASES)
@pytest.mark.parametrize("kind", ["normal", "ties", "bf16"])
def test_matches_oracle(T, E, k, scoring, bias, ng, tg, gscore, renorm, kind):
    g = torch.Generator().manual_seed(T * 31 + E)
    x = torch.randn(T, E, generator=g) * 2
    b = torch.randn(E, generator=g) * 0.05 if bias else None
    if kind == "ties":                     # equal logits and equal biases: ties between experts and groups
        x = torch.round(x)
        b = torch.round(b * 10) / 8 if bias else None
    if kind == "bf16":
        x = x.bfloat16()
    _check(x, k, scoring, b, ng, tg, gscore, renorm, 2.5, strided=3 if kind == "bf16" else 0)


@pytest.mark.gpu
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("ng,tg,gscore", [(1, 1, "max"), (4, 2, "top2"), (4, 2, "max")])
@pytest.mark.parametrize("bias", [False, True])
def test_masked_experts(scoring, ng, tg, gscore, bias):
    """-inf and NaN logits: some experts, all but one, a whole group, whole rows; +inf logits."""
    g = torch.Generator().manual_seed(5)
    x = torch.randn(64, 64, generator=g)
    x[torch.rand(64, 64, generator=g) < 0.4] = float("-inf")
    x[torch.rand(64, 64, generator=g) < 0.1] = float("nan")
    x[3] = float("-inf")
    x[4] = float("nan")
    x[5] = float("-inf")
    x[5, 37] = -2.0
    x[6, 16:32] = float("-inf")
    x[7, 9] = float("inf")
    x[8, 2] = x[8, 50] = float("inf")
    x[9] = float("inf")
    b = torch.randn(64, generator=g) if bias else None
    _check(x, 6, scoring, b, ng, tg, gscore, True, 1.0)
    _check(x, 6, scoring, b, ng, tg, gscore, False, 1.5)


def test_oracle_biases_that_are_not_finite():
    x = np.array([[0.0, 1.0, 2.0, 3.0]])
    b = np.array([np.nan, 0.5, -np.inf, -np.inf])
    assert O.route_scored(x, 4, "sigmoid", b)[0].tolist() == [[1, 0, 2, 3]]
    assert O.route_scored(x, 2, "sigmoid", np.array([0.0, np.inf, 0.0, np.inf]))[0].tolist() == [[1, 3]]


@pytest.mark.gpu
@pytest.mark.parametrize("E,ng,tg", [(64, 1, 1), (64, 4, 2), (256, 8, 4), (36, 6, 2)])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("gscore", ["max", "top2"])
def test_biases_that_are_not_finite(E, ng, tg, scoring, gscore):
    """-inf and NaN of either sign rank an expert with the masked ones, +inf before all others: some
    experts, a whole group, all but fewer than topk, all."""
    g = torch.Generator().manual_seed(E + ng)
    x = torch.randn(40, E, generator=g)
    x[1] = float("-inf")
    x[2, ::3] = float("nan")
    nan = torch.tensor([0x7fc00000, -0x400000], dtype=torch.int32).view(torch.float32)
    for kind in range(5):
        b = torch.randn(E, generator=g) * 0.1
        if kind == 0:
            b[torch.rand(E, generator=g) < 0.3] = float("-inf")
            b[::7], b[1::7] = nan[0], nan[1]
        elif kind == 1:
            b[:E // ng] = float("-inf") if ng > 1 else float("nan")
        elif kind == 2:
            b[2:] = nan[1]
        elif kind == 3:
            b[:] = nan[0]
        else:
            b[5::6] = float("inf")
            b[::5] = float("-inf")
        _check(x, 6, scoring, b, ng, tg, gscore, True, 1.0)
        _check(x, 6, scoring, b, ng, tg, gscore, False, 1.5)


@pytest.mark.gpu
def test_large_and_close_scores():
    """Saturated sigmoids, logits far apart, and sums s + b that differ by a few 2^-25."""
    g = torch.Generator().manual_seed(6)
    x = torch.randn(200, 96, generator=g) * 30
    _check(x, 8, "softmax", None, 1, 1, "max", True, 1.0)
    _check(x.clamp(-30, 30), 8, "sigmoid", torch.randn(96, generator=g) * 1e-3, 6, 3, "top2", True, 1.0)
    # s + b = 1/2 + 1/8 for every expert up to the rounding of b to 32 bits
    y = torch.randn(100, 64, generator=g)
    s = torch.sigmoid(y[:1].double())
    b = (0.625 - s[0]).float()
    _check(y[:1].expand(100, 64).contiguous(), 8, "sigmoid", b, 1, 1, "max", True, 1.0)
    _check(y[:1].expand(100, 64).contiguous(), 8, "sigmoid", b, 8, 4, "top2", True, 1.0)


@pytest.mark.gpu
def test_graph_and_streams():
    """The call on a side stream, and captured and replayed on new logits."""
    x = torch.randn(50, 64, device="cuda")
    ids = torch.empty(50, 4, dtype=torch.int32, device="cuda")
    w = torch.empty(50, 4, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    m.moe_route_scored(x, 4, ids=ids, w=w, stream=side)
    torch.cuda.synchronize()
    assert np.array_equal(ids.cpu().numpy(), O.route_scored(x.cpu().numpy(), 4)[0])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        m.moe_route_scored(x, 4, ids=ids, w=w)
    x.copy_(torch.randn(50, 64))
    g.replay()
    torch.cuda.synchronize()
    assert np.array_equal(ids.cpu().numpy(), O.route_scored(x.cpu().numpy(), 4)[0])


@pytest.mark.gpu
@pytest.mark.slow
def test_logits_past_32_bits_of_elements():
    T, E = 2 ** 31 // 1024 + 50, 1024                 # 4.3 GB of bf16 logits
    x = torch.randn(1, E, device="cuda").bfloat16().repeat(T, 1)
    x[-1] = torch.randn(E).bfloat16()
    ids, w = m.moe_route_scored(x, 8)
    for r in (0, T - 2, T - 1):
        rids, rw = O.route_scored(x[r:r + 1].double().cpu().numpy(), 8)
        assert np.array_equal(ids[r:r + 1].cpu().numpy(), rids)
        assert np.allclose(w[r:r + 1].cpu().numpy(), rw, rtol=1e-5)


@pytest.mark.gpu
@pytest.mark.parametrize("E,ng", [(256, 8), (160, 8), (1024, 32), (48, 4), (96, 1), (24, 1)])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_close_scores_are_decided_in_64_bits(E, ng, scoring):
    """Rows made of few distinct logits a last place apart, biases that nearly cancel the difference of
    the scores: neighbours and group sums within the error of 32 bits, in runs shorter and longer than
    the 32 candidates that are ordered at once."""
    g = torch.Generator().manual_seed(E)
    base = torch.tensor([0.5, 1.0, 1.5])
    x = base[torch.randint(0, 3, (120, E), generator=g)]
    x = x + torch.randint(-2, 3, (120, E), generator=g) * 2.0 ** -23
    b = torch.randint(-3, 4, (E,), generator=g) * 2.0 ** -24
    k = min(8, E // ng * max(1, ng // 2))
    for gscore in ("max", "top2"):
        _check(x, k, scoring, b, ng, max(1, ng // 2), gscore, True, 1.0)
        _check(x, k, scoring, None, ng, max(1, ng // 2), gscore, False, 1.0)
    wide = torch.randn(E, generator=g)                # every expert live, c within a few places of each other
    s = torch.sigmoid(wide.double()) if scoring == "sigmoid" else torch.softmax(wide.double(), 0)
    _check(wide.expand(40, E).contiguous(), k, scoring, (0.75 - s).float(), ng, max(1, ng // 2), "top2", True, 1.0)
