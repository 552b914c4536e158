"""The weights of moe_route_scored are formed in 64 bits and rounded once.

Tolerance. l - max and the score are within a few 2^-53 (1 + |l - max|) of the exact value, |l - max| < 2^8 here;
a sum of at most 1024 positive terms adds at most 2^-43, a reciprocal 2^-45, the scaling factor 2^-53: below 2^-40
in all, relative. The rounding to fp32 adds half a step, 2^-24, and 2^-150 where the weight is subnormal. The
oracle is within the same 2^-40.
"""
import numpy as np
import pytest
import torch

import mixture_experts_layer_21_b200 as m
from oracle import moe_oracle as O

pytestmark = pytest.mark.gpu


def _check(x, k, scoring, bias, ng, tg, gscore, renorm, scale):
    ids, w = m.moe_route_scored(x.cuda(), k, scoring, None if bias is None else bias.cuda(), ng, tg, gscore, renorm, scale)
    rids, rw = O.route_scored(x.double().numpy(), k, scoring, None if bias is None else bias.numpy(), ng, tg, gscore, renorm,
                              float(np.float32(scale)))
    assert np.array_equal(ids.cpu().numpy(), rids)
    d = np.abs(w.cpu().numpy().astype(np.float64) - rw)
    assert np.all(d <= (2.0 ** -24 + 2.0 ** -38) * np.abs(rw) + 2.0 ** -150), float((d / np.abs(rw)).max() * 2 ** 24)


@pytest.mark.parametrize("E,ng,tg,gscore", [(256, 8, 4, "top2"), (128, 1, 1, "max"), (160, 8, 3, "max"), (1024, 32, 7, "top2"),
                                            (33, 1, 1, "max"), (8, 1, 1, "max")])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("renorm", [False, True])
def test_rounded_once(E, ng, tg, gscore, scoring, bias, renorm):
    g = torch.Generator().manual_seed(E + ng)
    b = torch.randn(E, generator=g) * 0.05 if bias else None
    for spread, dtype in ((2.0, torch.float32), (2.0, torch.bfloat16), (12.0, torch.float32)):
        x = (torch.randn(300, E, generator=g) * spread).to(dtype)
        x[1, ::3] = float("-inf")
        _check(x, min(8, E), scoring, b, ng, tg, gscore, renorm, 2.5)


def test_one_expert_and_every_expert():
    g = torch.Generator().manual_seed(7)
    x = torch.randn(200, 32, generator=g) * 3
    for scoring in ("softmax", "sigmoid"):
        for renorm in (False, True):
            _check(x, 1, scoring, None, 1, 1, "max", renorm, 1.0)
            _check(x, 32, scoring, None, 1, 1, "max", renorm, 1.0)


def test_far_from_the_largest():
    """A bias that chooses experts 60 to 130 below the largest logit: weights down to fp32's subnormal values."""
    g = torch.Generator().manual_seed(8)
    x = torch.randn(200, 64, generator=g)
    x[:, 5] += 100
    x[:100, 5] += 20
    b = torch.zeros(64)
    b[5] = -3.0
    for renorm in (False, True):
        _check(x, 4, "softmax", b, 1, 1, "max", renorm, 1.0)
    _check(x - 110, 4, "sigmoid", None, 1, 1, "max", False, 1.0)
    _check(x - 110, 4, "sigmoid", None, 1, 1, "max", True, 1.0)
