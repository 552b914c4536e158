"""The first call of the MXFP4 x MXFP4 product on a device sets up every tile: products of all other sizes can
be captured after it, with nothing run before at their size. In a process of its own, where nothing has run."""
import subprocess
import sys

import pytest

from tests.conftest import ROOT

SCRIPT = """
import os, torch
import mixture_experts_layer_21_b200 as m
from tests.test_mxfp4 import _case

def operands(lens, gather, seed):
    ac, asc, wc, wsc, idx, al, cu, M = _case(lens, 264, 352, gather, seed=seed)
    w = m.moe_prepare_weights(m.Weight("mxfp4", wc.cuda(), wsc.cuda()))
    return ac.cuda(), asc.cuda(), w, cu.cuda(), None if idx is None else idx.cuda()

def setting(tile):
    os.environ["MOE_GEMM_PAIRS"] = "1" if tile == "pairs" else "0"
    os.environ["MOE_TOKEN_TILE"] = "16" if tile == "pairs" else tile

ops = {(t, g): operands([40, 0, 190, 17], g, 5) for t in ("16", "32", "64", "128", "pairs") for g in (False, True)}
torch.cuda.synchronize()
setting("16")
m.moe_grouped_gemm_mxfp4(*ops["16", False])
torch.cuda.synchronize()
graphs = {}
for (t, g), a in ops.items():
    setting(t)
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        out = m.moe_grouped_gemm_mxfp4(*a)
    graphs[t, g] = gr, out
for k, (gr, out) in graphs.items():
    gr.replay()
torch.cuda.synchronize()
for (t, g), a in ops.items():
    setting(t)
    assert torch.equal(graphs[t, g][1], m.moe_grouped_gemm_mxfp4(*a)), (t, g)
assert m.moe_get_device_error() == 0
print("captured", len(graphs))
"""


@pytest.mark.gpu
def test_every_tile_is_captured_after_one_call():
    r = subprocess.run([sys.executable, "-c", SCRIPT], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    assert "captured 10" in r.stdout
