"""Every call of the binding with ``stream=`` and nothing else made by the caller: what it allocates is memory
of that stream. The current stream meanwhile still has to read blocks, just freed, of the same sizes."""
import pytest
import torch

import mixture_experts_layer_21_b200 as m

pytestmark = pytest.mark.gpu


def _tensors(got):
    if torch.is_tensor(got):
        return [got]
    got = got.values() if isinstance(got, dict) else got
    return [t for t in got if torch.is_tensor(t)]


def _mxfp4_weights(G, N, K, seed):
    g = torch.Generator().manual_seed(seed)
    c = torch.randint(0, 256, (G, N, K // 2), generator=g, dtype=torch.uint8).cuda()
    s = torch.randint(118, 126, (G, N, K // 32), generator=g, dtype=torch.uint8).cuda()
    return m.moe_prepare_weights(m.Weight("mxfp4", c, s))


def _calls():
    """name -> a call that takes a stream; inputs are made once."""
    torch.manual_seed(3)
    T, H, I, E, k = 300, 512, 256, 8, 2
    M = T * k
    x = torch.randn(T, H, device="cuda").bfloat16()
    logits = torch.randn(T, E, device="cuda")
    gate, up = (torch.randn(M, I, device="cuda").bfloat16() for _ in range(2))
    ids, w = m.moe_route_topk(logits, k)
    p = m.moe_permute(ids, w, E, x=x)
    cu, idx, inv, rows = (p[n].clone() for n in ("cu_seqlens", "perm_token", "inv_perm", "x_perm"))
    pw = p["perm_w"].clone()
    y = torch.randn(M, H, device="cuda").bfloat16()
    codes, scales, _ = m.moe_quantize_mxfp4(x)
    w4 = _mxfp4_weights(E, I, H, 1)
    wb = m.Weight("bf16", torch.randn(E, I, H, device="cuda").bfloat16())
    wd = m.Weight("bf16", torch.randn(E, H, I, device="cuda").bfloat16())
    g = torch.Generator().manual_seed(2)
    wn = m.moe_prepare_weights(m.Weight("nvfp4", torch.randint(0, 256, (E, I, H // 2), generator=g, dtype=torch.uint8).cuda(),
                                        torch.full((E, I, H // 16), 0x38, dtype=torch.uint8, device="cuda"),
                                        torch.ones(E, device="cuda")))
    nc, nsb, ns, _ = m.moe_quantize_nvfp4(rows, deq=False)
    layer = m.MoEForward(wb, wb, wd, E, k, T_max=T)
    layer(x, logits, stream=torch.cuda.Stream())      # the first one waits for the workspace, made on the current stream
    return {
        "route_topk": lambda s: m.moe_route_topk(logits, k, stream=s),
        "route_topk_grouped": lambda s: m.moe_route_topk_grouped(logits, k, 4, 2, stream=s),
        "route_scored": lambda s: m.moe_route_scored(logits, k, stream=s),
        "add_rmsnorm": lambda s: m.moe_add_rmsnorm(x, residual=x, quant="mxfp4", deq=True, stream=s),
        "permute": lambda s: {n: t for n, t in m.moe_permute(ids, w, E, x=x, stream=s).items() if n != "ws"},
        "grouped_gemm": lambda s: m.moe_grouped_gemm(rows, w4, cu, stream=s),
        "grouped_gemm_nvfp4": lambda s: m.moe_grouped_gemm_nvfp4(nc, nsb, ns, wn, cu, stream=s),
        "grouped_gemm_mxfp4": lambda s: m.moe_grouped_gemm_mxfp4(codes, scales, w4, cu, idx, stream=s),
        "act_and_mul": lambda s: m.moe_act_and_mul(gate, up, pw, stream=s),
        "bias_act_and_mul": lambda s: m.moe_bias_act_and_mul(gate, up, cu, stream=s),
        "combine": lambda s: m.moe_combine(y, inv, w, stream=s),
        "quantize_nvfp4": lambda s: m.moe_quantize_nvfp4(x, stream=s),
        "quantize_mxfp8": lambda s: m.moe_quantize_mxfp8(x, stream=s),
        "quantize_mxfp4": lambda s: m.moe_quantize_mxfp4(x, deq=True, stream=s),
        "forward": lambda s: layer(x, logits, stream=s),
    }


NAMES = ["route_topk", "route_topk_grouped", "route_scored", "add_rmsnorm", "permute", "grouped_gemm",
         "grouped_gemm_nvfp4", "grouped_gemm_mxfp4", "act_and_mul", "bias_act_and_mul", "combine", "quantize_nvfp4",
         "quantize_mxfp8", "quantize_mxfp4", "forward"]


@pytest.mark.parametrize("name", NAMES)
def test_outputs_are_memory_of_the_given_stream(name):
    call = _calls()[name]
    want = [t.clone() for t in _tensors(call(None))]
    # blocks of the sizes that the call makes, and of its workspaces
    sizes = [t.numel() * t.element_size() for t in want] + [256, 1 << 20]
    side = torch.cuda.Stream()
    baits = [torch.full((n,), 0x5a, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(2)]
    seen = [torch.empty_like(b) for b in baits]
    torch.cuda.synchronize()
    torch.cuda._sleep(200_000_000)                    # about a tenth of a second
    for b, s in zip(baits, seen):
        s.copy_(b)                                    # still to come on the current stream
    del b
    baits.clear()
    got = _tensors(call(side))
    side.synchronize()
    done = torch.cuda.current_stream().query()
    torch.cuda.synchronize()
    assert not done                                   # the call did not wait for the current stream
    assert all(bool((s == 0x5a).all()) for s in seen)
    assert len(got) == len(want)
    for a, b in zip(got, want):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


@pytest.mark.parametrize("name", NAMES)
def test_captured_with_the_stream_named(name):
    """The capturing stream given as stream=: what the call allocates is the graph's."""
    call = _calls()[name]
    want = [t.clone() for t in _tensors(call(None))]
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = _tensors(call(torch.cuda.current_stream()))
    for _ in range(2):
        for t in got:
            t.zero_()
        g.replay()
    torch.cuda.synchronize()
    assert len(got) == len(want)
    for a, b in zip(got, want):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
