"""MXFP4 rows (moe_quantize_mxfp4), the MXFP4 x MXFP4 grouped product (moe_grouped_gemm_mxfp4), a run of
the operators around the layer together, and the calls they refuse.

Quantised codes and scales are bit-exact: the division by a power of two is exact. The product's
terms are exact; the tensor cores add 64 of them per instruction to the accumulator in fp32, each
instruction within 2^-22 of the magnitudes it adds, so an output lies within
(K/64 + 1) 2^-22 sum_k |a_k w_k| of the exact sum before its bf16 rounding (2^-8).
"""
import ctypes

import numpy as np
import pytest
import torch

import mixture_experts_layer_21_b200 as m
import workloads as W
from oracle import moe_oracle as O

L = m.lib()
INVALID, UNSUP, ALIGN, WS_SMALL, NOT_PREP, DEVICE, TIMEOUT = 1, 2, 3, 4, 8, 6, 7


# ------------------------------------------------------------------ refusals (CPU)

def _quant(**kw):
    d = dict(x=16, f32=0, stride=64, R=4, K=64, codes=16, scales=1, deq=None)
    d.update(kw)
    return L.moe_quantize_mxfp4(d["x"], d["f32"], d["stride"], d["R"], d["K"], d["codes"], d["scales"], d["deq"], None)


@pytest.mark.parametrize("kw,want", [
    (dict(R=-1), INVALID), (dict(K=-32), INVALID), (dict(stride=32), INVALID), (dict(K=48), ALIGN),
    (dict(stride=68), ALIGN), (dict(x=None), INVALID), (dict(codes=None), INVALID), (dict(scales=None), INVALID),
    (dict(x=8), ALIGN), (dict(codes=8), ALIGN), (dict(deq=8), ALIGN), (dict(R=0, x=None), 0),
    (dict(K=0, x=None), 0)])
def test_quantize_refuses(kw, want):
    assert _quant(**kw) == want


def _gemm(w=None, **kw):
    d = dict(a=16, s=1, rows=8, idx=None, M=8, cu=16, out=16, room=None, ws=16, nws=256)
    d.update(kw)
    return L.moe_grouped_gemm_mxfp4(d["a"], d["s"], d["rows"], d["idx"], d["M"],
                                    None if w is None else ctypes.byref(w), d["cu"], d["out"], d["room"], d["ws"], d["nws"],
                                    None)


def _w(fmt=1, G=2, N=64, K=64, prepared=True):
    w = m.moe_weight_t(fmt, G, N, K, 16, 16, None)
    if prepared:
        w.kdata, w.kscale, w.kalpha = 16, 16, 16
    return w


@pytest.mark.parametrize("w,kw,want", [
    (None, {}, INVALID), (_w(), dict(M=-1), INVALID), (_w(), dict(rows=-1), INVALID), (_w(), dict(rows=7), INVALID),
    (_w(), dict(rows=0, idx=16), INVALID), (_w(G=0), {}, INVALID), (_w(N=0), {}, INVALID), (_w(K=0), {}, INVALID),
    (_w(G=1025), {}, UNSUP), (_w(fmt=0), {}, UNSUP), (_w(fmt=2), {}, UNSUP), (_w(prepared=False), {}, NOT_PREP),
    (_w(K=48), {}, ALIGN), (_w(N=60), {}, ALIGN), (_w(), dict(a=8), ALIGN), (_w(), dict(out=8), ALIGN), (_w(), dict(room=8), ALIGN),
    (_w(), dict(a=None), INVALID), (_w(), dict(s=None), INVALID), (_w(), dict(cu=None), INVALID),
    (_w(), dict(out=None), INVALID), (_w(), dict(ws=None), INVALID), (_w(), dict(nws=255), WS_SMALL),
    (_w(), dict(M=0, a=None, cu=None), 0)])
def test_product_refuses(w, kw, want):
    assert _gemm(w, **kw) == want


def test_oracle_quantiser_is_the_nearest_grid_value():
    g = np.random.default_rng(0)
    x = (g.standard_normal((8, 64)) * np.exp2(g.integers(-40, 40, (8, 1)))).astype(np.float32)
    x[0, :32] = 0
    codes, scales = O.mxfp4_quantize_rows(x)
    v = O.mxfp4_dequantize_rows(codes, scales)
    p = np.repeat(O.e8m0_decode(scales), 32, axis=1)
    grid = np.concatenate((O.E2M1_MAG, -O.E2M1_MAG))
    best = np.abs(x[:, :, None] / p[:, :, None] - grid).min(axis=2)
    assert np.array_equal(np.abs(x / p - v / p), best)
    assert scales[0, 0] == 0 and not codes[0, :32].any()
    assert np.all(np.abs(x / p) < 8)


# ------------------------------------------------------------------ quantiser (GPU)

def _pack(codes):
    return codes[:, 0::2] | codes[:, 1::2] << 4


def _edge_rows(K):
    """Every e2m1 midpoint and its neighbours, zeros of both signs, the ends of the exponents."""
    mids = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.9375], np.float32)
    v = np.concatenate([mids, np.nextafter(mids, 0), np.nextafter(mids, 9), -mids, [0.0, -0.0, 4.0, -4.0]]).astype(np.float32)
    rows = []
    for p in (1.0, 2.0 ** -126, 2.0 ** -149, 2.0 ** 100, 2.0 ** 124):
        with np.errstate(over="ignore"):
            r = np.resize(v, K).astype(np.float64) * p
        rows.append(r.astype(np.float32))
    rows += [np.zeros(K, np.float32), np.full(K, -0.0, np.float32), np.full(K, np.finfo(np.float32).max, np.float32)]
    for bad in (np.nan, np.inf, -np.inf):
        r = np.resize(v, K).copy()
        r[K // 2] = bad
        rows.append(r)
    return np.stack(rows)


def _check_quant(x, strided=0, deq=True):
    xd = x.cuda()
    if strided:
        wide = torch.full((x.shape[0], x.shape[1] + strided), float("nan"), dtype=x.dtype, device="cuda")
        wide[:, :x.shape[1]] = xd
        xd = wide[:, :x.shape[1]]
    codes, scales, d = m.moe_quantize_mxfp4(xd, deq=deq)
    torch.cuda.synchronize()
    rc, rs = O.mxfp4_quantize_rows(x.float().numpy())
    assert np.array_equal(scales.cpu().numpy(), rs)
    assert np.array_equal(codes.cpu().numpy(), _pack(rc))
    assert (d is not None) == deq
    if deq:
        assert np.array_equal(d.double().cpu().numpy(), O.mxfp4_dequantize_rows(rc, rs), equal_nan=True)


@pytest.mark.gpu
@pytest.mark.parametrize("R,K", [(1, 32), (1, 2880), (131, 2880), (7, 7168), (1000, 96), (4097, 64), (3, 4096)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_quantize_matches_oracle(R, K, dtype):
    g = torch.Generator().manual_seed(R + K)
    x = (torch.randn(R, K, generator=g) * torch.exp2(4 * torch.randn(R, 1, generator=g))).to(dtype)
    _check_quant(x)
    _check_quant(x, strided=8, deq=False)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_quantize_edges(dtype):
    _check_quant(torch.from_numpy(_edge_rows(96)).to(dtype))


@pytest.mark.gpu
def test_quantize_many_values():
    """More 8-value chunks than one pass of the grid covers, checked on the GPU against a lookup of
    the value of every code in 64 bits."""
    x = torch.randn(20000, 2048, device="cuda").bfloat16()
    codes, scales, deq = m.moe_quantize_mxfp4(x, deq=True)
    tab = torch.tensor(np.concatenate((O.E2M1_MAG, -O.E2M1_MAG)), device="cuda")
    v = torch.stack((tab[(codes & 15).long()], tab[(codes >> 4).long()]), -1).view(20000, 64, 32)
    p = torch.exp2(scales.double() - 127).unsqueeze(-1)
    assert torch.equal((v * p).view(20000, 2048), deq.double())
    y = (x.double().view(20000, 64, 32) / p)
    assert float(y.abs().max()) < 8 and float(y.abs().amax(-1).min()) >= 4
    step = torch.where(y.abs() < 2, 0.5, torch.where(y.abs() < 4, 1.0, 2.0))
    assert bool(((y - v).abs() <= torch.where(y.abs() > 6, 2.0, step / 2)).all())


# ------------------------------------------------------------------ product (GPU)

def _case(lens, N, K, gather, seed, T=None, alpha=False, pad=0):
    """Random MXFP4 operands over the given segment lengths."""
    g = torch.Generator().manual_seed(seed)
    G, M = len(lens), sum(lens) + pad
    R = (T or max(1, M // 2)) if gather else max(M, 1)
    ac = torch.randint(0, 256, (R, K // 2), generator=g, dtype=torch.uint8)
    asc = torch.randint(118, 131, (R, K // 32), generator=g, dtype=torch.uint8)
    wc = torch.randint(0, 256, (G, N, K // 2), generator=g, dtype=torch.uint8)
    wsc = torch.randint(116, 128, (G, N, K // 32), generator=g, dtype=torch.uint8)
    idx = torch.randint(0, R, (M,), generator=g, dtype=torch.int32) if gather else None
    al = torch.rand(G, generator=g) + 0.5 if alpha else None
    cu = torch.tensor(np.cumsum(lens), dtype=torch.int32)
    return ac, asc, wc, wsc, idx, al, cu, M


def _product(case, out=None):
    ac, asc, wc, wsc, idx, al, cu, M = case
    w = m.moe_prepare_weights(m.Weight("mxfp4", wc.cuda(), wsc.cuda(), None if al is None else al.cuda()))
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    got = m.moe_grouped_gemm_mxfp4(ac.cuda(), asc.cuda(), w, cu.cuda(), None if idx is None else idx.cuda(), out=out,
                                   ws=ws)
    torch.cuda.synchronize()
    return got, m.moe_get_device_error(ws)


def _reference(case):
    ac, asc, wc, wsc, idx, al, cu, M = case
    a = O.mxfp4_dequantize_rows(O.unpack_e2m1(ac.numpy()), asc.numpy())
    if idx is not None:
        i = idx.numpy()
        a = np.where(((i >= 0) & (i < len(a)))[:, None], a[np.clip(i, 0, len(a) - 1)], 0.0)
    N, K = wc.shape[1], ac.shape[1] * 2
    ref, mag = np.zeros((M, N)), np.zeros((M, N))
    lo = 0
    for g, hi in enumerate(cu.numpy()):
        if hi > lo:
            wv = O.mxfp4_dequantize_rows(O.unpack_e2m1(wc[g].numpy()), wsc[g].numpy()) * (1.0 if al is None else float(al[g]))
            ref[lo:hi] = a[lo:hi] @ wv.T
            mag[lo:hi] = np.abs(a[lo:hi]) @ np.abs(wv).T
        lo = hi
    return ref, (K / 64 + 1) * 2.0 ** -22 * mag


def _check_product(case, err=0):
    got, e = _product(case)
    assert e == err
    ref, slack = _reference(case)
    got = got.double().cpu().numpy()
    d = np.abs(got - ref)
    assert np.all(d <= slack + (np.abs(ref) + slack) * 2.0 ** -8), float((d / (np.abs(ref) + slack + 1e-30)).max())


LENS = {"one": [1], "ragged": [3, 0, 17, 1, 0, 130, 64, 0], "exact": [16, 32, 128, 256], "long": [513, 300],
        "empty": [0, 0, 0], "tail": [0, 191, 193, 7], "many": [1] * 40 + [0] * 23 + [2]}


@pytest.mark.gpu
@pytest.mark.parametrize("lens", sorted(LENS))
@pytest.mark.parametrize("N,K", [(128, 256), (8, 32), (200, 96), (136, 2880), (384, 1056)])
@pytest.mark.parametrize("gather", [False, True])
def test_product_matches_oracle(lens, N, K, gather):
    _check_product(_case(LENS[lens], N, K, gather, seed=N + K, alpha=True, pad=5))


@pytest.mark.gpu
@pytest.mark.parametrize("K", [32, 64, 128, 160, 224, 288, 480, 512, 544, 1024, 4096, 7168])
def test_product_every_tail_of_k(K):
    _check_product(_case([20, 5], 72, K, False, seed=K))
    _check_product(_case([20, 5], 72, K, True, seed=K))


@pytest.mark.gpu
def test_product_many_tiles():
    """More tiles than SMs, and several token tiles per weight block."""
    _check_product(_case([700, 0, 450, 1000, 30], 2176, 512, True, seed=1, T=900))
    _check_product(_case([40] * 64, 1160, 320, False, seed=2))


@pytest.mark.gpu
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("tile", ["16", "32", "64", "128", "pairs"])
@pytest.mark.parametrize("lens,N,K", [([1, 0, 37, 200, 16, 129, 0], 200, 544), ([385, 31, 250], 640, 1824)])
def test_product_every_tile(lens, N, K, tile, gather, monkeypatch):
    """Every token tile and the CTA pairs, on segments shorter and longer than the tile: an odd number
    of weight blocks, a ring of stages that turns several times, tiles that follow one another on an SM."""
    monkeypatch.setenv("MOE_GEMM_PAIRS", "1" if tile == "pairs" else "0")
    if tile != "pairs":
        monkeypatch.setenv("MOE_TOKEN_TILE", tile)
    _check_product(_case(lens, N, K, gather, seed=len(lens), alpha=True, pad=3))


@pytest.mark.gpu
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("pairs", ["0", "1"])
def test_product_same_bits_many_times(pairs, gather, monkeypatch):
    """Long runs of the pipeline, over and over: 16 stages a tile, many tiles an SM, the same bits each time."""
    monkeypatch.setenv("MOE_GEMM_PAIRS", pairs)
    case = _case([700, 513, 190, 64], 4096, 4096, gather, seed=21, T=800)
    ac, asc, wc, wsc, idx, al, cu, M = case
    w = m.moe_prepare_weights(m.Weight("mxfp4", wc.cuda(), wsc.cuda()))
    args = [t.cuda() for t in (ac, asc)] + [w, cu.cuda(), None if idx is None else idx.cuda()]
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    want = m.moe_grouped_gemm_mxfp4(*args, ws=ws)
    for _ in range(50):
        assert torch.equal(m.moe_grouped_gemm_mxfp4(*args, ws=ws), want)
    assert m.moe_get_device_error(ws) == 0
    rows = [0, 699, 700, 1212, 1300, M - 1]           # and sampled rows against 64 bits
    a = O.mxfp4_dequantize_rows(O.unpack_e2m1(ac.numpy()), asc.numpy())
    seg = np.searchsorted(cu.numpy(), rows, side="right")
    for r, g in zip(rows, seg):
        v = a[r if idx is None else int(idx[r])]
        wv = O.mxfp4_dequantize_rows(O.unpack_e2m1(wc[g].numpy()), wsc[g].numpy())
        ref, mag = wv @ v, np.abs(wv) @ np.abs(v)
        slack = (4096 / 64 + 1) * 2.0 ** -22 * mag
        assert np.all(np.abs(want[r].double().cpu().numpy() - ref) <= slack + (np.abs(ref) + slack) * 2.0 ** -8)


@pytest.mark.gpu
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("pairs", ["0", "1"])
def test_product_wait_limit(pairs, gather, monkeypatch):
    """A pipeline wait that runs out is reported, the kernel returns by itself, and the next call on the
    same workspace is right."""
    monkeypatch.setenv("MOE_GEMM_PAIRS", pairs)
    case = _case([200, 90], 384, 32768, gather, seed=6, T=250)   # an epilogue waits for 128 stages
    monkeypatch.setenv("MOE_WAIT_LIMIT_CYCLES", "1")
    _, e = _product(case)
    assert e == TIMEOUT
    monkeypatch.delenv("MOE_WAIT_LIMIT_CYCLES")
    _check_product(case)


@pytest.mark.gpu
@pytest.mark.parametrize("lens,gather", [([5, 40, 3], False), ([150, 260], True)])
def test_product_rows_behind_and_determinism(lens, gather):
    """Rows past the last segment come out zero, rows past M_alloc stay; two runs give the same bits."""
    case = _case(lens, 264, 352, gather, seed=9, pad=11)
    M, N = case[-1], 264
    buf = torch.full((M + 4, N), 7.0, dtype=torch.bfloat16, device="cuda")
    got, e = _product(case, out=buf[:M])
    again, _ = _product(case)
    assert e == 0 and torch.equal(got, again)
    assert bool((buf[M - 11:M] == 0).all()) and bool((buf[M:] == 7).all())


@pytest.mark.gpu
@pytest.mark.parametrize("lens", [[9, 20], [140, 250]])
def test_product_bad_row_indices_are_zero_rows_and_reported(lens):
    case = _case(lens, 128, 320, True, seed=4, T=30)
    idx = case[4]
    idx[0], idx[5], idx[-1], idx[12] = -1, 30, 2 ** 31 - 1, -2 ** 31
    _check_product(case, err=DEVICE)


@pytest.mark.gpu
@pytest.mark.parametrize("gather", [False, True])
def test_product_nan_scale_poisons_its_row_alone(gather):
    case = _case([40, 9], 136, 352, gather, seed=8, T=25)
    clean, _ = _product(case)
    row = 3
    case[1][row, 10] = 255
    got, _ = _product(case)
    rows = torch.arange(case[-1]) if case[4] is None else case[4]
    hit = (rows == row).cuda()
    assert bool(hit.any()) and bool(got[hit].isnan().all()) and torch.equal(got[~hit], clean[~hit])


@pytest.mark.gpu
def test_product_bad_segment_ends_are_reported():
    """Ends that fall or pass M_alloc are clamped, as in the other grouped products."""
    case = list(_case([10, 20, 30], 128, 64, False, seed=3))
    case[6] = torch.tensor([10, 5, 9999], dtype=torch.int32)
    got, e = _product(tuple(case))
    assert e == DEVICE and got.shape == (60, 128)


@pytest.mark.gpu
def test_product_graph_on_two_streams():
    """Captured once, replayed on new operands; and two calls with workspaces of their own on two
    streams at once."""
    cases = [_case([100, 60, 0, 33], 256, 416, True, seed=s, T=70) for s in (1, 2)]
    dev = [[None if t is None else t.cuda() for t in c[:7]] for c in cases]
    ws = [m.moe_prepare_weights(m.Weight("mxfp4", d[2], d[3])) for d in dev]
    outs = [torch.empty(193, 256, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    err = [torch.zeros(256, dtype=torch.uint8, device="cuda") for _ in range(2)]
    want = [_product(c)[0] for c in cases]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for i, st in enumerate(streams):
            m.moe_grouped_gemm_mxfp4(dev[i][0], dev[i][1], ws[i], dev[i][6], dev[i][4], outs[i], err[i], st)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want[0]) and torch.equal(outs[1], want[1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        m.moe_grouped_gemm_mxfp4(dev[0][0], dev[0][1], ws[0], dev[0][6], dev[0][4], outs[0], err[0])
    second = _case([100, 60, 0, 33], 256, 416, True, seed=5, T=70)
    for i in (0, 1, 4):
        dev[0][i].copy_(second[i])
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], _product(second[:2] + cases[0][2:4] + second[4:])[0])


def test_room_for_gathered_rows(monkeypatch):
    size = lambda M, w: L.moe_grouped_gemm_mxfp4_rows_size(M, None if w is None else ctypes.byref(w))
    monkeypatch.setenv("MOE_GEMM_PAIRS", "1")
    assert size(7, _w(K=96)) == 7 * (48 + 3)
    assert size(2 ** 31 - 1, _w(K=4096)) == (2 ** 31 - 1) * 2176
    assert size(0, _w()) == size(-1, _w()) == size(7, None) == size(7, _w(K=0)) == 0
    monkeypatch.setenv("MOE_GEMM_PAIRS", "0")
    assert size(7, _w(K=96)) == 0
    monkeypatch.setenv("MOE_TOKEN_TILE", "64")
    assert size(7, _w(K=96)) == 7 * (48 + 3)
    monkeypatch.delenv("MOE_TOKEN_TILE")
    monkeypatch.delenv("MOE_GEMM_PAIRS")
    assert size(7, _w(G=2, N=64)) == 0                # few rows: gathered by the product


@pytest.mark.gpu
@pytest.mark.parametrize("lens,N,K", [([3, 0, 200, 1, 391], 136, 32), ([130, 70], 264, 7200), ([5] * 77 + [0] * 9, 72, 480)])
@pytest.mark.parametrize("shift", [0, 1])
def test_product_rows_gathered_first(lens, N, K, shift, monkeypatch):
    """The gather before the CTA pairs: bad indices in the segments, arbitrary ones behind them, scales at
    an odd address, more segments than a warp has lanes."""
    monkeypatch.setenv("MOE_GEMM_PAIRS", "1")
    case = list(_case(lens, N, K, True, seed=K, T=50, pad=9))
    M, idx = case[-1], case[4]
    idx[M - 9:] = torch.tensor([-1, 50, 2 ** 31 - 1, -2 ** 31, 0, 49, 7, -5, 1000])
    _check_product(case)
    idx[0], idx[2], idx[M - 10] = -1, 50, 2 ** 31 - 1
    ac, asc, wc, wsc, idx, al, cu, M = case
    w = m.moe_prepare_weights(m.Weight("mxfp4", wc.cuda(), wsc.cuda()))
    sc = torch.zeros(asc.numel() + 8, dtype=torch.uint8, device="cuda")[shift:shift + asc.numel()].view(asc.shape)
    sc.copy_(asc)
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    got = m.moe_grouped_gemm_mxfp4(ac.cuda(), sc, w, cu.cuda(), idx.cuda(), ws=ws)
    torch.cuda.synchronize()
    assert m.moe_get_device_error(ws) == DEVICE
    ref, slack = _reference(case)
    assert np.all(np.abs(got.double().cpu().numpy() - ref) <= slack + (np.abs(ref) + slack) * 2.0 ** -8)


@pytest.mark.gpu
@pytest.mark.parametrize("tile", ["16", "32", "64", "128", "pairs"])
def test_product_without_room_gathers_as_it_goes(tile, monkeypatch):
    monkeypatch.setenv(*("MOE_GEMM_PAIRS", "1") if tile == "pairs" else ("MOE_TOKEN_TILE", tile))
    case = _case([150, 0, 260], 264, 352, True, seed=13, T=90, pad=4)
    case[4][5] = 90
    ac, asc, wc, wsc, idx, al, cu, M = [t.cuda() if torch.is_tensor(t) else t for t in case]
    w = m.moe_prepare_weights(m.Weight("mxfp4", wc, wsc))
    out = torch.empty(M, 264, dtype=torch.bfloat16, device="cuda")
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    st = L.moe_grouped_gemm_mxfp4(ac.data_ptr(), asc.data_ptr(), 90, idx.data_ptr(), M, ctypes.byref(w.desc), cu.data_ptr(),
                                  out.data_ptr(), None, ws.data_ptr(), 256, torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    ref, slack = _reference(case)
    assert st == 0 and m.moe_get_device_error(ws) == DEVICE
    assert np.all(np.abs(out.double().cpu().numpy() - ref) <= slack + (np.abs(ref) + slack) * 2.0 ** -8)


@pytest.mark.gpu
def test_product_rows_gathered_first_on_streams_and_in_graphs(monkeypatch):
    """The room belongs to the call: two streams at once, its memory reused on the current stream meanwhile,
    and two captured graphs replayed on new indices."""
    monkeypatch.setenv("MOE_GEMM_PAIRS", "1")
    cases = [_case([400, 60, 0, 333], 512, 2048, True, seed=s, T=300) for s in (1, 2)]
    dev = [[None if t is None else t.cuda() for t in c[:7]] for c in cases]
    ws = [m.moe_prepare_weights(m.Weight("mxfp4", d[2], d[3])) for d in dev]
    outs = [torch.empty(793, 512, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    err = [torch.zeros(256, dtype=torch.uint8, device="cuda") for _ in range(2)]
    want = [_product(c)[0] for c in cases]
    streams = [torch.cuda.Stream() for _ in range(2)]
    call = lambda i, st=None: m.moe_grouped_gemm_mxfp4(dev[i][0], dev[i][1], ws[i], dev[i][6], dev[i][4], outs[i], err[i], st)
    torch.cuda.synchronize()
    for _ in range(10):
        for i, st in enumerate(streams):
            call(i, st)
            torch.full((793 * 1088,), 255, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want[0]) and torch.equal(outs[1], want[1])
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for i, g in enumerate(graphs):
        with torch.cuda.graph(g):
            call(i)
    second = [_case([400, 60, 0, 333], 512, 2048, True, seed=s, T=300) for s in (5, 6)]
    for i in range(2):
        dev[i][4].copy_(second[i][4])
    for st, g in zip(streams, graphs):
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st):
            for _ in range(5):
                g.replay()
    torch.cuda.synchronize()
    for i in range(2):
        assert torch.equal(outs[i], _product(cases[i][:4] + second[i][4:5] + cases[i][5:])[0])


@pytest.mark.gpu
@pytest.mark.slow
def test_rows_past_32_bits_of_elements():
    """Codes, outputs and quantised values whose offsets pass 2^31 elements: the last rows against 64 bits."""
    K, N, M = 1024, 32768, 70000                      # out: 2.3e9 values
    row = torch.randn(M, K, device="cuda").bfloat16()
    codes, scales, _ = m.moe_quantize_mxfp4(row)
    wt = torch.randn(N, K, device="cuda").bfloat16()
    wc, wsc, _ = m.moe_quantize_mxfp4(wt)
    w = m.moe_prepare_weights(m.Weight("mxfp4", wc.view(1, N, -1), wsc.view(1, N, -1)))
    out = m.moe_grouped_gemm_mxfp4(codes, scales, w, torch.tensor([M], dtype=torch.int32, device="cuda"))
    u = lambda t: t.cpu().numpy()
    for r in (0, 65535, 65536, M - 1):
        a = O.mxfp4_dequantize_rows(O.unpack_e2m1(u(codes[r:r + 1])), u(scales[r:r + 1]))[0]
        wv = O.mxfp4_dequantize_rows(O.unpack_e2m1(u(wc[-256:])), u(wsc[-256:]))
        ref, mag = wv @ a, np.abs(wv) @ np.abs(a)
        slack = (K / 64 + 1) * 2.0 ** -22 * mag
        assert np.all(np.abs(out[r, -256:].double().cpu().numpy() - ref) <= slack + (np.abs(ref) + slack) * 2.0 ** -8)
    del out, row, codes
    R, K = 300000, 8192                               # 2.5e9 values in
    x = torch.randn(1, K, device="cuda").bfloat16().repeat(R, 1)
    x[-1] *= 3
    c, s, d = m.moe_quantize_mxfp4(x, deq=True)
    for r in (0, R - 2, R - 1):
        rc, rs = O.mxfp4_quantize_rows(x[r:r + 1].float().cpu().numpy())
        assert np.array_equal(u(c[r:r + 1]), _pack(rc)) and np.array_equal(u(s[r:r + 1]), rs)
        assert np.array_equal(d[r:r + 1].double().cpu().numpy(), O.mxfp4_dequantize_rows(rc, rs))
    n = m.moe_add_rmsnorm(x, quant="mxfp4")
    assert torch.equal(n["codes"][0], n["codes"][R - 2])
    _, y = O.add_rmsnorm(x[-1:].double().cpu().numpy())
    assert np.all(np.abs(n["y"][-1:].double().cpu().numpy() - y) <= np.abs(y) * (2.0 ** -8 + 1e-5) + 1e-38)


# ------------------------------------------------------------------ together (GPU)

@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 33, 400])
def test_expert_layer_in_four_bits(T):
    """Norm to MXFP4 rows, routing by scores, permutation, gate and up products that gather the token
    rows, activation, MXFP4 rows, down product, combine: every step against the oracle on the step's
    own inputs."""
    H, I, E, k = 256, 352, 16, 4
    g = torch.Generator().manual_seed(T)
    x, res = (torch.randn(T, H, generator=g).bfloat16().cuda() for _ in range(2))
    gain = (1 + 0.1 * torch.randn(H, generator=g)).bfloat16().cuda()
    router = (torch.randn(H, E, generator=g) / 16).cuda()
    bias = (0.02 * torch.randn(E, generator=g)).cuda()
    raw = {n: torch.randn(E, *s, generator=g) * 0.1 for n, s in (("gate", (I, H)), ("up", (I, H)), ("down", (H, I)))}
    w = {}
    for n, t in raw.items():  # bf16 weights into the MXFP4 format by the same quantiser
        c, s, _ = m.moe_quantize_mxfp4(t.bfloat16().cuda().view(-1, t.shape[2]))
        w[n] = m.moe_prepare_weights(m.Weight("mxfp4", c.view(E, t.shape[1], -1), s.view(E, t.shape[1], -1)))
    n = m.moe_add_rmsnorm(x, gain, res, quant="mxfp4")
    ids, tw = m.moe_route_scored(n["y"].float() @ router, k, "sigmoid", bias, 4, 2, "top2", True, 2.5)
    p = m.moe_permute(ids, tw, E)
    gate, up = (m.moe_grouped_gemm_mxfp4(n["codes"], n["scales"], w[q], p["cu_seqlens"], p["perm_token"])
                for q in ("gate", "up"))
    h = m.moe_act_and_mul(gate, up, p["perm_w"])
    hc, hs, _ = m.moe_quantize_mxfp4(h)
    y = m.moe_grouped_gemm_mxfp4(hc, hs, w["down"], p["cu_seqlens"])
    out = m.moe_combine(y, p["inv_perm"])
    torch.cuda.synchronize()
    assert m.moe_get_device_error(p["ws"]) == 0
    f = lambda t: t.double().cpu().numpy()
    u = lambda t: t.cpu().numpy()
    rids, rw = O.route_scored(f(n["y"].float() @ router), k, "sigmoid", f(bias), 4, 2, "top2", True, 2.5)
    assert np.array_equal(u(ids), rids)
    a = O.mxfp4_dequantize_rows(O.unpack_e2m1(u(n["codes"])), u(n["scales"]))
    hv = O.mxfp4_dequantize_rows(O.unpack_e2m1(u(hc)), u(hs))
    wv = {q: np.stack([O.mxfp4_dequantize_rows(O.unpack_e2m1(u(w[q].data[e])), u(w[q].scale[e])) for e in range(E)]) for q in w}
    for t in range(T):
        want, room = np.zeros(H), np.zeros(H)
        for j in range(k):
            e, r = int(rids[t, j]), int(p["inv_perm"][t, j])
            gm, um = (np.abs(a[t]) @ np.abs(wv[q][e]).T for q in ("gate", "up"))
            for got, q, mag in ((gate, "gate", gm), (up, "up", um)):
                ref = a[t] @ wv[q][e].T
                assert np.all(np.abs(f(got[r]) - ref) <= 2.0 ** -8 * np.abs(ref) + 1e-4 * mag)
            # the down product on the rows it was given
            ref = hv[r] @ wv["down"][e].T
            slack = (I / 64 + 1) * 2.0 ** -22 * (np.abs(hv[r]) @ np.abs(wv["down"][e]).T)
            want += ref
            room += slack + (np.abs(ref) + slack) * 2.0 ** -8
        assert np.all(np.abs(f(out[t]) - want) <= room + (np.abs(want) + room) * (2.0 ** -8 + 2.0 ** -22))
    ref_h = O.act_and_mul(f(gate), f(up), "silu") * f(p["perm_w"])[:, None]
    assert np.all(np.abs(f(h) - ref_h) <= (2.0 ** -8 + 1e-5) * np.abs(ref_h) + 1e-30)
    assert np.array_equal(u(hc), _pack(O.mxfp4_quantize_rows(f(h))[0]))
