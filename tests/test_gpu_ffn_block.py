"""The operators of a feed-forward block together, as a program uses them: y = x + Wd . (act(Wg n)
* (Wu n)), n = LN(x), forward and backward, each stage against 64-bit products of what the stage
before it gave; captured into a graph and replayed, on other streams, side by side, and with
operands of the smallest alignment that the entry points allow."""
import numpy as np
import pytest
import torch

import block_scaled_fp4_04_b200 as fp4
import oracle
from ffn_testutil import (MAX_SLOPE, act64, act_error, assert_close, assert_codes_of, dequantized, product64)
from fp4_testutil import gpu_quantize, random_input

pytestmark = pytest.mark.gpu
EPS = 1e-5


def _block(m, k, f, seed=0):
    x = random_input(m, k, 100 + seed, torch.bfloat16, outliers=False)
    w, b = (torch.randn(k, generator=torch.Generator().manual_seed(s)) * 0.2 + c for s, c in ((1, 1.0), (2, 0.0)))
    wg, wu, wd = (random_input(r, c, s, torch.float32, std=0.06, outliers=False) for r, c, s in ((f, k, 3), (f, k, 4), (k, f, 5)))
    return x.cuda(), w.cuda(), b.cuda(), wg.cuda(), wu.cuda(), wd.cuda()


def _forward(x, w, b, qg, qu, qd, g_n, g_h, ws):
    n, mean, rstd = fp4.layernorm(x, w, b, EPS, fmt=fp4.NVFP4, global_in=g_n)
    h, g, u = fp4.gemm_gated(n, qg, qu, fp4.ACT_SILU, save=True, quantized_out=g_h, workspace=ws)
    y = fp4.gemm_epilogue(h, qd, residual=x, workspace=ws)
    return n, mean, rstd, h, g, u, y


@pytest.mark.parametrize("m,k,f", [(1, 256, 512), (16, 512, 1024), (130, 256, 544), (300, 512, 9600)])
def test_block_forward_and_backward(m, k, f):
    x, w, b, wg, wu, wd = _block(m, k, f)
    f2, k2 = f - f % 32, k
    # weights quantized once in 16 x 16 blocks: the transposes serve the backward pass
    stacked = fp4.quantize(torch.cat((wg, wu)), fp4.NVFP4, 256)
    qg, qu = fp4.quantize(wg, fp4.NVFP4, 256), fp4.quantize(wu, fp4.NVFP4, 256)
    qd = fp4.quantize(wd, fp4.NVFP4, 256)
    ws = fp4.Workspace()
    # calibration: amax of the norm's and of the gated product's results
    amax = torch.empty(1, device="cuda")
    y32 = torch.empty(m, k, device="cuda")
    fp4.fp4_layernorm(x, m, k, fp4.BF16, w, b, EPS, y32, fp4.F32, amax_out=amax)
    assert amax.item() == y32.abs().max().item()
    g_n, g_h = torch.empty(1, device="cuda"), torch.tensor([0.01], device="cuda")
    fp4.fp4_global_scale(amax, g_n)
    n, mean, rstd, h, g, u, y = _forward(x, w, b, qg, qu, qd, g_n, g_h, ws)
    torch.cuda.synchronize()
    assert fp4.fp4_get_status() == fp4.OK
    assert_codes_of(n.codes, n.scales, g_n, y32, fp4.NVFP4, "norm")
    a = dequantized(n)
    g64, eg = product64(a, dequantized(qg))
    u64, eu = product64(a, dequantized(qu))
    assert_close(g, g64, eg, "G")
    assert_close(u, u64, eu, "U")
    # H's codes: within half an E2M1 step of H, plus what the FP32 H and the block scale may be off
    v, _ = act64(g64, "silu")
    h64 = v * u64
    eh = (MAX_SLOPE * eg + act_error(g64, v)) * u64.abs() + eu * v.abs()
    hv = torch.from_numpy(dequantized(h))
    step = h64.abs().view(m, -1, 16).amax(2, keepdim=True).expand(m, f // 16, 16).reshape(m, f) / 6.0
    # the largest gap (4 to 6) has two units of the scale; the E4M3 scale is within 1/16 of amax / 6
    # (or 2^-10 of g where it is subnormal), and a value above 6 units saturates
    assert ((hv - h64).abs() <= step * 1.5 + eh + 0.01 * 2.0 ** -6 * 6).all()
    y64, ey = product64(hv.numpy(), dequantized(qd))
    t64 = y64 + x.cpu().double()
    assert_close(y, t64, ey + 2.0 ** -23 * t64.abs(), "y")

    # backward from dy
    dy = random_input(m, k, 7, torch.bfloat16, outliers=False).cuda()
    qdy = fp4.quantize(dy, fp4.NVFP4, 16)
    dh = fp4.gemm(qdy, fp4.transposed(qd))
    dh64, e = product64(dequantized(qdy), dequantized(fp4.transposed(qd)))
    assert_close(dh, dh64, e, "dH")
    dz, dbias = fp4.act_backward(dh, g, u, fp4.ACT_SILU, dbias=True)
    gd, ud, dhd = (t.cpu().double() for t in (g, u, dh))
    vv, slope = act64(gd, "silu")
    z64 = torch.cat((dhd * ud * slope, dhd * vv), 1)
    err = torch.cat(((dhd * ud).abs() * (act_error(gd, torch.ones_like(gd)) * (1 + gd.abs())),
                     dhd.abs() * act_error(gd, vv)), 1) + 2.0 ** -22 * z64.abs()
    assert_close(dz, z64, err, "dZ")
    assert_close(dbias, z64.sum(0), err.sum(0) + (m + 72) * 2.0 ** -24 * z64.abs().sum(0), "bias gradients")
    qz = fp4.quantize(dz, fp4.NVFP4, 16)
    dn = fp4.gemm(qz, fp4.transposed(stacked))
    dn64, e = product64(dequantized(qz), dequantized(fp4.transposed(stacked)))
    assert_close(dn, dn64, e, "dn")
    dx, dw, db = fp4.layernorm_backward(dn, x, w, mean, rstd, dres=dy)
    dnd, xd, md, rd = (t.cpu().double() for t in (dn, x, mean, rstd))
    xh = (xd - md[:, None]) * rd[:, None]
    aw = dnd * w.cpu().double()
    c1, c2 = aw.mean(1, keepdim=True), (aw * xh).mean(1, keepdim=True)
    dx64 = rd[:, None] * (aw - c1 - xh * c2) + dy.cpu().double()
    ex = rd[:, None] * 2.0 ** -17 * (aw.abs() + aw.abs().mean(1, keepdim=True) + xh.abs() * (aw * xh).abs().mean(1, keepdim=True))
    assert_close(dx, dx64, ex + 2.0 ** -23 * dx64.abs(), "dx")
    for got, terms in ((dw, dnd * xh), (db, dnd)):
        assert_close(got, terms.sum(0), (m + 40) * 2.0 ** -23 * terms.abs().sum(0), "norm parameters")
    torch.cuda.synchronize()
    assert fp4.fp4_get_status() == fp4.OK
    assert (f2, k2) == (f, k)


def _same_but_for_the_order_of_sums(a, b):
    """The down projection is split over K here and its FP32 partial sums meet in any order: the
    BF16 results differ by a rounding step at most, and hardly ever."""
    d = (a.double() - b.double()).abs()
    assert (d <= 2.0 ** -7 * torch.maximum(a.double().abs(), b.double().abs()) + 1e-6).all()
    assert (d != 0).double().mean() < 0.01


def test_block_captured_and_replayed():
    """One graph of the whole forward pass, replayed on other inputs, gives what the calls give."""
    m, k, f = 300, 512, 9600
    x, w, b, wg, wu, wd = _block(m, k, f)
    qg, qu, qd = (fp4.quantize(t, fp4.NVFP4, 16) for t in (wg, wu, wd))
    g_n, g_h = (torch.tensor([v], device="cuda") for v in (0.003, 0.01))
    ws = fp4.Workspace()
    _forward(x, w, b, qg, qu, qd, g_n, g_h, ws)  # first call outside the capture
    torch.cuda.synchronize()
    graph, static = torch.cuda.CUDAGraph(), x.clone()
    with torch.cuda.graph(graph):
        out = _forward(static, w, b, qg, qu, qd, g_n, g_h, ws)
        dz = fp4.act_backward(out[4], out[4], out[5], fp4.ACT_SILU, dbias=True)
        dx = fp4.layernorm_backward(static, static, w, out[1], out[2])
    for seed in (1, 2):
        x2 = random_input(m, k, 200 + seed, torch.bfloat16, outliers=False).cuda()
        static.copy_(x2)
        graph.replay()
        want = _forward(x2, w, b, qg, qu, qd, g_n, g_h, fp4.Workspace())
        wz = fp4.act_backward(want[4], want[4], want[5], fp4.ACT_SILU, dbias=True)
        wx = fp4.layernorm_backward(x2, x2, w, want[1], want[2])
        torch.cuda.synchronize()
        assert torch.equal(out[0].codes, want[0].codes) and torch.equal(out[0].scales, want[0].scales)
        assert torch.equal(out[4], want[4]) and torch.equal(out[5], want[5])
        assert torch.equal(out[3].codes, want[3].codes)
        _same_but_for_the_order_of_sums(out[6], want[6])
        for p, q in zip(dz + dx, wz + wx):
            assert torch.equal(p, q)
    assert fp4.fp4_get_status() == fp4.OK


def test_decode_captured_and_replayed_with_its_workspace():
    """The single-launch decode keeps a counter in its workspace: replays and eager calls in turn."""
    m, f, k = 5, 640, 2048
    x = random_input(m, k, 1, torch.bfloat16).cuda()
    qg, qu = (gpu_quantize(random_input(f, k, s, torch.float32, std=0.05, outliers=False).cuda(), fp4.NVFP4, 16) for s in (2, 3))
    ws = torch.zeros(fp4.fp4_gemm_gated_bf16a_workspace_size(m, f, k), dtype=torch.uint8, device="cuda")
    h = torch.empty(m, f, device="cuda")
    xc = torch.empty(m, k // 2, dtype=torch.uint8, device="cuda")
    xs = torch.empty(fp4.fp4_scales_bytes(m, k, fp4.NVFP4), dtype=torch.uint8, device="cuda")
    xg = torch.empty(1, device="cuda")

    def call():
        fp4.fp4_gemm_gated_bf16a(x, qg.codes, qg.scales, qg.g, qu.codes, qu.scales, qu.g, m, f, k, None, None,
                                 fp4.ACT_SILU, h, fp4.F32, None, None, xc, xs, xg, ws, ws.numel())

    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for i in range(4):
        x.copy_(random_input(m, k, 10 + i, torch.bfloat16))
        h.fill_(float("nan"))
        graph.replay() if i % 2 else call()
        torch.cuda.synchronize()
        a = dequantized(fp4.Quantized(xc, xs, xg, m, k, fp4.NVFP4))
        g64, eg = product64(a, dequantized(qg))
        u64, eu = product64(a, dequantized(qu))
        v, _ = act64(g64, "silu")
        assert_close(h, v * u64, (MAX_SLOPE * eg + act_error(g64, v)) * u64.abs() + eu * v.abs() + 2.0 ** -22 * (v * u64).abs())
    assert fp4.fp4_get_status() == fp4.OK


def test_other_streams_and_calls_side_by_side():
    """Two blocks on two streams at once, each with its own workspace, behind long-running work on
    their streams: the same bits as one after the other."""
    m, k, f = 300, 512, 9600
    blocks = [_block(m, k, f, seed) for seed in (0, 1)]
    g_n, g_h = (torch.tensor([v], device="cuda") for v in (0.003, 0.01))
    qs = [[fp4.quantize(t, fp4.NVFP4, 16) for t in bl[3:]] for bl in blocks]
    want = [_forward(*bl[:3], *q, g_n, g_h, fp4.Workspace()) for bl, q in zip(blocks, qs)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in blocks]
    spaces = [fp4.Workspace() for _ in blocks]
    big = torch.randn(4096, 4096, device="cuda")
    torch.cuda.synchronize()
    got = [None, None]
    for i, st in enumerate(streams):
        with torch.cuda.stream(st):
            late = torch.zeros_like(blocks[i][0])
            big @ big
            late.copy_(blocks[i][0])  # the input is only there once the product before it is done
            got[i] = _forward(late, *blocks[i][1:3], *qs[i], g_n, g_h, spaces[i])
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        for i in (1, 2, 4, 5):
            assert torch.equal(a[i], b[i])
        _same_but_for_the_order_of_sums(a[6], b[6])
        assert torch.equal(a[0].codes, b[0].codes) and torch.equal(a[3].codes, b[3].codes)
    # a stream given to a call: outputs belong to it
    st = streams[0]
    y, mean, rstd = fp4.layernorm(blocks[0][0], blocks[0][1], blocks[0][2], EPS, stream=st)
    st.synchronize()
    z, _, _ = fp4.layernorm(blocks[0][0], blocks[0][1], blocks[0][2], EPS)
    z2, _, _ = fp4.layernorm(blocks[0][0], blocks[0][1], blocks[0][2], EPS, stream=st.cuda_stream)
    torch.cuda.synchronize()
    assert torch.equal(y, z) and torch.equal(y, z2)
    assert fp4.fp4_get_status() == fp4.OK


def test_one_workspace_for_all():
    """Calls that share one zero-filled workspace one after the other leave it so, the backward
    passes with their partial sums among them."""
    m, k, f = 16, 2048, 512
    x = random_input(m, k, 1, torch.bfloat16).cuda()
    qx = fp4.quantize(x, fp4.NVFP4, 16)
    qg, qu = (gpu_quantize(random_input(f, k, s, torch.float32, std=0.05, outliers=False).cuda(), fp4.NVFP4, 16) for s in (2, 3))
    ws = fp4.Workspace()
    buf = ws.get(1 << 26)
    first = fp4.gemm_gated(qx, qg, qu, workspace=ws, out_dtype=torch.float32)
    mean, rstd = x.float().mean(1), torch.ones(m, device="cuda")
    dx = torch.empty_like(x)
    dw = torch.empty(k, device="cuda")
    fp4.fp4_layernorm_backward(x, x, m, k, fp4.BF16, None, mean, rstd, None, dx, fp4.BF16, dw, None, buf, buf.numel())
    z, db = torch.empty_like(x), torch.empty(k, device="cuda")
    fp4.fp4_act_backward(x, x, None, m, k, fp4.BF16, fp4.ACT_GELU, z, fp4.BF16, db, workspace=buf,
                         workspace_bytes=buf.numel())
    torch.cuda.synchronize()
    assert not buf.any()
    again = fp4.gemm_gated(qx, qg, qu, workspace=ws, out_dtype=torch.float32)
    torch.cuda.synchronize()
    assert not buf.any() and fp4.fp4_get_status() == fp4.OK
    assert torch.allclose(first, again, rtol=1e-5, atol=1e-5 * first.abs().max().item())


@pytest.mark.parametrize("m,f,k,dtype", [(300, 9600, 64, torch.bfloat16), (300, 9604, 64, torch.float32),
                                         (300, 9608, 64, torch.bfloat16), (40, 640, 2048, torch.bfloat16)])
def test_smallest_alignment(m, f, k, dtype):
    """Outputs and residual 16-byte, biases 4-byte aligned and no more."""
    qa = gpu_quantize(random_input(m, k, 1, torch.bfloat16).cuda(), fp4.NVFP4, 16)
    qg, qu = (gpu_quantize(random_input(f, k, s, torch.float32, std=0.1, outliers=False).cuda(), fp4.NVFP4, 16) for s in (2, 3))
    pad = 16 // torch.empty(0, dtype=dtype).element_size()
    flat = [torch.full((m * f + 2 * pad,), 7.0, dtype=dtype, device="cuda") for _ in range(4)]
    h, g, u, r = (t[pad:-pad] for t in flat)
    r.copy_(random_input(1, m * f, 4, dtype, outliers=False)[0])
    bias = torch.randn(f + 1, generator=torch.Generator().manual_seed(5)).cuda()[1:]
    need = max(fp4.fp4_gemm_gated_workspace_size(m, f, k, fp4.NVFP4, False),
               fp4.fp4_gemm_epilogue_workspace_size(m, f, k, fp4.NVFP4, False))
    ws = torch.zeros(max(16, need), dtype=torch.uint8, device="cuda")
    oc = fp4.BF16 if dtype == torch.bfloat16 else fp4.F32
    fp4.fp4_gemm_gated(fp4.NVFP4, qa.codes, qa.scales, qa.g, qg.codes, qg.scales, qg.g, qu.codes, qu.scales, qu.g, m, f, k,
                       bias, bias, fp4.ACT_SILU, h, oc, g, u, workspace=ws, workspace_bytes=need)
    torch.cuda.synchronize()
    a = dequantized(qa)
    z = []
    for q, out in ((qg, g), (qu, u)):
        p, e = product64(a, dequantized(q))
        z.append((p + bias.cpu().double(), e + 2.0 ** -22 * (p.abs() + bias.cpu().double().abs())))
        assert_close(out.view(m, f), *z[-1])
    v, _ = act64(z[0][0], "silu")
    assert_close(h.view(m, f), v * z[1][0], (MAX_SLOPE * z[0][1] + act_error(z[0][0], v)) * z[1][0].abs() + z[1][1] * v.abs()
                 + 2.0 ** -22 * (v * z[1][0]).abs())
    want = z[0][0] + r.cpu().double().view(m, f)
    fp4.fp4_gemm_epilogue_ex(fp4.NVFP4, qa.codes, qa.scales, qa.g, qg.codes, qg.scales, qg.g, m, f, k, bias, fp4.ACT_NONE, r,
                             oc, r, oc, g, workspace=ws, workspace_bytes=need)
    torch.cuda.synchronize()
    assert_close(r.view(m, f), want, z[0][1] + 2.0 ** -22 * want.abs())
    assert_close(g.view(m, f), *z[0])
    for t in flat:
        assert (t[:pad] == 7.0).all() and (t[-pad:] == 7.0).all(), "written outside"
    assert fp4.fp4_get_status() == fp4.OK


def test_norm_with_unaligned_parameters():
    m, n = 33, 1024
    x = random_input(m, n, 1, torch.bfloat16, outliers=False).cuda()
    w, b = (torch.randn(n + 1, generator=torch.Generator().manual_seed(s)).cuda()[1:] for s in (1, 2))
    y, y2 = torch.empty(m, n, device="cuda"), torch.empty(m, n, device="cuda")
    fp4.fp4_layernorm(x, m, n, fp4.BF16, w, b, EPS, y, fp4.F32)
    fp4.fp4_layernorm(x, m, n, fp4.BF16, w.clone(), b.clone(), EPS, y2, fp4.F32)
    torch.cuda.synchronize()
    assert torch.allclose(y, y2, rtol=1e-5, atol=1e-5)


def test_negative_zero_and_extremes_through_the_epilogue():
    """Zero sums stay zero (SILU(0) U = 0), and sums of hundreds saturate to x or 0, not NaN."""
    m, f, k = 128, 128, 64
    one = np.full((f, k // 2), 0x22, np.uint8)          # every element 1.0
    sc = oracle.swizzle_scales(np.full((f, k // 16), 0x38, np.uint8))
    dev = [torch.from_numpy(t).cuda() for t in (one, sc)]
    for g in (0.0, 8.0, -8.0):
        gs = torch.tensor([g], device="cuda")
        h, gg, uu = (torch.empty(m, f, device="cuda") for _ in range(3))
        for act, hi, lo in ((fp4.ACT_SILU, 512.0, 0.0), (fp4.ACT_GELU, 512.0, 0.0), (fp4.ACT_GELU_TANH, 512.0, 0.0)):
            fp4.fp4_gemm_gated(fp4.NVFP4, dev[0], dev[1], None, dev[0], dev[1], gs, dev[0], dev[1], None, m, f, k, None, None,
                               act, h, fp4.F32, gg, uu)
            torch.cuda.synchronize()
            assert (gg == g * k).all() and (uu == k).all()
            want = 0.0 if g <= 0 else g * k * k
            assert (h == want).all(), (act, g, h[0, 0].item())
