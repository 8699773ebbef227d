"""A mixture-of-experts block on the GPU, from the router's choices to the summed tokens, as a program
runs it: in MXFP4 (gated experts) and in 8-bit integers, with slots that have no expert, eager and
replayed from a graph.  Each step is checked against 64 bits on what the step before it gave."""
import numpy as np
import pytest
import torch

import block_scaled_fp4_04_b200 as fp4
import oracle
from ffn_testutil import act64, assert_close, product64
from fp4_testutil import gpu_quantize, random_input
from moe_testutil import combine64, i8_rows, product_i8, router_ids, sort_reference

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def _grouped_values(q: fp4.Quantized, offsets, srow_of_row):
    """Values of MXFP4 rows with scales in the grouped layout."""
    blocks = q.cols // 32
    rows = q.scales.numel() // (-(-blocks // 4) * 4)
    sc = oracle.unswizzle_scales(q.scales.cpu().numpy(), rows, blocks)
    n = int(offsets[-1])
    return oracle.dequantize(q.codes[:n].cpu().numpy(), sc[srow_of_row[:n]], 1.0, fp4.MXFP4)


@pytest.mark.parametrize("tokens,topk,experts,width,inner,drop", [(16, 4, 8, 256, 128, 0.0), (200, 3, 5, 384, 160, 0.3),
                                                                (1, 2, 4, 512, 384, 0.0)])
def test_gated_experts_in_mxfp4(tokens, topk, experts, width, inner, drop):
    ids = router_ids(tokens, topk, experts, 3, drop)
    offsets, row_of, srow = sort_reference(ids, experts)
    n, rows = int(offsets[-1]), tokens * topk
    srow_of_row = np.zeros(rows, np.int64)
    on = (row_of >= 0).numpy()
    srow_of_row[row_of.numpy()[on]] = srow.numpy()[on]
    x = random_input(tokens, width, 1, BF16)
    w = torch.rand(tokens, topk, generator=torch.Generator().manual_seed(2))
    gate, up, down = ([gpu_quantize(random_input(*s, 10 * k + e, F32, std=0.05, outliers=False).cuda(), fp4.MXFP4, 32)
                       for e in range(experts)]
                      for k, s in enumerate([(inner, width), (inner, width), (width, inner)]))
    stack = [(torch.stack([q.codes for q in qs]), torch.cat([q.scales for q in qs])) for qs in (gate, up, down)]
    ids_d, x_d, w_d = ids.cuda(), x.cuda(), w.cuda()

    def block():
        r = fp4.moe_sort(ids_d, experts)
        a = fp4.moe_dispatch(x_d, r, fp4.MXFP4)
        h = torch.full((rows, inner), float("nan"), dtype=BF16, device="cuda")
        fp4.fp4_gemm_gated_grouped(fp4.MXFP4, experts, r.offsets, a.codes, a.scales, None, *stack[0], None, *stack[1], None,
                                   rows, inner, width, None, None, fp4.ACT_SILU, h, fp4.BF16)
        hc = torch.zeros(rows, inner // 2, dtype=torch.uint8, device="cuda")
        hs = torch.empty(fp4.fp4_scales_bytes_grouped(rows, experts, inner, fp4.MXFP4), dtype=torch.uint8, device="cuda")
        fp4.fp4_quantize_grouped(h, rows, inner, fp4.BF16, fp4.MXFP4, experts, r.offsets, hc, hs, None)
        y = torch.full((rows, width), float("nan"), dtype=BF16, device="cuda")
        fp4.fp4_gemm_grouped(fp4.MXFP4, experts, r.offsets, hc, hs, None, *stack[2], None, rows, width, inner, y, fp4.BF16)
        out = fp4.moe_combine(y, r, w_d, residual=x_d)
        return r, a, h, fp4.Quantized(hc, hs, None, rows, inner, fp4.MXFP4), y, out

    r, a, h, hq, y, out = block()
    torch.cuda.synchronize()
    assert fp4.fp4_get_status() == fp4.OK
    assert torch.equal(r.row_of.cpu(), row_of)
    assert torch.isnan(h[n:]).all() and torch.isnan(y[n:]).all(), "rows behind the last expert's"
    av, hv = _grouped_values(a, offsets, srow_of_row), _grouped_values(hq, offsets, srow_of_row)

    def weight(qs, e):
        q = qs[e]
        return oracle.dequantize(q.codes.cpu().numpy(), oracle.unswizzle_scales(q.scales.cpu().numpy(), q.rows, q.cols // 32),
                                 1.0, fp4.MXFP4)

    for e in range(experts):
        lo, hi = int(offsets[e]), int(offsets[e + 1])
        if lo == hi:
            continue
        g, eg = product64(av[lo:hi], weight(gate, e))
        u, eu = product64(av[lo:hi], weight(up, e))
        act, _ = act64(g, "silu")
        # the slope of SILU is at most 1.1, its own error 2^-20 of it and 2^-22 (|g| + 1) in all
        err = 1.13 * eg * (u.abs() + eu) + act.abs() * eu + (2.0 ** -19 * act.abs() + 2.0 ** -22 * (g.abs() + 1)) * u.abs()
        assert_close(h[lo:hi], act * u, err, f"gated, expert {e}")
        d, ed = product64(hv[lo:hi], weight(down, e))
        assert_close(y[lo:hi], d, ed, f"down, expert {e}")
    want, mag = combine64(torch.nan_to_num(y.cpu()), row_of, w, x)
    assert_close(out, want, (topk + 1) * 2.0 ** -24 * mag, "combine")

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        again = block()
    x2 = random_input(tokens, width, 7, BF16).cuda()
    for xs in (x2, x.cuda()):
        x_d.copy_(xs)
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(again[-1], out)


@pytest.mark.parametrize("tokens,topk,experts,width,inner,drop", [(16, 4, 32, 288, 512, 0.0), (500, 3, 5, 160, 272, 0.3),
                                                                (1, 2, 4, 512, 384, 0.0), (900, 8, 8, 128, 256, 0.1)])
def test_experts_in_8_bits(tokens, topk, experts, width, inner, drop):
    ids = router_ids(tokens, topk, experts, 3, drop)
    offsets, row_of, _ = sort_reference(ids, experts)
    n, rows = int(offsets[-1]), tokens * topk
    x = random_input(tokens, width, 1, BF16)
    w = torch.rand(tokens, topk, generator=torch.Generator().manual_seed(2))
    up_w, down_w = random_input(experts * inner, width, 4, F32, std=0.05), random_input(experts * width, inner, 5, F32, std=0.05)
    up = fp4.quantize_i8(up_w.view(experts, inner, width).cuda())
    down = fp4.quantize_i8(down_w.view(experts, width, inner).cuda())
    bias = torch.randn(experts, inner, generator=torch.Generator().manual_seed(6)) * 0.1
    ids_d, x_d, w_d, b_d = ids.cuda(), x.cuda(), w.cuda(), bias.cuda()
    ws = fp4.Workspace()

    def block():
        r = fp4.moe_sort(ids_d, experts)
        a = fp4.moe_dispatch_i8(x_d, r)
        h = torch.full((rows, inner), float("nan"), dtype=BF16, device="cuda")
        fp4.gemm_i8(a, up, b_d, fp4.ACT_SILU, offsets=r.offsets, workspace=ws, out=h)
        hq = fp4.quantize_i8(h, r.offsets)
        y = fp4.gemm_i8(hq, down, out_dtype=F32, offsets=r.offsets, workspace=ws)
        return r, a, h, hq, y, fp4.moe_combine(y, r, w_d, residual=x_d, out_dtype=BF16)

    r, a, h, hq, y, out = block()
    torch.cuda.synchronize()
    assert fp4.fp4_get_status() == fp4.OK, "rows behind the last expert's, which hold NaN, are not quantized"
    assert torch.isnan(h[n:]).all()
    want_q, want_s = i8_rows(h[:n].cpu())
    assert torch.equal(hq.codes[:n].cpu(), want_q) and torch.equal(hq.scales[:n].cpu(), want_s)
    ac, as_, hc, hs = a.codes.cpu(), a.scales.cpu(), hq.codes.cpu(), hq.scales.cpu()
    upc, ups, dnc, dns = up.codes.cpu(), up.scales.cpu(), down.codes.cpu(), down.scales.cpu()
    for e in range(experts):
        lo, hi = int(offsets[e]), int(offsets[e + 1])
        if lo == hi:
            continue
        want, err = product_i8(ac[lo:hi], as_[lo:hi], upc[e], ups[e], bias[e], "silu")
        assert_close(h[lo:hi], want, err, f"up, expert {e}")
        want, err = product_i8(hc[lo:hi], hs[lo:hi], dnc[e], dns[e])
        assert_close(y[lo:hi], want, err, f"down, expert {e}")
    live = y.clone()
    live[n:] = 0
    want, mag = combine64(live.cpu(), row_of, w, x)
    assert_close(out, want, (topk + 1) * 2.0 ** -24 * mag, "combine")

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        again = block()
    x2 = random_input(tokens, width, 7, BF16).cuda()
    for xs in (x2, x.cuda(), x2, x.cuda()):
        x_d.copy_(xs)
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(again[-1], out)
    assert not ws.buf.any()


@pytest.mark.parametrize("fmt", [fp4.NVFP4, fp4.MXFP4])
@pytest.mark.parametrize("rows,behind,experts,cols", [(300, 77, 4, 96), (128, 128, 3, 64), (1000, 1, 40, 2048)])
def test_grouped_quantizer_leaves_rows_behind_the_last_expert(fmt, rows, behind, experts, cols):
    n = rows - behind
    cuts = sorted(torch.randint(0, n + 1, (experts - 1,), generator=torch.Generator().manual_seed(1)).tolist())
    off = torch.tensor([0, *cuts, n], dtype=torch.int32, device="cuda")
    x = random_input(rows, cols, 3, BF16).cuda()
    bad = x.clone()
    bad[n:] = float("nan")
    g = torch.tensor([1e-3], device="cuda")
    got = []
    for src in (bad, x):
        codes = torch.full((rows, cols // 2), 0x5A, dtype=torch.uint8, device="cuda")
        scales = torch.full((fp4.fp4_scales_bytes_grouped(rows, experts, cols, fmt),), 0xA5, dtype=torch.uint8, device="cuda")
        gout = torch.empty(1, device="cuda")
        fp4.fp4_quantize_grouped(src, rows, cols, fp4.BF16, fmt, experts, off, codes, scales, gout, g)
        assert fp4.fp4_get_status() == fp4.OK
        assert (codes[n:] == 0x5A).all()
        got.append((codes, scales))
    assert all(torch.equal(a, b) for a, b in zip(*got))
