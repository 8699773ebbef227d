"""The gated GEMM (dense, decode, from BF16, by experts) and the epilogue with activation,
residual and pre-activation, against 64-bit products of the dequantized operands."""
import numpy as np
import pytest
import torch

import block_scaled_fp4_04_b200 as fp4
import oracle
from ffn_testutil import (ACTS, CODE, MAX_SLOPE, act64, act_error, assert_close, assert_codes_of, codes_like, dequantized,
                          product64)
from fp4_testutil import assert_quant_equal, gpu_quantize, oracle_quantize, random_input

pytestmark = pytest.mark.gpu


def _blk(fmt):
    return 16 if fmt == fp4.NVFP4 else 32


def _bias(n, seed):
    return torch.from_numpy((np.random.default_rng(seed).standard_normal(n) * 0.7).astype(np.float32))


def _linear64(a, b, bias):
    z, e = product64(a, b)
    if bias is not None:
        z = z + bias.double()
    return z, e + 2.0 ** -23 * z.abs() + 2.0 ** -24 * (bias.double().abs() if bias is not None else 0.0)


def _gated64(g, eg, u, eu, act):
    v, _ = act64(g, act)
    slope = 1.0 if act in ("none", "relu") else MAX_SLOPE
    ev = slope * eg + act_error(g, v)
    return v * u, ev * u.abs() + eu * v.abs() + ev * eu + 2.0 ** -23 * (v * u).abs()


GATED = [
    # m, f, k, fmt: the path it takes
    (1, 64, 32, fp4.NVFP4),          # decode kernel, one K step, one partial tile
    (1, 1000, 2080, fp4.NVFP4),      # decode, ragged last weight tile, K tail
    (16, 1024, 2048, fp4.NVFP4),     # decode
    (7, 515, 4096, fp4.NVFP4),       # decode, odd F and M
    (32, 384, 8192, fp4.NVFP4),      # decode, 32 rows
    (5, 96, 64, fp4.MXFP4),          # general kernel, one partial tile
    (16, 512, 2880, fp4.MXFP4),      # stream-K
    (33, 640, 2048, fp4.NVFP4),      # stream-K, 33 rows
    (130, 257, 1056, fp4.NVFP4),     # stream-K, odd F, ragged rows
    (200, 333, 96, fp4.MXFP4),       # whole tiles, ragged columns
    (300, 9600, 256, fp4.NVFP4),     # CTA pairs, ragged rows
    (2560, 2000, 512, fp4.MXFP4),    # CTA pairs, ragged columns
    (2560, 2048, 320, fp4.NVFP4),    # CTA pairs, K tail
    (129, 19000, 64, fp4.NVFP4),     # single CTAs, whole tiles
]


@pytest.mark.parametrize("m,f,k,fmt", GATED)
@pytest.mark.parametrize("out,act,save,bias", [(torch.float32, "silu", True, True), (torch.bfloat16, "gelu_tanh", False, False),
                                               (torch.bfloat16, "gelu", True, False), (torch.float32, "relu", False, True),
                                               (torch.float32, "none", False, False)])
def test_gemm_gated(m, f, k, fmt, out, act, save, bias):
    xa = random_input(m, k, m + 7 * k, torch.bfloat16)
    wg, wu = (random_input(f, k, f + s, torch.float32, std=0.05, outliers=False) for s in (11, 12))
    qa, qg, qu = (gpu_quantize(t.cuda(), fmt, _blk(fmt)) for t in (xa, wg, wu))
    bg, bu = (_bias(f, 1), _bias(f, 2)) if bias else (None, None)
    need = fp4.fp4_gemm_gated_workspace_size(m, f, k, fmt, False)
    ws = torch.zeros(max(need, 16), dtype=torch.uint8, device="cuda")
    h, g, u = (torch.full((m, f), float("nan"), dtype=out, device="cuda") for _ in range(3))
    dev = [None if b is None else b.cuda() for b in (bg, bu)]
    for _ in range(2):  # the workspace is left as it was found
        fp4.fp4_gemm_gated(fmt, qa.codes, qa.scales, qa.g, qg.codes, qg.scales, qg.g, qu.codes, qu.scales, qu.g, m, f, k,
                           dev[0], dev[1], ACTS[act], h, CODE[out], g if save else None, u if save else None,
                           workspace=ws, workspace_bytes=need)
        torch.cuda.synchronize()
        assert fp4.fp4_get_status() == fp4.OK
        assert not ws.any(), "workspace not left zero-filled"
    a = dequantized(qa)
    g64, eg = _linear64(a, dequantized(qg), bg)
    u64, eu = _linear64(a, dequantized(qu), bu)
    h64, eh = _gated64(g64, eg, u64, eu, act)
    assert_close(h, h64, eh, "H")
    if save:
        assert_close(g, g64, eg, "G")
        assert_close(u, u64, eu, "U")


@pytest.mark.parametrize("m,f,k", [(1, 32, 64), (130, 288, 512), (16, 512, 2048), (2560, 2048, 256), (300, 9632, 64)])
def test_gemm_gated_codes_feed_the_down_projection(m, f, k):
    """The NVFP4 copy of H is that of quantizing the FP32 H; alone it is the same, and it is the
    A operand of the next product."""
    xa = random_input(m, k, 3, torch.bfloat16)
    wg, wu = (random_input(f, k, s, torch.float32, std=0.1, outliers=False) for s in (4, 5))
    qa, qg, qu = (gpu_quantize(t.cuda(), fp4.NVFP4, 16) for t in (xa, wg, wu))
    need = fp4.fp4_gemm_gated_workspace_size(m, f, k, fp4.NVFP4, True)
    ws = torch.zeros(max(need, 16), dtype=torch.uint8, device="cuda")
    gh, amax = torch.tensor([0.003], device="cuda"), torch.full((1,), 9e9, device="cuda")
    codes, scales = codes_like(m, f, fp4.NVFP4)
    h = torch.empty(m, f, device="cuda")
    args = (fp4.NVFP4, qa.codes, qa.scales, qa.g, qg.codes, qg.scales, qg.g, qu.codes, qu.scales, qu.g, m, f, k, None,
            None, fp4.ACT_SILU)
    fp4.fp4_gemm_gated(*args, h, fp4.F32, Hcodes=codes, Hscales=scales, gH=gh, amax_out=amax, workspace=ws,
                       workspace_bytes=need)
    torch.cuda.synchronize()
    assert fp4.fp4_get_status() == fp4.OK and not ws.any()
    assert_codes_of(codes, scales, gh, h, fp4.NVFP4)
    assert amax.item() == h.abs().max().item()
    n = 96
    qd = gpu_quantize(random_input(n, f, 6, torch.float32, std=0.05, outliers=False).cuda(), fp4.NVFP4, 16)
    qh = fp4.Quantized(codes, scales, gh, m, f, fp4.NVFP4)
    y = fp4.gemm(qh, qd, torch.float32)
    y64, e = product64(dequantized(qh), dequantized(qd))
    assert_close(y, y64, e, "down projection")


@pytest.mark.parametrize("m,f,k", [(1, 96, 512), (16, 1024, 2048), (32, 200, 8192), (31, 333, 1056), (33, 640, 512),
                                   (200, 512, 1024)])
@pytest.mark.parametrize("out,act,save", [(torch.bfloat16, "silu", False), (torch.float32, "gelu", True)])
def test_gemm_gated_bf16a(m, f, k, out, act, save):
    x = random_input(m, k, m + k, torch.bfloat16)
    wg, wu = (random_input(f, k, f + s, torch.float32, std=0.05, outliers=False) for s in (1, 2))
    qg, qu = (gpu_quantize(t.cuda(), fp4.NVFP4, 16) for t in (wg, wu))
    bg, bu = _bias(f, 7), _bias(f, 8)
    ws = torch.zeros(fp4.fp4_gemm_gated_bf16a_workspace_size(m, f, k), dtype=torch.uint8, device="cuda")
    codes, scales = codes_like(m, k, fp4.NVFP4)
    gx = torch.empty(1, device="cuda")
    ox = oracle_quantize(x, fp4.NVFP4, 16)
    for call in range(3):
        h, g, u = (torch.full((m, f), float("nan"), dtype=out, device="cuda") for _ in range(3))
        fp4.fp4_gemm_gated_bf16a(x.cuda(), qg.codes, qg.scales, qg.g, qu.codes, qu.scales, qu.g, m, f, k, bg.cuda(),
                                 bu.cuda(), ACTS[act], h, CODE[out], g if save else None, u if save else None, codes,
                                 scales, gx, ws, ws.numel(), fp4.GEMM_WEIGHTS_READY if call else 0)
        torch.cuda.synchronize()
        assert fp4.fp4_get_status() == fp4.OK
    qx = fp4.Quantized(codes, scales, gx, m, k, fp4.NVFP4)
    assert_quant_equal(qx, ox, "activations")
    a = dequantized(qx)
    g64, eg = _linear64(a, dequantized(qg), bg)
    u64, eu = _linear64(a, dequantized(qu), bu)
    h64, eh = _gated64(g64, eg, u64, eu, act)
    assert_close(h, h64, eh, "H")
    if save:
        assert_close(g, g64, eg, "G")
        assert_close(u, u64, eu, "U")


@pytest.mark.parametrize("counts,f,k,fmt", [
    ([5, 0, 130, 1], 200, 96, fp4.MXFP4),          # an expert without rows, ragged columns
    ([0, 0, 7], 129, 256, fp4.NVFP4),
    ([128, 256, 300, 17, 0, 64], 384, 2880, fp4.MXFP4),
    ([1300, 1400], 256, 512, fp4.NVFP4),           # CTA pairs
    ([1500, 0, 2400], 333, 96, fp4.NVFP4),         # CTA pairs, ragged columns
    ([1500, 0, 2400], 336, 96, fp4.MXFP4),         # many rows, whole sectors
])
@pytest.mark.parametrize("out,save", [(torch.bfloat16, False), (torch.float32, True)])
def test_gemm_gated_grouped(counts, f, k, fmt, out, save):
    E, rows = len(counts), sum(counts)
    off = torch.tensor([0] + list(np.cumsum(counts)), dtype=torch.int32)
    x = random_input(rows, k, rows, torch.bfloat16)
    offs = off.cuda()
    codes = torch.empty(rows, k // 2, dtype=torch.uint8, device="cuda")
    scales = torch.empty(fp4.fp4_scales_bytes_grouped(rows, E, k, fmt), dtype=torch.uint8, device="cuda")
    gx = torch.ones(1, device="cuda")
    ws = torch.zeros(fp4.fp4_quantize_workspace_size(), dtype=torch.uint8, device="cuda")
    fp4.fp4_quantize_grouped(x.cuda(), rows, k, fp4.BF16, fmt, E, offs, codes, scales, gx, None, ws, ws.numel())
    w = [[gpu_quantize(random_input(f, k, 10 * e + s, torch.float32, std=0.05 + 0.01 * e, outliers=False).cuda(), fmt,
                       _blk(fmt)) for e in range(E)] for s in (1, 2)]
    cat = [(torch.stack([q.codes for q in qs]), torch.cat([q.scales for q in qs]), torch.cat([q.g for q in qs])) for qs in w]
    bg, bu = _bias((E, f), 3), _bias((E, f), 4)
    # a row before and a row after the call's rows must stay as they are
    big = [torch.full((rows + 2, f + f % 8), 7.0, dtype=out, device="cuda") for _ in range(3)]
    bufs = [torch.full((rows * f + 8,), 7.0, dtype=out, device="cuda") for _ in range(3)]
    h, g, u = bufs
    del big
    fp4.fp4_gemm_gated_grouped(fmt, E, offs, codes, scales, gx, *cat[0], *cat[1], rows, f, k, bg.cuda(), bu.cuda(),
                               fp4.ACT_SILU, h, CODE[out], g if save else None, u if save else None)
    torch.cuda.synchronize()
    assert fp4.fp4_get_status() == fp4.OK
    assert all((b[rows * f:] == 7.0).all() for b in bufs), "written past the last row"
    oq = oracle.quantize(np.ascontiguousarray(x.view(torch.int16).numpy().view(np.uint16)), fmt, _blk(fmt))
    a = oracle.dequantize(oq["codes"], oq["scales"], oq["g"], fmt)
    for e in range(E):
        lo, hi = int(off[e]), int(off[e + 1])
        if lo == hi:
            continue
        g64, eg = _linear64(a[lo:hi], dequantized(w[0][e]), bg[e])
        u64, eu = _linear64(a[lo:hi], dequantized(w[1][e]), bu[e])
        h64, eh = _gated64(g64, eg, u64, eu, "silu")
        assert_close(h[:rows * f].view(rows, f)[lo:hi], h64, eh, f"H of expert {e}")
        if save:
            assert_close(g[:rows * f].view(rows, f)[lo:hi], g64, eg, f"G of expert {e}")
            assert_close(u[:rows * f].view(rows, f)[lo:hi], u64, eu, f"U of expert {e}")



@pytest.mark.parametrize("counts,pad,f,k,fmt", [
    ([5, 0, 130], 70, 200, 96, fp4.MXFP4),
    ([0, 0], 40, 128, 256, fp4.NVFP4),             # no rows at all
    ([1300, 700], 1000, 256, 512, fp4.NVFP4),      # CTA pairs
])
def test_gemm_gated_grouped_leaves_rows_behind_the_last_expert(counts, pad, f, k, fmt):
    E, rows = len(counts), sum(counts)
    total = rows + pad
    offs = torch.tensor([0] + list(np.cumsum(counts)), dtype=torch.int32).cuda()
    qx = gpu_quantize(random_input(total, k, 3, torch.bfloat16).cuda(), fmt, _blk(fmt))
    scales = torch.full((fp4.fp4_scales_bytes_grouped(total, E, k, fmt),), 0x38 if fmt == fp4.NVFP4 else 127,
                        dtype=torch.uint8, device="cuda")
    w = [gpu_quantize(random_input(E * f, k, s, torch.float32, std=0.05, outliers=False).cuda(), fmt, _blk(fmt))
         for s in (1, 2)]
    ws = [torch.full((E * fp4.fp4_scales_bytes(f, k, fmt),), 0x38 if fmt == fp4.NVFP4 else 127, dtype=torch.uint8,
                     device="cuda") for _ in w]

    def run(n):
        out = [torch.full((total * f + 8,), 7.0, device="cuda") for _ in range(3)]
        fp4.fp4_gemm_gated_grouped(fmt, E, offs, qx.codes, scales, None, w[0].codes, ws[0], None, w[1].codes, ws[1], None,
                                   n, f, k, None, None, fp4.ACT_SILU, out[0], fp4.F32, out[1], out[2])
        torch.cuda.synchronize()
        assert fp4.fp4_get_status() == fp4.OK
        return out

    # With scales of 1 the products are multiples of 1/4 and their sums stay below 2^22 of
    # those: exact in FP32 in any order, so both calls give the same bits.
    padded = run(total)
    assert all((b[rows * f:] == 7.0).all() for b in padded), "a row behind the last expert's was written"
    if rows:
        for b, c in zip(padded, run(rows)):
            assert torch.equal(b, c)


EPI = [
    # m, n, k, fmt
    (1, 333, 2080, fp4.NVFP4),       # decode kernel
    (16, 1024, 2048, fp4.NVFP4),     # decode kernel
    (32, 256, 4096, fp4.NVFP4),
    (16, 640, 2048, fp4.MXFP4),      # swapped operands, N-tile 16, stream-K
    (20, 5000, 96, fp4.MXFP4),       # swapped, whole tiles
    (48, 640, 2048, fp4.NVFP4),      # swapped, N-tile 64
    (130, 384, 1024, fp4.NVFP4),     # 128-wide tiles
    (200, 1001, 96, fp4.MXFP4),      # odd N: element stores
    (256, 256, 8192, fp4.NVFP4),     # stream-K in place
    (129, 38000, 64, fp4.NVFP4),     # 256-wide tiles, CTA pairs and ragged columns
    (2560, 2048, 512, fp4.MXFP4),    # CTA pairs
]


@pytest.mark.parametrize("m,n,k,fmt", EPI)
@pytest.mark.parametrize("out,res,act,save,bias", [
    (torch.bfloat16, torch.bfloat16, "none", False, True), (torch.float32, torch.float32, "gelu", True, True),
    (torch.bfloat16, torch.float32, "silu", True, False), (torch.float32, None, "gelu_tanh", False, True),
    (torch.float32, torch.bfloat16, "relu", False, False), (torch.bfloat16, None, "relu", True, True)])
def test_gemm_epilogue_ex(m, n, k, fmt, out, res, act, save, bias):
    xa = random_input(m, k, m + 7 * k, torch.bfloat16)
    xb = random_input(n, k, n + 11 * k, torch.float32, std=0.05, outliers=False)
    qa, qb = gpu_quantize(xa.cuda(), fmt, _blk(fmt)), gpu_quantize(xb.cuda(), fmt, _blk(fmt))
    b = _bias(n, 5) if bias else None
    r = None if res is None else random_input(m, n, 6, res, outliers=False)
    need = fp4.fp4_gemm_epilogue_workspace_size(m, n, k, fmt, False)
    ws = torch.zeros(max(need, 16), dtype=torch.uint8, device="cuda")
    d, pre = (torch.full((m, n), float("nan"), dtype=out, device="cuda") for _ in range(2))

    def call(d, r):
        fp4.fp4_gemm_epilogue_ex(fmt, qa.codes, qa.scales, qa.g, qb.codes, qb.scales, qb.g, m, n, k,
                                 None if b is None else b.cuda(), ACTS[act], r, CODE[res] if res else 0, d, CODE[out],
                                 pre if save else None, workspace=ws, workspace_bytes=need)
        torch.cuda.synchronize()
        assert fp4.fp4_get_status() == fp4.OK
        assert not ws.any(), "workspace not left zero-filled"

    call(d, None if r is None else r.cuda())
    z64, ez = _linear64(dequantized(qa), dequantized(qb), b)
    v, _ = act64(z64, act)
    t64 = v + (r.double() if r is not None else 0.0)
    slope = 1.0 if act in ("none", "relu") else MAX_SLOPE
    et = slope * ez + act_error(z64, v) + 2.0 ** -23 * t64.abs()
    assert_close(d, t64, et, "D")
    if save:
        assert_close(pre, z64, ez, "pre")
    if res == out:  # the residual stream updated in place
        d2 = r.cuda().clone()
        call(d2, d2)
        assert_close(d2, t64, et, "in place")


@pytest.mark.parametrize("m,n,k", [(16, 288, 2048), (130, 384, 512), (2560, 2048, 256)])
def test_gemm_epilogue_ex_codes(m, n, k):
    qa = gpu_quantize(random_input(m, k, 1, torch.bfloat16).cuda(), fp4.NVFP4, 16)
    qb = gpu_quantize(random_input(n, k, 2, torch.float32, std=0.05, outliers=False).cuda(), fp4.NVFP4, 16)
    r = random_input(m, n, 3, torch.bfloat16, outliers=False).cuda()
    need = fp4.fp4_gemm_epilogue_workspace_size(m, n, k, fp4.NVFP4, True)
    ws = torch.zeros(max(need, 16), dtype=torch.uint8, device="cuda")
    codes, scales = codes_like(m, n, fp4.NVFP4)
    gd, amax, d = torch.tensor([0.004], device="cuda"), torch.empty(1, device="cuda"), torch.empty(m, n, device="cuda")
    fp4.fp4_gemm_epilogue_ex(fp4.NVFP4, qa.codes, qa.scales, qa.g, qb.codes, qb.scales, qb.g, m, n, k, None, fp4.ACT_GELU,
                             r, fp4.BF16, d, fp4.F32, None, codes, scales, gd, amax, ws, need)
    torch.cuda.synchronize()
    assert fp4.fp4_get_status() == fp4.OK and not ws.any()
    assert_codes_of(codes, scales, gd, d, fp4.NVFP4)
    assert amax.item() == d.abs().max().item()


def test_gemm_epilogue_ex_without_extras_is_the_plain_epilogue():
    m, n, k = 130, 384, 1024
    qa = gpu_quantize(random_input(m, k, 1, torch.bfloat16).cuda(), fp4.NVFP4, 16)
    qb = gpu_quantize(random_input(n, k, 2, torch.float32, std=0.05, outliers=False).cuda(), fp4.NVFP4, 16)
    b = _bias(n, 5).cuda()
    d, e = (torch.empty(m, n, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    head = (fp4.NVFP4, qa.codes, qa.scales, qa.g, qb.codes, qb.scales, qb.g, m, n, k, b, fp4.ACT_RELU)
    fp4.fp4_gemm_epilogue(*head, d, fp4.BF16)
    fp4.fp4_gemm_epilogue_ex(*head, None, fp4.F32, e, fp4.BF16)
    assert torch.equal(d, e)
