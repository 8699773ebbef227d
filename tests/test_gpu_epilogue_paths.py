"""The product's epilogues on the paths that a plan can take: values that are no numbers, whole and
split tiles of every width, rows that are no whole sectors."""
import numpy as np
import pytest
import torch

import block_scaled_fp4_04_b200 as fp4
from ffn_testutil import (ACTS, CODE, MAX_SLOPE, act64, act_error, assert_close, assert_codes_of, codes_like, dequantized,
                          product64)
from fp4_testutil import gpu_quantize, random_input

pytestmark = pytest.mark.gpu


def _blk(fmt):
    return 16 if fmt == fp4.NVFP4 else 32


def _operands(m, n, k, fmt, std=0.05):
    return (gpu_quantize(random_input(m, k, m + 7 * k, torch.bfloat16).cuda(), fmt, _blk(fmt)),
            gpu_quantize(random_input(n, k, n + 11 * k, torch.float32, std=std, outliers=False).cuda(), fmt, _blk(fmt)))


@pytest.mark.parametrize("m,n,k,fmt", [
    (16, 1024, 2048, fp4.NVFP4),     # decode kernel
    (5, 640, 2048, fp4.MXFP4),       # operands swapped, split over K
    (48, 1000, 96, fp4.NVFP4),       # operands swapped, whole tiles
    (130, 384, 512, fp4.NVFP4),      # 128-wide tiles
    (256, 256, 8192, fp4.NVFP4),     # the same, split over K
    (130, 333, 96, fp4.MXFP4),       # odd rows
    (2560, 2048, 64, fp4.NVFP4),     # CTA pairs
])
@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
def test_relu_of_a_nan_is_one_on_every_path(m, n, k, fmt, out):
    """A column whose bias is NaN is NaN with and without the pre-activation, and the others the same."""
    qa, qb = _operands(m, n, k, fmt)
    bias = torch.randn(n, generator=torch.Generator().manual_seed(1)).cuda()
    bias[3] = float("nan")
    oc = fp4.BF16 if out == torch.bfloat16 else fp4.F32
    ws = torch.zeros(max(16, fp4.fp4_gemm_epilogue_workspace_size(m, n, k, fmt, True),
                         fp4.fp4_gemm_epilogue_workspace_size(m, n, k, fmt, False)), dtype=torch.uint8, device="cuda")
    d, e, f, pre = (torch.empty(m, n, dtype=out, device="cuda") for _ in range(4))
    amax = torch.zeros(1, device="cuda")
    head = (fmt, qa.codes, qa.scales, qa.g, qb.codes, qb.scales, qb.g, m, n, k, bias, fp4.ACT_RELU)
    tail = dict(workspace=ws, workspace_bytes=ws.numel())
    fp4.fp4_gemm_epilogue(*head, d, oc, **tail)
    fp4.fp4_gemm_epilogue_ex(*head, None, fp4.F32, e, oc, pre, **tail)
    fp4.fp4_gemm_epilogue(*head, f, oc, amax_out=amax, **tail)
    torch.cuda.synchronize()
    for t in (d, e, f):
        assert torch.isnan(t[:, 3]).all() and torch.isnan(t).sum() == m
        # the sums of a split product can differ in their last bits from call to call
        keep = torch.arange(n, device="cuda") != 3
        want = pre.float().clamp(min=0.0)[:, keep]
        assert ((t.float()[:, keep] - want).abs() <= 2.0 ** -7 * want + 1e-5 * want.max()).all()
    assert torch.isnan(amax).all()
    assert not ws.any() and fp4.fp4_get_status() == fp4.OK


@pytest.mark.parametrize("act", [fp4.ACT_RELU, fp4.ACT_SILU, fp4.ACT_GELU, fp4.ACT_GELU_TANH, fp4.ACT_NONE])
@pytest.mark.parametrize("m", [8, 130])
def test_gated_keeps_a_nan(act, m):
    f, k = 256, 512
    qa, qw = _operands(m, f, k, fp4.NVFP4)
    bias = torch.zeros(f, device="cuda")
    bias[3] = float("nan")
    h = torch.empty(m, f, device="cuda")
    n = fp4.fp4_gemm_gated_workspace_size(m, f, k, fp4.NVFP4, False)
    ws = torch.zeros(max(n, 16), dtype=torch.uint8, device="cuda")
    fp4.fp4_gemm_gated(fp4.NVFP4, qa.codes, qa.scales, qa.g, qw.codes, qw.scales, qw.g, qw.codes, qw.scales, qw.g, m, f, k,
                       bias, None, act, h, fp4.F32, workspace=ws, workspace_bytes=n)
    torch.cuda.synchronize()
    assert torch.isnan(h[:, 3]).all() and torch.isnan(h).sum() == m


@pytest.mark.parametrize("m,n,k,fmt", [(1, 512, 2048, fp4.NVFP4), (7, 640, 4096, fp4.NVFP4), (5, 300, 2048, fp4.MXFP4),
                                       (130, 257, 8192, fp4.NVFP4)])
def test_partial_sums_of_odd_products_need_a_word_s_alignment(m, n, k, fmt):
    qa, qb = _operands(m, n, k, fmt)
    need = fp4.fp4_gemm_workspace_size(m, n, k, fmt)
    assert need > 0
    d, e = (torch.empty(m, n, device="cuda") for _ in range(2))
    ws = torch.zeros(need + 16, dtype=torch.uint8, device="cuda")
    head = (fmt, qa.codes, qa.scales, qa.g, qb.codes, qb.scales, qb.g, m, n, k)
    fp4.fp4_gemm(*head, d, fp4.F32, ws, need)
    fp4.fp4_gemm(*head, e, fp4.F32, ws[4:], need)
    torch.cuda.synchronize()
    # up to 64 parts of a sum in any order, each rounded to half a step of the sum of magnitudes,
    # which is below 64 times the largest of these sums of random signs
    assert (d - e).abs().max() <= 2 * 64 * 2.0 ** -24 * 64 * d.abs().max()
    assert not ws.any() and fp4.fp4_get_status() == fp4.OK


def _bias(n, seed):
    return torch.from_numpy((np.random.default_rng(seed).standard_normal(n) * 0.7).astype(np.float32))


def _linear64(a, b, bias):
    """(a b^T + bias, the bound of its FP32 error: the product's, two roundings of the sum)."""
    z, e = product64(a, b)
    if bias is not None:
        z = z + bias.double()
        e = e + 2.0 ** -24 * bias.double().abs()
    return z, e + 2.0 ** -23 * z.abs()


def _epilogue(m, n, k, fmt, out, res, act, save, bias, split, offset=0):
    """fp4_gemm_epilogue_ex against 64 bits; `split`: whether the plan splits K (the workspace says
    so); outputs and residual start `offset` bytes behind their allocation."""
    qa, qb = _operands(m, n, k, fmt)
    b = _bias(n, 5) if bias else None
    r = None if res is None else random_input(m, n, 6, res, outliers=False)
    need = fp4.fp4_gemm_epilogue_workspace_size(m, n, k, fmt, False)
    assert (need > 0) == split, "the plan no longer takes the path this case is for"
    ws = torch.zeros(max(need, 16), dtype=torch.uint8, device="cuda")

    def new(dtype):
        pad = offset // torch.empty(0, dtype=dtype).element_size()
        return torch.full((m * n + pad,), float("nan"), dtype=dtype, device="cuda")[pad:].view(m, n)

    d, pre = new(out), new(out)
    rd = None
    if r is not None:
        rd = new(res)
        rd.copy_(r)

    def call(d, rd):
        fp4.fp4_gemm_epilogue_ex(fmt, qa.codes, qa.scales, qa.g, qb.codes, qb.scales, qb.g, m, n, k,
                                 None if b is None else b.cuda(), ACTS[act], rd, CODE[res] if res else 0, d, CODE[out],
                                 pre if save else None, workspace=ws, workspace_bytes=need)
        torch.cuda.synchronize()
        assert fp4.fp4_get_status() == fp4.OK
        assert not ws.any(), "workspace not left zero-filled"

    call(d, rd)
    z64, ez = _linear64(dequantized(qa), dequantized(qb), b)
    v, _ = act64(z64, act)
    t64 = v + (r.double() if r is not None else 0.0)
    et = (1.0 if act in ("none", "relu") else MAX_SLOPE) * ez + act_error(z64, v) + 2.0 ** -23 * t64.abs()
    assert_close(d, t64, et, "D")
    if save:
        assert_close(pre, z64, ez, "pre")
    if res == out:  # in place
        call(rd, rd)
        assert_close(rd, t64, et, "in place")


EXTRAS = [(torch.bfloat16, torch.bfloat16, "none", False, True), (torch.float32, torch.float32, "gelu", True, True),
          (torch.bfloat16, torch.float32, "silu", True, False), (torch.float32, torch.bfloat16, "relu", True, True)]


@pytest.mark.parametrize("m,n,k,fmt,split", [
    (48, 1000, 96, fp4.NVFP4, False),     # 64 columns of swapped operands, a warp with some of its rows
    (33, 333, 96, fp4.MXFP4, False),
    (50, 1001, 2048, fp4.NVFP4, True),    # split, single partial sums
    (64, 1000, 1056, fp4.MXFP4, True),    # split, partial sums by fours
    (20, 1001, 2048, fp4.MXFP4, True),    # 32 columns
    (5, 333, 2048, fp4.MXFP4, True),      # 16 columns
])
@pytest.mark.parametrize("out,res,act,save,bias", EXTRAS)
def test_epilogue_of_few_rows(m, n, k, fmt, split, out, res, act, save, bias):
    _epilogue(m, n, k, fmt, out, res, act, save, bias, split)


@pytest.mark.parametrize("m,n,k,fmt,split,offset", [
    (130, 257, 8192, fp4.NVFP4, True, 0),     # split in place, rows of partial sums padded to 260
    (130, 131, 16384, fp4.MXFP4, True, 0),
    (130, 260, 8192, fp4.NVFP4, True, 16),
    (2560, 2001, 64, fp4.NVFP4, False, 0),    # CTA pairs, odd rows
    (2560, 2004, 64, fp4.MXFP4, False, 0),    # CTA pairs, rows of no whole sectors
    (2560, 2048, 64, fp4.NVFP4, False, 16),   # CTA pairs, whole sectors that start between two
    (129, 19001, 64, fp4.NVFP4, False, 0),    # 256-wide tiles on single CTAs, odd rows
    (129, 19004, 64, fp4.MXFP4, False, 0),
    (129, 19008, 64, fp4.MXFP4, False, 16),
])
@pytest.mark.parametrize("out,res,act,save,bias", EXTRAS)
def test_epilogue_in_place(m, n, k, fmt, split, offset, out, res, act, save, bias):
    _epilogue(m, n, k, fmt, out, res, act, save, bias, split, offset)


@pytest.mark.parametrize("m,n,k,fmt,split", [(130, 288, 8192, fp4.NVFP4, True), (20, 96, 16384, fp4.MXFP4, True),
                                             (130, 384, 512, fp4.MXFP4, False), (2560, 2080, 64, fp4.MXFP4, False)])
def test_epilogue_to_codes(m, n, k, fmt, split):
    """NVFP4 codes and the maximum of the result, from operands of either format, whole and split."""
    qa, qb = _operands(m, n, k, fmt)
    r = random_input(m, n, 3, torch.bfloat16, outliers=False).cuda()
    need = fp4.fp4_gemm_epilogue_workspace_size(m, n, k, fmt, True)
    assert (need > 0) == split, "the plan no longer takes the path this case is for"
    ws = torch.zeros(max(need, 16), dtype=torch.uint8, device="cuda")
    codes, scales = codes_like(m, n, fp4.NVFP4)
    gd, amax = torch.tensor([0.004], device="cuda"), torch.empty(1, device="cuda")
    d, pre = (torch.empty(m, n, device="cuda") for _ in range(2))
    for _ in range(2):
        fp4.fp4_gemm_epilogue_ex(fmt, qa.codes, qa.scales, qa.g, qb.codes, qb.scales, qb.g, m, n, k, None, fp4.ACT_GELU, r,
                                 fp4.BF16, d, fp4.F32, pre, codes, scales, gd, amax, ws, need)
        torch.cuda.synchronize()
        assert fp4.fp4_get_status() == fp4.OK and not ws.any()
        assert_codes_of(codes, scales, gd, d, fp4.NVFP4)
        assert amax.item() == d.abs().max().item()
    z64, ez = _linear64(dequantized(qa), dequantized(qb), None)
    v, _ = act64(z64, "gelu")
    t64 = v + r.cpu().double()
    assert_close(pre, z64, ez, "pre")
    assert_close(d, t64, MAX_SLOPE * ez + act_error(z64, v) + 2.0 ** -23 * t64.abs(), "D")


GATED = [
    (1, 257, 8192, fp4.MXFP4, True),       # split, odd F: rows of partial sums padded to 260
    (20, 257, 8192, fp4.MXFP4, True),
    (17, 384, 8192, fp4.NVFP4, True),      # the first row count past the decode kernel
    (130, 131, 16384, fp4.NVFP4, True),    # split, more than one tile of rows
    (130, 160, 16384, fp4.MXFP4, True),
    (16, 512, 2880, fp4.MXFP4, False),     # whole tiles: too little to save
    (33, 640, 2048, fp4.NVFP4, False),
    (2560, 2001, 64, fp4.NVFP4, False),    # CTA pairs, odd rows
    (2560, 2004, 64, fp4.MXFP4, False),
    (129, 19001, 64, fp4.NVFP4, False),    # single CTAs, odd rows
]


@pytest.mark.parametrize("m,f,k,fmt,split", GATED)
@pytest.mark.parametrize("out,act,bias", [(torch.float32, "silu", True), (torch.bfloat16, "gelu_tanh", False)])
def test_gated_plans(m, f, k, fmt, split, out, act, bias):
    qa, qg = _operands(m, f, k, fmt)
    qu = gpu_quantize(random_input(f, k, 13, torch.float32, std=0.05, outliers=False).cuda(), fmt, _blk(fmt))
    bg, bu = (_bias(f, 1), _bias(f, 2)) if bias else (None, None)
    need = fp4.fp4_gemm_gated_workspace_size(m, f, k, fmt, False)
    assert (need > 0) == split, "the plan no longer takes the path this case is for"
    ws = torch.zeros(max(need, 16), dtype=torch.uint8, device="cuda")
    h, g, u = (torch.full((m, f), float("nan"), dtype=out, device="cuda") for _ in range(3))
    dev = [None if b is None else b.cuda() for b in (bg, bu)]
    for _ in range(2):
        fp4.fp4_gemm_gated(fmt, qa.codes, qa.scales, qa.g, qg.codes, qg.scales, qg.g, qu.codes, qu.scales, qu.g, m, f, k,
                           dev[0], dev[1], ACTS[act], h, CODE[out], g, u, workspace=ws, workspace_bytes=need)
        torch.cuda.synchronize()
        assert fp4.fp4_get_status() == fp4.OK
        assert not ws.any(), "workspace not left zero-filled"
    a = dequantized(qa)
    g64, eg = _linear64(a, dequantized(qg), bg)
    u64, eu = _linear64(a, dequantized(qu), bu)
    assert_close(g, g64, eg, "G")
    assert_close(u, u64, eu, "U")
    v, _ = act64(g64, act)
    ev = MAX_SLOPE * eg + act_error(g64, v)
    assert_close(h, v * u64, ev * u64.abs() + eu * v.abs() + ev * eu + 2.0 ** -23 * (v * u64).abs(), "H")


@pytest.mark.parametrize("m,f,k,fmt,split", [(130, 160, 16384, fp4.NVFP4, True), (20, 96, 16384, fp4.MXFP4, True),
                                             (1, 128, 8192, fp4.NVFP4, True), (130, 288, 512, fp4.MXFP4, False)])
def test_gated_to_codes(m, f, k, fmt, split):
    """NVFP4 codes and the maximum of H, from operands of either format, whole and split."""
    qa, qg = _operands(m, f, k, fmt)
    qu = gpu_quantize(random_input(f, k, 13, torch.float32, std=0.05, outliers=False).cuda(), fmt, _blk(fmt))
    need = fp4.fp4_gemm_gated_workspace_size(m, f, k, fmt, True)
    assert (need > 0) == split, "the plan no longer takes the path this case is for"
    ws = torch.zeros(max(need, 16), dtype=torch.uint8, device="cuda")
    gh, amax = torch.tensor([0.01], device="cuda"), torch.empty(1, device="cuda")
    h = torch.empty(m, f, device="cuda")
    for _ in range(2):
        codes, scales = codes_like(m, f, fp4.NVFP4)
        fp4.fp4_gemm_gated(fmt, qa.codes, qa.scales, qa.g, qg.codes, qg.scales, qg.g, qu.codes, qu.scales, qu.g, m, f, k,
                           None, None, fp4.ACT_SILU, h, fp4.F32, Hcodes=codes, Hscales=scales, gH=gh, amax_out=amax,
                           workspace=ws, workspace_bytes=need)
        torch.cuda.synchronize()
        assert fp4.fp4_get_status() == fp4.OK and not ws.any()
        assert_codes_of(codes, scales, gh, h, fp4.NVFP4)
        assert amax.item() == h.abs().max().item()
    a = dequantized(qa)
    g64, eg = _linear64(a, dequantized(qg), None)
    u64, eu = _linear64(a, dequantized(qu), None)
    v, _ = act64(g64, "silu")
    ev = MAX_SLOPE * eg + act_error(g64, v)
    assert_close(h, v * u64, ev * u64.abs() + eu * v.abs() + ev * eu + 2.0 ** -23 * (v * u64).abs(), "H")


@pytest.mark.parametrize("m,n,k", [(16, 288, 2048), (130, 288, 8192), (2560, 2048, 64)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_codes_of_a_value_that_has_none_latch(m, n, k, bad):
    """As fp4_quantize does; a result without codes keeps the value and latches nothing."""
    qa, qb = _operands(m, n, k, fp4.NVFP4)
    bias = torch.zeros(n, device="cuda")
    ws = torch.zeros(max(16, *(size(m, n, k, fp4.NVFP4, in_place) for in_place in (True, False)
                               for size in (fp4.fp4_gemm_epilogue_workspace_size, fp4.fp4_gemm_gated_workspace_size))),
                     dtype=torch.uint8, device="cuda")
    codes, scales = codes_like(m, n, fp4.NVFP4)
    gd, d = torch.tensor([0.01], device="cuda"), torch.empty(m, n, device="cuda")
    head = (fp4.NVFP4, qa.codes, qa.scales, qa.g, qb.codes, qb.scales, qb.g)
    tail = dict(workspace=ws, workspace_bytes=ws.numel())
    calls = [
        lambda c, s: fp4.fp4_gemm_epilogue(*head, m, n, k, bias, fp4.ACT_NONE, d, fp4.F32, c, s, gd, **tail),
        lambda c, s: fp4.fp4_gemm_epilogue_ex(*head, m, n, k, bias, fp4.ACT_NONE, d, fp4.F32, d, fp4.F32, None, c, s, gd,
                                              **tail),
        lambda c, s: fp4.fp4_gemm_gated(*head, qb.codes, qb.scales, qb.g, m, n, k, bias, None, fp4.ACT_NONE, d, fp4.F32,
                                        Hcodes=c, Hscales=s, gH=gd, **tail),
    ]
    for value, status in ((0.0, fp4.OK), (bad, fp4.ERR_NONFINITE)):
        bias[n - 1] = value
        for call in calls:
            d.zero_()
            call(codes, scales)
            assert fp4.fp4_get_status() == status
            d.zero_()
            call(None, None)
            assert fp4.fp4_get_status() == fp4.OK
            assert torch.isfinite(d[:, n - 1]).all() == (status == fp4.OK)
    assert not ws.any()
