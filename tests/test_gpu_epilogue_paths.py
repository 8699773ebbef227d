"""The product's epilogues on the paths that a plan can take: values that are no numbers, whole and
split tiles of every width, rows that are no whole sectors."""
import pytest
import torch

import block_scaled_fp4_04_b200 as fp4
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
