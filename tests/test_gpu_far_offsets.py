"""Matrices of more than 2^31 elements: the last rows are those of the same call on them alone."""
import pytest
import torch

import block_scaled_fp4_04_b200 as fp4

pytestmark = pytest.mark.gpu


def _filled(rows, cols, dtype, seed, last):
    """Zeros but for the first and the last rows."""
    t = torch.zeros(rows, cols, dtype=dtype, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(seed)
    for part in (t[:last], t[-last:]):
        part.copy_(torch.randn(last, cols, generator=g, device="cuda"))
    return t


@pytest.mark.parametrize("rows,cols,dtype", [(270001, 8192, torch.bfloat16), (70001, 32768, torch.bfloat16),
                                             (260003, 8259, torch.bfloat16), (270001, 8192, torch.float32)])
def test_norm(rows, cols, dtype):
    last = 129
    x, dy = _filled(rows, cols, dtype, 1, last), _filled(rows, cols, dtype, 2, last)
    w = torch.linspace(0.5, 2.0, cols, device="cuda")
    y, mean, rstd = fp4.layernorm(x, w, None)
    for at in (slice(0, last), slice(rows - last, rows)):
        z, m, r = fp4.layernorm(x[at].clone(), w, None)
        # (few rows take another kernel, whose sums have another order)
        assert (mean[at] - m).abs().max() <= 1e-6 and ((rstd[at] - r) / r).abs().max() <= 1e-5
        assert ((y[at].float() - z.float()).abs() <= 2.0 ** -7 * z.float().abs() + 1e-4).all()  # a BF16 step
    del y
    dx, dw, db = fp4.layernorm_backward(dy, x, w, mean, rstd)
    for at in (slice(0, last), slice(rows - last, rows)):
        d, _, _ = fp4.layernorm_backward(dy[at].clone(), x[at].clone(), w, mean[at].clone(), rstd[at].clone())
        assert ((dx[at].float() - d.float()).abs() <= 2.0 ** -7 * d.float().abs() + 1e-4).all()
    ends = [torch.cat((t[:last], t[-last:])) for t in (x, dy)] + [torch.cat((t[:last], t[-last:])) for t in (mean, rstd)]
    _, dw2, db2 = fp4.layernorm_backward(ends[1], ends[0], w, ends[2], ends[3])
    for a, b in ((dw, dw2), (db, db2)):
        assert (a - b).abs().max() <= 1e-4 * b.abs().max()
    assert fp4.fp4_get_status() == fp4.OK


@pytest.mark.parametrize("gated", [True, False])
def test_act_backward(gated):
    rows, cols, last = (135001, 16384, 70) if not gated else (68001, 16384, 70)
    dh, g = (_filled(rows, cols, torch.bfloat16, s, last) for s in (1, 2))
    u = _filled(rows, cols, torch.bfloat16, 3, last) if gated else None
    dz, db = fp4.act_backward(dh, g, u, fp4.ACT_GELU, dbias=True)
    assert dz.numel() > 1 << 31
    for at in (slice(0, last), slice(rows - last, rows)):
        z = fp4.act_backward(dh[at].clone(), g[at].clone(), None if u is None else u[at].clone(), fp4.ACT_GELU)
        assert torch.equal(dz[at], z)
    assert not dz[last:-last].any()
    ends = [None if t is None else torch.cat((t[:last], t[-last:])) for t in (dh, g, u)]
    _, db2 = fp4.act_backward(*ends, fp4.ACT_GELU, dbias=True)
    assert (db - db2).abs().max() <= 1e-4 * db2.abs().max()


@pytest.mark.parametrize("n", [32768, 32801])
def test_products(n):
    m, k, last = 65600, 64, 200
    qa = fp4.quantize(_filled(m, k, torch.bfloat16, 1, last), fp4.MXFP4)
    qb = fp4.quantize(torch.randn(n, k, generator=torch.Generator(device="cuda").manual_seed(2), device="cuda"), fp4.MXFP4)
    r = _filled(m, n, torch.bfloat16, 3, last)
    bias = torch.ones(n, device="cuda")
    d, pre = fp4.gemm_epilogue(qa, qb, bias, fp4.ACT_SILU, r, save=True)
    h, g, _ = fp4.gemm_gated(qa, qb, qb, fp4.ACT_SILU, bias, bias, save=True)
    assert d.numel() > 1 << 31
    # a block's rows begin at a multiple of 128: their scales are a slice
    lo = (m - last) // 128 * 128
    scales = qa.scales[fp4.fp4_scales_bytes(lo, k, fp4.MXFP4):].clone()
    q2 = fp4.Quantized(qa.codes[lo:].clone(), scales, qa.g, m - lo, k, fp4.MXFP4)
    d2, pre2 = fp4.gemm_epilogue(q2, qb, bias, fp4.ACT_SILU, r[lo:].clone(), save=True)
    h2, g2, _ = fp4.gemm_gated(q2, qb, qb, fp4.ACT_SILU, bias, bias, save=True)
    for a, b in ((d, d2), (pre, pre2), (h, h2), (g, g2)):
        assert torch.equal(a[lo:], b)
    assert fp4.fp4_get_status() == fp4.OK
