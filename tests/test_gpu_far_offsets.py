"""Matrices of more than 2^31 elements: the last rows are those of the same call on them alone.  Few
rows with a K beyond the decode kernel's."""
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


@pytest.mark.parametrize("m,n,more", [(1, 64, 0), (16, 64, 0), (32, 64, 0), (1, 64, 32), (16, 64, 32), (32, 64, 32),
                                      (16, 9500, 32)])  # (the last: enough tiles not to split K)
def test_few_rows_with_the_longest_k(m, n, more):
    """The last K that the decode kernel takes, and the first that it does not."""
    k = 2048 * torch.cuda.get_device_properties(0).multi_processor_count + more
    x = torch.randn(m, k, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda").to(torch.bfloat16)
    w = torch.randn(n, k, generator=torch.Generator(device="cuda").manual_seed(2), device="cuda").mul_(0.02)
    qa, qb = fp4.quantize(x, fp4.NVFP4), fp4.quantize(w, fp4.NVFP4)
    del w

    def values(q, rows):
        out = torch.empty(rows, k, device="cuda")
        fp4.fp4_dequantize(q.codes, q.scales, q.g, rows, k, fp4.NVFP4, out)
        return out

    a, b = values(qa, m).double(), values(qb, n)
    parts = (b[i:i + 1000].double() for i in range(0, n, 1000))
    z, size = (torch.cat(t, 1) for t in zip(*((a @ p.t(), a.abs() @ p.abs().t()) for p in parts)))
    del b
    err = 1e-6 * size + 2.0 ** -22 * z.abs()  # the products' bound, and the scales'
    square = 2 * err * (z.abs() + err) + 2.0 ** -23 * z * z
    r = torch.ones(m, n, device="cuda")
    ws = fp4.Workspace()
    assert ((fp4.gemm(qa, qb, torch.float32, ws) - z).abs() <= err).all()
    d, pre = fp4.gemm_epilogue(qa, qb, residual=r, out_dtype=torch.float32, save=True, workspace=ws)
    assert ((pre - z).abs() <= err).all() and ((d - 1 - z).abs() <= err + 2.0 ** -23 * (z.abs() + 1)).all()
    h, g, u = fp4.gemm_gated(qa, qb, qb, fp4.ACT_NONE, out_dtype=torch.float32, save=True, workspace=ws)
    assert ((g - z).abs() <= err).all() and ((u - z).abs() <= err).all() and ((h - z * z).abs() <= square).all()
    xc = torch.empty(m, k // 2, dtype=torch.uint8, device="cuda")
    xs = torch.empty(fp4.fp4_scales_bytes(m, k, fp4.NVFP4), dtype=torch.uint8, device="cuda")
    xg, d = torch.empty(1, device="cuda"), torch.empty(m, n, device="cuda")
    buf = ws.get(max(fp4.fp4_gemm_bf16a_workspace_size(m, n, k), fp4.fp4_gemm_gated_bf16a_workspace_size(m, n, k)))
    fp4.fp4_gemm_gated_bf16a(x, qb.codes, qb.scales, qb.g, qb.codes, qb.scales, qb.g, m, n, k, None, None, fp4.ACT_NONE, d,
                             fp4.F32, None, None, xc, xs, xg, buf, buf.numel())
    assert ((d - z * z).abs() <= square).all() and torch.equal(xc, qa.codes) and torch.equal(xg, qa.g)
    fp4.fp4_gemm_bf16a(x, qb.codes, qb.scales, qb.g, m, n, k, d, fp4.F32, xc, xs, xg, buf, buf.numel())
    assert ((d - z).abs() <= err).all() and torch.equal(xc, qa.codes) and torch.equal(xg, qa.g)
    assert not ws.buf.any() and fp4.fp4_get_status() == fp4.OK
