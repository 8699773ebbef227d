"""Layer norm (forward, backward) and the activation's backward pass on the device, against
64-bit formulas, their differences, and the oracle's quantizer for the code outputs."""
import math

import numpy as np
import pytest
import torch

import block_scaled_fp4_04_b200 as fp4
from ffn_testutil import (ACTS, CODE, HALF_STEP, act64, act_error, assert_close, assert_codes_of, codes_like)

pytestmark = pytest.mark.gpu
EPS = 1e-5


def _rand(shape, seed, dtype=torch.float32, std=1.0, mean=0.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * std + mean).to(dtype)


def _cuda(*ts):
    return [None if t is None else t.cuda() for t in ts]


# ---------------------------------------------------------------- layer norm
def _ln64(x, w, b, eps):
    x = x.double()
    mean = x.mean(1, keepdim=True)
    var = (x - mean).square().mean(1, keepdim=True)
    rstd = (var + eps).rsqrt()
    y = (x - mean) * rstd
    if w is not None:
        y = y * w.double()
    if b is not None:
        y = y + b.double()
    return y, mean[:, 0], rstd[:, 0], var[:, 0]


def _ln_error(x, w, y, mean, rstd, var, n):
    """FP32 error of y.  A sum of n terms through per-thread chains of at most 32 (64 for very
    long rows: ceil(n / 4096)) and a tree of 14 is off by (chain + 14) 2^-24 of the terms' sum of
    magnitudes; the mean's error shifts x - mean, the variance's scales it by half its relative
    error; three more roundings follow."""
    chain = (32 + math.ceil(n / 2048) + 14) * 2.0 ** -24
    x = x.double()
    dmean = chain * x.abs().mean(1) + 2.0 ** -24 * mean.abs()
    drel = chain + dmean * rstd * 2 + 2.0 ** -22  # relative error of rstd
    aw = 1.0 if w is None else w.double().abs()
    xh = (x - mean[:, None]).abs() * rstd[:, None]
    return (dmean * rstd)[:, None] * aw + xh * aw * (drel[:, None] + 2.0 ** -22) + y.abs() * 2.0 ** -23, dmean, drel


LN_SHAPES = [(1, 1), (3, 7), (5, 32), (130, 256), (2, 513), (7, 1000), (16, 2880), (33, 8192), (9, 5760), (3, 16384),
             (2, 28672), (4, 12289), (300, 64), (1, 20011), (9, 1002), (5, 4098), (3, 8190),
             # enough rows for the rings
             (2387, 800), (2400, 1032), (2500, 2048), (2370, 2880), (2369, 5760), (2371, 4096), (2368, 8192),
             (2369, 16384)]


@pytest.mark.parametrize("rows,n", LN_SHAPES)
@pytest.mark.parametrize("dtype,out", [(torch.float32, torch.float32), (torch.bfloat16, torch.bfloat16),
                                       (torch.bfloat16, torch.float32), (torch.float32, torch.bfloat16)])
def test_layernorm(rows, n, dtype, out):
    x = _rand((rows, n), rows * 31 + n, dtype, 1.5, 0.7)
    w, b = _rand((n,), 1, std=0.5, mean=1.0), _rand((n,), 2, std=0.5)
    for use_w, use_b in ((True, True), (False, False)):
        ww, bb = (w if use_w else None), (b if use_b else None)
        xd, wd, bd = _cuda(x, ww, bb)
        y = torch.full((rows, n), float("nan"), dtype=out, device="cuda")
        mean, rstd, amax = (torch.full((k,), float("nan"), device="cuda") for k in (rows, rows, 1))
        fp4.fp4_layernorm(xd, rows, n, CODE[dtype], wd, bd, EPS, y, CODE[out], mean, rstd, amax_out=amax)
        y64, m64, r64, v64 = _ln64(x, ww, bb, EPS)
        err, dmean, drel = _ln_error(x, ww, y64, m64, r64, v64, n)
        assert_close(y, y64, err, "y")
        assert_close(mean, m64, dmean, "mean")
        assert_close(rstd, r64, drel * r64, "rstd")
        top = y64.abs().max().item()
        assert abs(amax.item() - top) <= err.max().item() + 2.0 ** -23 * top
    assert fp4.fp4_get_status() == fp4.OK


@pytest.mark.parametrize("rows,n", [(1, 1), (3, 7), (33, 8192), (300, 1002), (3, 20011), (5, 40000), (2500, 2048),
                                    (2400, 1032), (2369, 5760), (2369, 16384)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_layernorm_in_place(rows, n, dtype):
    x = _rand((rows, n), rows + n, dtype, 1.5, 0.7).cuda()
    w, b = _cuda(_rand((n,), 1, std=0.5, mean=1.0), _rand((n,), 2, std=0.5))
    y, mean, rstd = fp4.layernorm(x, w, b)
    z, mean2, rstd2 = fp4.layernorm(x, w, b, out=x)
    assert z.data_ptr() == x.data_ptr()
    assert torch.equal(z, y) and torch.equal(mean, mean2) and torch.equal(rstd, rstd2)


def test_layernorm_of_constant_and_shifted_rows():
    """A constant row has variance 0: y is the bias, rstd 1 / sqrt(eps).  A large common offset
    does not spoil the variance (two passes, no difference of squares)."""
    n = 512
    x = torch.full((2, n), 3.0)
    x[1] = 1000.0 + torch.arange(n) % 2  # exact in FP32: mean 1000.5, variance 1/4
    w, b = _rand((n,), 3), _rand((n,), 4)
    y, mean, rstd = torch.empty(2, n, device="cuda"), torch.empty(2, device="cuda"), torch.empty(2, device="cuda")
    fp4.fp4_layernorm(x.cuda(), 2, n, fp4.F32, w.cuda(), b.cuda(), EPS, y, fp4.F32, mean, rstd)
    assert torch.equal(y[0].cpu(), b) and mean[0].item() == 3.0
    assert abs(rstd[0].item() * math.sqrt(np.float32(EPS)) - 1) < 2.0 ** -22
    assert mean[1].item() == 1000.5
    assert abs(rstd[1].item() * math.sqrt(0.25 + np.float32(EPS)) - 1) < 2.0 ** -22


@pytest.mark.parametrize("fmt", [fp4.NVFP4, fp4.MXFP4])
@pytest.mark.parametrize("rows,n", [(1, 32), (130, 288), (128, 1024), (37, 2880), (5, 8192), (3, 20000),
                                    (2400, 2880), (2371, 1024)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_layernorm_codes(fmt, rows, n, dtype):
    """The codes are those of quantizing the FP32 y that the same call stores; pads are 0."""
    x = _rand((rows, n), n + rows, dtype)
    x[:, :: max(1, n // 8)] *= 30.0
    w, b = _rand((n,), 5, std=0.3, mean=1.0), _rand((n,), 6, std=0.3)
    codes, scales = codes_like(rows, n, fmt)
    y = torch.empty(rows, n, device="cuda")
    g = torch.tensor([0.013], device="cuda")
    gin = g if fmt == fp4.NVFP4 else None
    xd, wd, bd = _cuda(x, w, b)
    fp4.fp4_layernorm(xd, rows, n, CODE[dtype], wd, bd, EPS, y, fp4.F32, fmt=fmt, codes=codes, scales=scales,
                      global_in=gin)
    assert fp4.fp4_get_status() == fp4.OK
    assert_codes_of(codes, scales, g, y, fmt, "with y")
    codes2, scales2 = codes_like(rows, n, fmt)
    fp4.fp4_layernorm(xd, rows, n, CODE[dtype], wd, bd, EPS, None, fp4.F32, fmt=fmt, codes=codes2, scales=scales2,
                      global_in=gin)
    assert torch.equal(codes, codes2) and torch.equal(scales, scales2)


def test_layernorm_nonfinite_codes_latch():
    x = torch.ones(4, 64)
    x[2, 5] = float("inf")
    codes, scales = codes_like(4, 64, fp4.MXFP4)
    fp4.fp4_layernorm(x.cuda(), 4, 64, fp4.F32, None, None, EPS, None, fp4.F32, fmt=fp4.MXFP4, codes=codes,
                      scales=scales)
    assert fp4.fp4_get_status() == fp4.ERR_NONFINITE
    assert fp4.fp4_get_status() == fp4.OK


def _ln_grad64(dy, x, w, mean, rstd, dres):
    dy, x, mean, rstd = (t.double() for t in (dy, x, mean, rstd))
    xh = (x - mean[:, None]) * rstd[:, None]
    a = dy if w is None else dy * w.double()
    c1, c2 = a.mean(1, keepdim=True), (a * xh).mean(1, keepdim=True)
    dx = rstd[:, None] * (a - c1 - xh * c2)
    if dres is not None:
        dx = dx + dres.double()
    return dx, (dy * xh).sum(0), dy.sum(0), xh, a, c1, c2


@pytest.mark.parametrize("rows,n", [(1, 1), (3, 7), (700, 32), (130, 256), (513, 513), (7, 1000), (301, 2880), (33, 8192),
                                    (5, 16384), (2, 28672), (600, 64), (3, 12289), (149, 5760),
                                    (1187, 800), (1200, 1032), (1500, 2048), (1184, 2880), (1190, 5760),
                                    (1185, 8192), (300, 16384), (700, 2881), (20, 5003), (300, 16400),
                                    (400, 1002), (7, 4098), (6, 8190), (5, 16386), (70, 250)])
@pytest.mark.parametrize("dtype,out", [(torch.float32, torch.float32), (torch.bfloat16, torch.bfloat16),
                                       (torch.bfloat16, torch.float32)])
@pytest.mark.parametrize("res", [True, False])
def test_layernorm_backward(rows, n, dtype, out, res):
    x, dy = _rand((rows, n), n, dtype, 1.5, 0.3), _rand((rows, n), rows, dtype)
    w = _rand((n,), 1, std=0.5, mean=1.0) if res else None
    dres = _rand((rows, n), 9, dtype) if res else None
    _, m64, r64, _ = _ln64(x, None, None, EPS)
    mean, rstd = m64.float(), r64.float()
    dx64, dw64, db64, xh, a, c1, c2 = _ln_grad64(dy, x, w, mean, rstd, dres)
    dyd, xd, wd, md, rd, sd = _cuda(dy, x, w, mean, rstd, dres)
    ws = torch.full((fp4.fp4_layernorm_backward_workspace_size(rows, n),), 0xFF, dtype=torch.uint8, device="cuda")
    got = []
    for _ in range(2):
        dx = torch.full((rows, n), float("nan"), dtype=out, device="cuda")
        dw, db = (torch.full((n,), float("nan"), device="cuda") for _ in range(2))
        fp4.fp4_layernorm_backward(dyd, xd, rows, n, CODE[dtype], wd, md, rd, sd, dx, CODE[out], dw, db, ws, ws.numel())
        got.append((dx, dw, db))
    assert all(torch.equal(p, q) for p, q in zip(*got)), "not the same bits twice"
    # sums of n terms: chains of at most 64 terms and a tree (as the forward pass)
    chain = (64 + math.ceil(n / 512) + 14) * 2.0 ** -24
    r = rstd.double()[:, None]
    err = r * (chain * (a.abs().mean(1, keepdim=True) + xh.abs() * (a * xh).abs().mean(1, keepdim=True))
               + 2.0 ** -21 * (a.abs() + c1.abs() + (xh * c2).abs()) + 2.0 ** -22 * x.double().abs() * r * c2.abs())
    if dres is not None:
        err = err + 2.0 ** -24 * dx64.abs()
    assert_close(dx, dx64, err, "dx")
    # column sums: at most ceil(rows / parts) terms one after another, then the parts
    serial = (rows / min(rows, 148) + 600) * 2.0 ** -24
    xerr = 2.0 ** -22 * (x.double().abs() + mean.double().abs()[:, None]) * r
    assert_close(dw, dw64, serial * (dy.double() * xh).abs().sum(0) + (dy.double().abs() * xerr).sum(0), "dw")
    assert_close(db, db64, serial * dy.double().abs().sum(0), "db")
    # one of the two gradients alone, and dx in dy's place
    dw2 = torch.empty(n, device="cuda")
    inplace = dyd.clone()
    if out == dtype:
        fp4.fp4_layernorm_backward(inplace, xd, rows, n, CODE[dtype], wd, md, rd, sd, inplace, CODE[out], dw2, None, ws,
                                   ws.numel())
        assert torch.equal(inplace, dx) and torch.equal(dw2, dw)


def test_layernorm_backward_formula_against_differences():
    """The 64-bit formula that the kernels are held to is the derivative of the forward pass."""
    rows, n, h = 3, 11, 1e-6
    x, dy, w, b = (_rand(s, k).double() for k, s in enumerate([(rows, n), (rows, n), (n,), (n,)]))

    def loss(x, w, b):
        return (_ln64(x, w, b, EPS)[0] * dy).sum()

    _, m, r, _ = _ln64(x, None, None, EPS)
    dx, dw, db = _ln_grad64(dy, x, w, m, r, None)[:3]
    for t, grad in ((x, dx), (w, dw), (b, db)):
        num = torch.empty_like(t).view(-1)
        for i in range(t.numel()):
            p, q = t.clone(), t.clone()
            p.view(-1)[i] += h
            q.view(-1)[i] -= h
            args = [[p if u is t else u for u in (x, w, b)], [q if u is t else u for u in (x, w, b)]]
            num[i] = (loss(*args[0]) - loss(*args[1])) / (2 * h)
        assert torch.allclose(num.view(t.shape), grad, atol=1e-7, rtol=1e-6)


# ---------------------------------------------------------------- activation backward
@pytest.mark.parametrize("act", list(ACTS))
def test_act_slopes_against_differences(act):
    x = torch.linspace(-6, 6, 997).double() + 1e-4  # off the kink of ReLU
    h = 1e-6
    num = (act64(x + h, act)[0] - act64(x - h, act)[0]) / (2 * h)
    assert torch.allclose(num, act64(x, act)[1], atol=1e-8)


def _act_grad64(dh, g, u, act):
    v, slope = act64(g, act)
    dh = dh.double()
    e1, es = act_error(g, v), act_error(g, torch.ones_like(v)) * (1 + g.double().abs())
    if u is None:
        return dh * slope, dh.abs() * es
    u = u.double()
    return (torch.cat((dh * u * slope, dh * v), 1),
            torch.cat(((dh * u).abs() * (es + 2.0 ** -23), dh.abs() * (e1 + 2.0 ** -23 * v.abs())), 1))


@pytest.mark.parametrize("act", list(ACTS))
@pytest.mark.parametrize("dtype,out", [(torch.float32, torch.float32), (torch.bfloat16, torch.bfloat16),
                                       (torch.bfloat16, torch.float32)])
@pytest.mark.parametrize("rows,n,gated", [(1, 1, True), (3, 33, False), (130, 256, True), (70, 2880, False), (9, 28672, True),
                                          (513, 100, True), (1000, 96, False), (70, 1002, True), (33, 131, True)])
def test_act_backward(act, dtype, out, rows, n, gated):
    dh, g = _rand((rows, n), n + rows, dtype), _rand((rows, n), n, dtype, 2.5)
    u = _rand((rows, n), rows, dtype) if gated else None
    g[0, 0] = 0.0
    if n > 8:
        g[0, 1:7] = torch.tensor([-30.0, 30.0, -90.0, 90.0, -3e38, 3e38])
    z64, err = _act_grad64(dh, g, u, act)
    w = 2 * n if gated else n
    ws = torch.full((fp4.fp4_act_backward_workspace_size(rows, n, gated),), 0xFF, dtype=torch.uint8, device="cuda")
    dhd, gd, ud = _cuda(dh, g, u)
    got = []
    for _ in range(2):
        z = torch.full((rows, w), float("nan"), dtype=out, device="cuda")
        db, amax = torch.full((w,), float("nan"), device="cuda"), torch.full((1,), float("nan"), device="cuda")
        fp4.fp4_act_backward(dhd, gd, ud, rows, n, CODE[dtype], ACTS[act], z, CODE[out], db, amax_out=amax, workspace=ws,
                             workspace_bytes=ws.numel())
        got.append((z, db, amax))
    assert all(torch.equal(p, q) for p, q in zip(*got)), "not the same bits twice"
    fin = torch.isfinite(z64.to(out))
    zf = torch.where(fin.cuda(), z, torch.zeros_like(z))
    assert_close(zf, torch.where(fin, z64, torch.zeros_like(z64)), torch.where(fin, err, torch.zeros_like(err)), "dZ")
    serial = (rows / 8 + 16 + 64) * 2.0 ** -24
    colfin = torch.isfinite(z64.float()).all(0) & (z64.abs().sum(0) < 1e30)
    assert_close(db[colfin.cuda()], z64.sum(0)[colfin], (serial * z64.abs().sum(0) + err.sum(0))[colfin], "dbias")


@pytest.mark.parametrize("fmt", [fp4.NVFP4, fp4.MXFP4])
@pytest.mark.parametrize("rows,n,gated", [(1, 32, True), (130, 96, True), (37, 2880, True), (128, 288, False), (5, 544, False)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_act_backward_codes(fmt, rows, n, gated, dtype):
    dh, g = _rand((rows, n), n, dtype), _rand((rows, n), n + 1, dtype, 2.0)
    u = _rand((rows, n), n + 2, dtype) if gated else None
    w = 2 * n if gated else n
    codes, scales = codes_like(rows, w, fmt)
    z, gs = torch.empty(rows, w, device="cuda"), torch.tensor([0.002], device="cuda")
    gin = gs if fmt == fp4.NVFP4 else None
    dhd, gd, ud = _cuda(dh, g, u)
    fp4.fp4_act_backward(dhd, gd, ud, rows, n, CODE[dtype], fp4.ACT_SILU, z, fp4.F32, fmt=fmt, codes=codes,
                         scales=scales, global_in=gin)
    assert fp4.fp4_get_status() == fp4.OK
    assert_codes_of(codes, scales, gs, z, fmt)
    codes2, scales2 = codes_like(rows, w, fmt)
    fp4.fp4_act_backward(dhd, gd, ud, rows, n, CODE[dtype], fp4.ACT_SILU, None, fp4.F32, fmt=fmt, codes=codes2,
                         scales=scales2, global_in=gin)
    assert torch.equal(codes, codes2) and torch.equal(scales, scales2)


def test_half_steps_are_those_of_the_types():
    for t, h in HALF_STEP.items():
        assert h == torch.finfo(t).eps / 2
