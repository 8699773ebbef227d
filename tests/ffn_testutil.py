"""64-bit references and derived tolerances of the operators around the FP4 products (layer
norm, gated GEMM, activation backward, epilogue with residual)."""
from __future__ import annotations

import math

import numpy as np
import torch

import block_scaled_fp4_04_b200 as fp4
import oracle
from fp4_testutil import host_input

ACTS = {"none": fp4.ACT_NONE, "relu": fp4.ACT_RELU, "silu": fp4.ACT_SILU, "gelu": fp4.ACT_GELU,
        "gelu_tanh": fp4.ACT_GELU_TANH}
HALF_STEP = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
CODE = {torch.float32: fp4.F32, torch.bfloat16: fp4.BF16}


def act64(x: torch.Tensor, act: str):
    """(value, slope) of an activation in 64 bits."""
    x = x.double()
    if act == "none":
        return x, torch.ones_like(x)
    if act == "relu":
        return x.clamp(min=0.0), (x > 0).double()
    if act == "silu":
        s = torch.sigmoid(x)
        return x * s, s + x * s * (1 - s)
    if act == "gelu":
        phi = torch.special.ndtr(x)
        return x * phi, phi + x * torch.exp(-x * x / 2) / math.sqrt(2 * math.pi)
    c = math.sqrt(2 / math.pi)
    t = torch.tanh(c * (x + 0.044715 * x ** 3))
    return x / 2 * (1 + t), (1 + t) / 2 + x / 2 * (1 - t * t) * c * (1 + 3 * 0.044715 * x * x)


def act_error(x: torch.Tensor, value: torch.Tensor) -> torch.Tensor:
    """Bound of the FP32 error of an activation's value, and of its slope with value = 1.

    The argument y of the exponential is at most |x| (1 + |x|^2 / 10) for |x| below the region
    where the sigmoid is 0 or 1 to 2^-24, takes a few roundings (2^-22 |y| together), and an
    error d of it changes s by at most s d; the exponential and the reciprocal add 2^-21 each;
    erf is good to 2^-23 absolute, and is multiplied by |x|."""
    x = x.double().abs()
    y = torch.minimum(1.6 * x * (1 + 0.045 * x * x), torch.full_like(x, 100.0))
    return value.double().abs() * (2.0 ** -20 + 2.0 ** -21 * y) + 2.0 ** -22 * (x + 1)


MAX_SLOPE = 1.13  # of SILU (1.0998) and GELU (1.129)


def dequantized(q: fp4.Quantized) -> np.ndarray:
    """Values of a quantized operand on the device, by the oracle's decoder."""
    blk = 16 if q.fmt == fp4.NVFP4 else 32
    sc = oracle.unswizzle_scales(q.scales.cpu().numpy(), q.rows, q.cols // blk)
    return oracle.dequantize(q.codes.cpu().numpy(), sc, q.g.item(), q.fmt)


def product64(a: np.ndarray, b: np.ndarray):
    """a b^T in 64 bits and the kernel's bound of its FP32 error (1e-6 sum |a b|)."""
    a, b = torch.from_numpy(a), torch.from_numpy(b)
    return a @ b.t(), 1e-6 * (a.abs() @ b.abs().t())


def assert_close(got: torch.Tensor, want: torch.Tensor, err: torch.Tensor, label=""):
    """|got - want| <= err plus half a step of got's type."""
    g = got.detach().cpu().double()
    tol = err + HALF_STEP[got.dtype] * (want.abs() + err) + 1e-37
    bad = torch.nonzero(~((g - want).abs() <= tol))
    assert bad.numel() == 0, (f"{label}: {len(bad)} of {g.numel()} outside tolerance; first {bad[0].tolist()}: "
                              f"got {g[tuple(bad[0])]}, want {want[tuple(bad[0])]}, tol {tol[tuple(bad[0])]}")


def assert_codes_of(codes, scales, g, values: torch.Tensor, fmt: int, label=""):
    """Codes and scale atoms (pads included) are those of quantizing the FP32 values."""
    rows, cols = values.shape
    blk = 16 if fmt == fp4.NVFP4 else 32
    oq = oracle.quantize(host_input(values), fmt, blk, g_in=np.float32(g.item()) if fmt == fp4.NVFP4 else None)
    bad = np.argwhere(codes.cpu().numpy() != oq["codes"])
    assert bad.size == 0, f"{label}: {len(bad)} code bytes differ, first {bad[:3].tolist()}"
    bad = np.flatnonzero(scales.cpu().numpy() != oracle.swizzle_scales(oq["scales"]))
    assert bad.size == 0, f"{label}: {bad.size} scale bytes differ, first {bad[:3].tolist()}"


def codes_like(rows, cols, fmt):
    """Output buffers for codes, filled with a pattern that must not survive."""
    return (torch.full((rows, cols // 2), 0x5A, dtype=torch.uint8, device="cuda"),
            torch.full((fp4.fp4_scales_bytes(rows, cols, fmt),), 0xA5, dtype=torch.uint8, device="cuda"))
