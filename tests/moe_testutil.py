"""64-bit references of the operators that bring tokens to their experts and back, and of the
products in 8-bit integers."""
from __future__ import annotations

import numpy as np
import torch

import block_scaled_fp4_04_b200 as fp4
from ffn_testutil import MAX_SLOPE, act64, act_error


def router_ids(tokens, topk, experts, seed, drop=0.0, dtype=torch.int64):
    """Distinct experts per token where there are enough, a share `drop` of them -1."""
    g = torch.Generator().manual_seed(seed)
    if topk <= experts:
        ids = torch.rand(tokens, experts, generator=g).topk(topk, 1).indices
    else:
        ids = torch.randint(0, experts, (tokens, topk), generator=g)
    return torch.where(torch.rand(tokens, topk, generator=g) < drop, -1, ids).to(dtype)


def sort_reference(ids: torch.Tensor, experts: int):
    """(offsets, row_of, scale_row_of) by counting, slot by slot."""
    flat = ids.reshape(-1).numpy()
    ok = (flat >= 0) & (flat < experts)
    count = np.bincount(flat[ok], minlength=experts)
    offsets = np.concatenate(([0], np.cumsum(count)))
    starts = np.concatenate(([0], np.cumsum((count + 127) // 128)))[:-1] * 128
    row_of = np.full(flat.size, -1, np.int64)
    srow = np.full(flat.size, -1, np.int64)
    for e in range(experts):
        at = np.flatnonzero(flat == e)
        row_of[at] = offsets[e] + np.arange(at.size)
        srow[at] = starts[e] + np.arange(at.size)
    shape = tuple(ids.shape)
    return [torch.from_numpy(np.ascontiguousarray(a)).int() for a in (offsets, row_of.reshape(shape), srow.reshape(shape))]


def dispatched(x: torch.Tensor, row_of: torch.Tensor, fill: torch.Tensor) -> torch.Tensor:
    """fill with the tokens' rows in the experts' order."""
    y = fill.clone()
    t, j = torch.nonzero(row_of >= 0, as_tuple=True)
    y[row_of[t, j].long()] = x[t].to(y.dtype)
    return y


def combine64(y, row_of, weights, residual=None):
    """(sum_j w y, sum of the terms' magnitudes) in 64 bits."""
    on = row_of >= 0
    w = torch.ones(row_of.shape, dtype=torch.float64) if weights is None else weights.double()
    terms = torch.where(on[..., None], y.double()[row_of.clamp(min=0).long()] * w[..., None], 0.0)
    out, mag = terms.sum(1), terms.abs().sum(1)
    return (out, mag) if residual is None else (out + residual.double(), mag + residual.double().abs())


def i8_rows(x: torch.Tensor):
    """8-bit rows and scales by the definition: each 64-bit operation rounded to 32 bits."""
    x = x.double()
    top = x.abs().max(-1).values
    s = (top / 127).float().double().clamp(min=2.0 ** -126)
    s = torch.where(top == 0, torch.ones_like(s), s)
    inv = (1 / s).float().double()
    return torch.round((x * inv[..., None]).float()).to(torch.int8), s.float()


def random_i8(shape, seed, extreme=False):
    """Values over the whole range, or only the ends, and positive scales."""
    g = torch.Generator().manual_seed(seed)
    if extreme:
        q = torch.where(torch.rand(shape, generator=g) < 0.5, -128, 127).to(torch.int8)
    else:
        q = torch.randint(-128, 128, shape, generator=g, dtype=torch.int8)
    return q, torch.rand(shape[:-1], generator=g) * 0.02 + 1e-3


def product_i8(a, sa, b, sb, bias=None, act="none"):
    """(result, FP32 error bound) of act(sa sb sum + bias): the sum is exact; its conversion and the two
    products round by 2^-24 each, the bias's sum once more."""
    z0 = (a.double() @ b.double().t()) * sa.double()[:, None] * sb.double()[None]
    z = z0 if bias is None else z0 + bias.double()
    value, _ = act64(z, act)
    err = MAX_SLOPE * (3.01 * 2.0 ** -24 * z0.abs() + 2.0 ** -24 * z.abs() + 1e-37)
    return value, err + (act_error(z, value) if act not in ("none", "relu") else 0.0)


def to_cuda(r):
    return [None if t is None else t.cuda() for t in r]
