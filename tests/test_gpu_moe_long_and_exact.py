"""The sort beyond 2^21 slots, where a warp's segment no longer stays in registers, and the whole way's
gradients on values that FP32 holds exactly, so that formula and difference are equal."""
import pytest
import torch

import block_scaled_fp4_04_b200 as fp4
from moe_testutil import router_ids, sort_reference

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("tokens,topk,experts,drop", [
    (1 << 21, 1, 7, 0.0),        # the last size with segments of 512
    ((1 << 21) + 1, 1, 5, 0.3), (700001, 4, 300, 0.1), (1 << 20, 3, 1024, 0.0), (2500000, 1, 1, 0.5)])
@pytest.mark.parametrize("dtype", [torch.int32, torch.int64])
def test_sort_of_long_segments(tokens, topk, experts, drop, dtype):
    g = torch.Generator().manual_seed(tokens)
    ids = torch.randint(0, experts, (tokens, topk), generator=g, dtype=dtype)
    ids[torch.rand(tokens, topk, generator=g) < drop] = -1
    r = fp4.moe_sort(ids.cuda(), experts)
    for got, want, name in zip((r.offsets, r.row_of, r.scale_row_of), sort_reference(ids, experts),
                               ("offsets", "row_of", "scale_row_of")):
        assert torch.equal(got.cpu(), want), name


@pytest.mark.parametrize("tokens,topk,experts,cols", [(40, 3, 6, 100), (64, 2, 4, 64), (33, 5, 8, 129), (20, 9, 16, 50)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_gradients_equal_differences_of_exact_values(tokens, topk, experts, cols, dtype):
    """The sum <dout, combine(scale dispatch(x), w)> is linear in x and in w.  Whole numbers up to 8 in x and
    dout, quarters up to 2 in w, powers of two in scale: rows are whole numbers up to 32 and dy quarters up
    to 16 (7 bits, exact in BF16), every sum a multiple of 1/4 below 2^18 (exact in FP32 in any order).  So the
    derivative along a direction is the difference itself, with no tolerance."""
    g = torch.Generator().manual_seed(tokens)
    routing = fp4.moe_sort(router_ids(tokens, topk, experts, 3, 0.2).cuda(), experts)
    x, dx_dir, dout = (torch.randint(-8, 9, (tokens, cols), generator=g).to(dtype).cuda() for _ in range(3))
    w, dw_dir = (torch.randint(-8, 9, (tokens, topk), generator=g).float().cuda() / 4 for _ in range(2))
    scale = 2.0 ** torch.randint(0, 3, (tokens * topk, 1), generator=g).to(dtype).cuda()

    def rows(x):
        return fp4.moe_dispatch(x, routing) * scale

    def loss(y, w):
        return (fp4.moe_combine(y, routing, w, out_dtype=F32).double() * dout.double()).sum().item()

    y = rows(x)
    dy, dw = fp4.moe_combine_backward(dout, y, routing, w)
    dx = fp4.moe_dispatch_backward(dy * scale, routing, out_dtype=F32)
    along_x, along_w = (dx.double() * dx_dir.double()).sum().item(), (dw.double() * dw_dir.double()).sum().item()
    assert along_x == loss(rows(dx_dir), w) and along_w == loss(y, dw_dir)
    assert along_x != 0 and along_w != 0  # the directions say something
    # and element by element, against the formula
    row_of = routing.row_of.cpu()
    on = (row_of >= 0)[..., None].double()
    at = row_of.clamp(min=0).long()
    sc, d = scale.cpu().double()[at], dout.cpu().double()
    assert torch.equal(dx.cpu().double(), (on * sc * w.cpu().double()[..., None]).sum(1) * d)
    assert torch.equal(dw.cpu().double(), (on * sc * (x.cpu().double() * d)[:, None]).sum(2))
