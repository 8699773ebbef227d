"""The largest number of rows that the 8-bit products take (2^31 - 256): their tiles' sums pass 31 bits."""
import pytest
import torch

import block_scaled_fp4_04_b200 as fp4
from moe_testutil import random_i8

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("by_expert", [False, True])
def test_the_largest_number_of_rows(by_expert):
    m, n, k = (1 << 31) - 256, 1, 16
    at = torch.tensor([0, 127, 128, 255, 256, (1 << 30) + 5, 2139095041, m - 257, m - 256, m - 129, m - 1])
    q, _ = random_i8((len(at), k), 1)
    b, _ = random_i8((n, k), 2)
    a = torch.zeros(m, k, dtype=torch.int8, device="cuda")
    a[at.cuda()] = q.cuda()
    sa, sb = torch.ones(m, device="cuda"), torch.ones(n, device="cuda")
    sa[m - 1] = 0.5
    d = torch.full((m, n), 7.0, dtype=torch.float32, device="cuda")
    if by_expert:  # all rows but one are the second of three experts'
        off = torch.tensor([0, 1, m, m], dtype=torch.int32, device="cuda")
        assert fp4.fp4_gemm_i8_grouped_workspace_size(3, m, n, k) == 0
        fp4.fp4_gemm_i8_grouped(3, off, a, sa, b.cuda().repeat(3, 1), sb.repeat(3), m, n, k, None, fp4.ACT_NONE, d, fp4.F32)
    else:
        assert fp4.fp4_gemm_i8_workspace_size(m, n, k) == 0
        fp4.fp4_gemm_i8(a, sa, b.cuda(), sb, m, n, k, None, fp4.ACT_NONE, d, fp4.F32)
    assert fp4.fp4_get_status() == fp4.OK
    want = (q.double() @ b.double().t()).squeeze(1)  # whole numbers below 2^18: exact in FP32
    want[-1] *= 0.5
    assert torch.equal(d[at.cuda(), 0].cpu().double(), want)
    d[at.cuda()] = 0
    assert not d.any()
