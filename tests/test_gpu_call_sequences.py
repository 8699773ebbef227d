"""Calls that follow one another on a stream without a synchronization between them."""
import pytest
import torch

import block_scaled_fp4_04_b200 as fp4
from fp4_testutil import random_input

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("middle", ["layernorm", "quantize"])
@pytest.mark.parametrize("gated", [False, True])
def test_weights_written_two_kernels_before_a_product_that_may_read_them_early(middle, gated):
    """FP4_GEMM_WEIGHTS_READY: the weights were written before the kernel just before the product.
    Here by the kernel before that one, whose work takes longer than the start of the next two."""
    m, n, k = 128, 2048, 512
    w = [random_input(n, k, s, torch.bfloat16, std=0.02 * s, outliers=False).cuda() for s in (1, 3)]
    one = torch.ones(n, k, dtype=torch.bfloat16, device="cuda")
    x = random_input(m, k, 5, torch.bfloat16, outliers=False).cuda()
    gw, gx = torch.tensor([1e-4], device="cuda"), torch.tensor([2e-3], device="cuda")
    codes = torch.zeros(n, k // 2, dtype=torch.uint8, device="cuda")
    scales = torch.zeros(fp4.fp4_scales_bytes(n, k, fp4.NVFP4), dtype=torch.uint8, device="cuda")
    xc = torch.zeros(m, k // 2, dtype=torch.uint8, device="cuda")
    xs = torch.zeros(fp4.fp4_scales_bytes(m, k, fp4.NVFP4), dtype=torch.uint8, device="cuda")
    xg = torch.empty(1, device="cuda")

    def run(i, d, wait):
        # the codes of w[i], as the gradient of an activation whose slope is 1 everywhere
        fp4.fp4_act_backward(w[i], one, None, n, k, fp4.BF16, fp4.ACT_RELU, None, fp4.F32, None, fp4.NVFP4, codes, scales,
                             gw)
        wait()
        if middle == "layernorm":
            fp4.fp4_layernorm(x, m, k, fp4.BF16, None, None, 1e-5, None, fp4.F32, None, None, fp4.NVFP4, xc, xs, gx)
        else:
            fp4.fp4_quantize(x, m, k, fp4.BF16, fp4.NVFP4, 16, xc, xs, xg, None, None, gx)
        wait()
        if gated:
            fp4.fp4_gemm_gated(fp4.NVFP4, xc, xs, gx, codes, scales, gw, codes, scales, gw, m, n, k, None, None,
                               fp4.ACT_SILU, d, fp4.F32, flags=fp4.GEMM_WEIGHTS_READY)
        else:
            fp4.fp4_gemm_ex(fp4.NVFP4, xc, xs, gx, codes, scales, gw, m, n, k, d, fp4.F32,
                            flags=fp4.GEMM_WEIGHTS_READY)

    want = [torch.empty(m, n, device="cuda") for _ in w]
    for i in (0, 1):
        run(i, want[i], torch.cuda.synchronize)
        torch.cuda.synchronize()
    assert not torch.equal(want[0], want[1])
    got = [torch.empty(m, n, device="cuda") for _ in range(100)]
    for r, d in enumerate(got):
        run(r % 2, d, lambda: None)
    torch.cuda.synchronize()
    # no sum is split over K at this size: the same bits every time
    wrong = [r for r, d in enumerate(got) if not torch.equal(d, want[r % 2])]
    assert not wrong, f"{len(wrong)} of {len(got)} products read weights that were not there yet"
    assert fp4.fp4_get_status() == fp4.OK
