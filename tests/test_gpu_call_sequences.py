"""Calls that follow one another on a stream without a synchronization between them."""
import pytest
import torch

import block_scaled_fp4_04_b200 as fp4
from fp4_testutil import gpu_quantize, random_input

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


class _FromBf16:
    """A product from BF16 activations (gated or not) with its output buffers."""

    def __init__(self, m, n, k, seed, gated=False):
        self.m, self.n, self.k, self.gated = m, n, k, gated
        self.q = gpu_quantize(random_input(n, k, seed, torch.float32, outliers=False).cuda(), fp4.NVFP4, 16)
        self.d = torch.empty(m, n, device="cuda")
        self.codes = torch.empty(m, k // 2, dtype=torch.uint8, device="cuda")
        self.scales = torch.empty(fp4.fp4_scales_bytes(m, k, fp4.NVFP4), dtype=torch.uint8, device="cuda")
        self.g = torch.empty(1, device="cuda")

    def size(self):
        return (fp4.fp4_gemm_gated_bf16a_workspace_size if self.gated else fp4.fp4_gemm_bf16a_workspace_size)(
            self.m, self.n, self.k)

    def __call__(self, x, ws):
        q, d = self.q, self.d
        d.fill_(float("nan"))
        if self.gated:
            fp4.fp4_gemm_gated_bf16a(x, q.codes, q.scales, q.g, q.codes, q.scales, q.g, self.m, self.n, self.k, None, None,
                                     fp4.ACT_NONE, d, fp4.F32, None, None, self.codes, self.scales, self.g, ws, ws.numel())
        else:
            fp4.fp4_gemm_bf16a(x, q.codes, q.scales, q.g, self.m, self.n, self.k, d, fp4.F32, self.codes, self.scales,
                               self.g, ws, ws.numel())
        return d.clone(), self.codes.clone(), self.scales.clone(), self.g.clone()


@pytest.mark.parametrize("m,k,n,gated", [(16, 1024, 512, False), (5, 2048, 640, True), (32, 512, 256, False)])
def test_one_workspace_for_products_of_other_shapes(m, k, n, gated):
    """A second shape's partial sums end among the first one's slots and counters: each call finds
    the workspace as the one before it left it, zero-filled."""
    # where the first shape's slots start, in rows of the second one's sums
    halves = 2 if gated else 1
    wider = n * halves + (-(-n // 128) * 4 * halves + 256 + 40 * 128) // (m * 4)
    a, b = _FromBf16(m, n, k, 1, gated), _FromBf16(m, wider, k, 2)
    ws = torch.zeros(max(a.size(), b.size()), dtype=torch.uint8, device="cuda")
    plain = fp4.fp4_gemm_workspace_size(m, wider, k, fp4.NVFP4)
    for call in range(4):
        # activations of another size each time: an old maximum would give another scale
        x = (random_input(m, k, 10 + call, torch.float32, outliers=False) * 4.0 ** -call).to(torch.bfloat16).cuda()
        for f in (a, b):
            got = f(x, ws)
            torch.cuda.synchronize()
            assert fp4.fp4_get_status() == fp4.OK
            assert not ws.any(), "workspace not left zero-filled"
            want = f(x, torch.zeros(f.size(), dtype=torch.uint8, device="cuda"))
            for p, q in zip(got[1:], want[1:]):
                assert torch.equal(p, q)
            check_gemm_like(got[0], want[0])
            # (a tensor as the divisor: by a number, torch multiplies with its rounded reciprocal)
            assert torch.equal(got[3].cpu(), x.abs().max().float().cpu().reshape(1) / torch.tensor([2688.0]))
        d = torch.empty(m, wider, device="cuda")
        fp4.fp4_gemm(fp4.NVFP4, b.codes, b.scales, b.g, b.q.codes, b.q.scales, b.q.g, m, wider, k, d, fp4.F32, ws, plain)
        check_gemm_like(d, want[0])
    x[m // 2, 7] = float("inf")  # refused on the device; the workspace is clean all the same
    a(x, ws)
    assert fp4.fp4_get_status() == fp4.ERR_NONFINITE and not ws.any()


def test_a_capture_that_needs_a_larger_workspace():
    """Calls captured with a workspace that is too small, eager calls with it before and after the
    first replay, and when the graph is gone."""
    m, n, k = 16, 640, 2048
    qa, qb = (gpu_quantize(random_input(r, k, s, torch.float32, outliers=False).cuda(), fp4.NVFP4, 16)
              for r, s in ((m, 1), (n, 2)))
    want = fp4.gemm(qa, qb, torch.float32)
    ws = fp4.Workspace()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        junk = torch.full((1 << 20,), 255, dtype=torch.uint8, device="cuda")
        del junk
        d1 = fp4.gemm(qa, qb, torch.float32, ws)
        d2 = fp4.gemm_epilogue(qa, qb, residual=d1, out_dtype=torch.float32, workspace=ws)
    for _ in range(3):
        check_gemm_like(fp4.gemm(qa, qb, torch.float32, ws), want)
        d1.fill_(float("nan"))
        graph.replay()
        check_gemm_like(d1, want)
        check_gemm_like(d2 / 2, want)
    torch.cuda.synchronize()
    del graph, d1, d2
    torch.cuda.empty_cache()
    check_gemm_like(fp4.gemm(qa, qb, torch.float32, ws), want)
    torch.cuda.synchronize()
    assert not ws.buf.any() and fp4.fp4_get_status() == fp4.OK


def check_gemm_like(got, want):
    """The same products, their FP32 partial sums added in any order: sums of at most 8 parts (K <=
    2048 in steps of 256), each within 2^-24 of the sum of magnitudes, which random signs keep
    within 64 times the largest result."""
    assert (got - want).abs().max() <= 2 * 8 * 2.0 ** -24 * 64 * want.abs().max()
