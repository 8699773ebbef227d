"""Products in 8-bit integers on the GPU: the row quantizer bit by bit, the products against exact
sums in 64 bits, dense and by experts."""
import pytest
import torch

import block_scaled_fp4_04_b200 as fp4
from ffn_testutil import ACTS, CODE, assert_close
from fp4_testutil import random_input
from moe_testutil import i8_rows, product_i8, random_i8

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("rows,cols", [(1, 16), (3, 32), (16, 8192), (129, 2880), (1000, 48), (7, 32784), (2, 131088)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_quantize(rows, cols, dtype):
    x = random_input(rows, cols, rows + cols, dtype)
    x[0, 0] = 0.0
    if rows > 2:
        x[1] = 0                       # a row of zeros
        x[2] = x[2] * 2.0 ** -124      # whose scale is the smallest one (a subnormal row in FP32)
    if rows > 6:
        x[3] = x[3] * 2.0 ** 100
        x[4] = 0
        x[4, cols - 1] = -3.0          # one value
        x[5] = torch.arange(cols) % 255 - 127.0      # whole numbers stay
        x[6] = (torch.arange(cols) % 254 - 126.5)    # ties
        x[6, 0] = 127.0
    q, s = i8_rows(x)
    codes = torch.full((rows, cols), 99, dtype=torch.int8, device="cuda")
    scales = torch.full((rows,), -1.0, device="cuda")
    fp4.fp4_quantize_i8(x.cuda(), rows, cols, CODE[dtype], codes, scales)
    assert torch.equal(scales.cpu(), s)
    assert torch.equal(codes.cpu(), q)
    assert fp4.fp4_get_status() == fp4.OK


def test_quantize_reports_what_is_not_finite():
    for bad in (float("inf"), float("-inf"), float("nan")):
        for at in (0, 4095):
            x = torch.ones(5, 4096, dtype=BF16)
            x[3, at] = bad
            fp4.quantize_i8(x.cuda())
            assert fp4.fp4_get_status() == fp4.ERR_NONFINITE
    assert fp4.fp4_get_status() == fp4.OK


def _gemm(a, sa, b, sb, bias=None, act="none", out=F32, flags=0, ws=None):
    m, k = a.shape
    n = b.shape[0]
    d = torch.full((m, n), float("nan"), dtype=out, device="cuda")
    size = fp4.fp4_gemm_i8_workspace_size(m, n, k)
    if ws is None:
        ws = torch.zeros(max(size, 1), dtype=torch.uint8, device="cuda")
    fp4.fp4_gemm_i8(a, sa, b, sb, m, n, k, bias, ACTS[act], d, CODE[out], ws, ws.numel(), flags)
    torch.cuda.synchronize()
    assert fp4.fp4_get_status() == fp4.OK
    assert not ws.any(), "workspace not left zero-filled"
    return d


SHAPES = [(1, 1, 16), (1, 128, 128), (3, 5, 48), (16, 256, 128), (16, 640, 4096), (17, 300, 272), (32, 129, 1024),
          (33, 1000, 512), (64, 257, 2880), (65, 130, 144), (100, 100, 16), (128, 512, 512), (129, 128, 256),
          (200, 2000, 640), (256, 256, 256), (300, 5000, 320), (513, 2049, 1040), (1999, 1111, 912), (2500, 3000, 128),
          (20, 300, 4400), (32, 1001, 4112), (50, 257, 4112), (64, 2000, 8192)]


@pytest.mark.parametrize("m,n,k", SHAPES)
def test_gemm_sums_are_exact(m, n, k):
    """Scales of 1 and sums below 2^24: FP32 holds every result exactly."""
    a, b = random_i8((m, k), m + k)[0], random_i8((n, k), n + 1)[0]
    if k * 128 * 128 > 2 ** 24:
        a = a // 16
        if k * 8 * 128 > 2 ** 24:
            a = a.clamp(-1, 1)
    one_m, one_n = torch.ones(m, device="cuda"), torch.ones(n, device="cuda")
    d = _gemm(a.cuda(), one_m, b.cuda(), one_n)
    want = a.double() @ b.double().t()
    assert want.abs().max() <= 2 ** 24
    bad = torch.nonzero(d.cpu().double() != want)
    assert len(bad) == 0, f"{len(bad)} of {d.numel()} differ, first {bad[0].tolist()}"


@pytest.mark.parametrize("m,n,k", SHAPES)
@pytest.mark.parametrize("out", [BF16, F32])
@pytest.mark.parametrize("act,with_bias", [("none", False), ("relu", True), ("silu", True), ("gelu", False), ("gelu_tanh", True)])
def test_gemm(m, n, k, out, act, with_bias):
    (a, sa), (b, sb) = random_i8((m, k), m + k), random_i8((n, k), n + 1)
    sb = sb / (20 * k ** 0.5)  # results around 1, where the activations bend
    bias = torch.randn(n, generator=torch.Generator().manual_seed(3)) if with_bias else None
    d = _gemm(a.cuda(), sa.cuda(), b.cuda(), sb.cuda(), None if bias is None else bias.cuda(), act, out)
    want, err = product_i8(a, sa, b, sb, bias, act)
    assert_close(d, want, err, f"{m}x{n}x{k} {act}")


@pytest.mark.parametrize("m,k", [(1, 131056), (40, 131056), (300, 65536)])
def test_gemm_of_the_largest_sums(m, k):
    """Every product at an end of the range; all of one sign in some rows."""
    n = 300
    (a, sa), (b, sb) = random_i8((m, k), 5, True), random_i8((n, k), 6, True)
    a[0] = -128
    b[0] = -128
    b[1] = 127
    d = _gemm(a.cuda(), sa.cuda(), b.cuda(), sb.cuda())
    want, err = product_i8(a, sa, b, sb)
    assert_close(d, want, err)
    assert want[0, 0] > 2 ** 14 * k * 1e-6 * 0.9


@pytest.mark.parametrize("m,n,k", [(1, 8192, 8192), (16, 4096, 8192), (50, 3000, 4096), (25, 3000, 8192), (60, 500, 8192), (128, 1024, 8192),
                                   (8192, 512, 512)])
def test_gemm_has_the_same_bits_every_time(m, n, k):
    (a, sa), (b, sb) = random_i8((m, k), 1), random_i8((n, k), 2)
    a, sa, b, sb = a.cuda(), sa.cuda(), b.cuda(), sb.cuda()
    ws = torch.zeros(max(1, fp4.fp4_gemm_i8_workspace_size(m, n, k)), dtype=torch.uint8, device="cuda")
    first = _gemm(a, sa, b, sb, ws=ws)
    for _ in range(10):
        assert torch.equal(_gemm(a, sa, b, sb, ws=ws), first)


@pytest.mark.parametrize("n", [256, 4096, 28672])
@pytest.mark.parametrize("m,k", [(16, 512), (5, 8192), (64, 2048)])
def test_early_weights_after_the_quantizer(m, n, k):
    """Weights that are ready: the product starts while the quantizer runs; calls back to back on
    changing activations, one workspace."""
    w = fp4.quantize_i8(random_input(n, k, 1, BF16, std=0.02).cuda())
    xs = [random_input(m, k, s, BF16).cuda() for s in (2, 3)]
    size = fp4.fp4_gemm_i8_workspace_size(m, n, k)
    ws = torch.zeros(max(1, size), dtype=torch.uint8, device="cuda")
    want = [fp4.gemm_i8(fp4.quantize_i8(x), w, out_dtype=F32) for x in xs]
    torch.cuda.synchronize()
    codes, scales = torch.zeros(m, k, dtype=torch.int8, device="cuda"), torch.zeros(m, device="cuda")
    got = [torch.empty(m, n, device="cuda") for _ in range(20)]
    for i, d in enumerate(got):
        fp4.fp4_quantize_i8(xs[i % 2], m, k, fp4.BF16, codes, scales)
        fp4.fp4_gemm_i8(codes, scales, w.codes, w.scales, m, n, k, None, fp4.ACT_NONE, d, fp4.F32, ws, ws.numel(),
                        fp4.GEMM_WEIGHTS_READY)
    torch.cuda.synchronize()
    wrong = [i for i, d in enumerate(got) if not torch.equal(d, want[i % 2])]
    assert not wrong, f"calls {wrong}"
    assert not ws.any()


def test_one_workspace_for_all_shapes():
    shapes = [(16, 4096, 2048), (128, 640, 4096), (1, 1000, 8192), (60, 2048, 1024), (32, 500, 4096)]
    ws = torch.zeros(max(fp4.fp4_gemm_i8_workspace_size(*s) for s in shapes), dtype=torch.uint8, device="cuda")
    for m, n, k in shapes * 2:
        (a, sa), (b, sb) = random_i8((m, k), m), random_i8((n, k), n)
        want, err = product_i8(a, sa, b, sb)
        assert_close(_gemm(a.cuda(), sa.cuda(), b.cuda(), sb.cuda(), ws=ws), want, err)


def _offsets(rows, experts, seed, skew=False, behind=0):
    g = torch.Generator().manual_seed(seed)
    if skew:  # one expert takes nearly all
        counts = torch.zeros(experts, dtype=torch.int64)
        counts[experts // 2] = rows - behind
    else:
        at = torch.randint(0, experts, (rows - behind,), generator=g)
        counts = torch.bincount(at, minlength=experts)
    return torch.cat((torch.zeros(1, dtype=torch.int64), counts.cumsum(0))).int()


@pytest.mark.parametrize("rows,experts,n,k,skew,behind", [
    (1, 1, 16, 16, False, 0), (7, 4, 100, 64, False, 2), (64, 32, 576, 288, False, 0), (64, 64, 130, 2880, True, 10),
    (300, 8, 257, 512, False, 0), (500, 5, 300, 144, True, 33), (1500, 3, 640, 272, False, 100), (3000, 20, 512, 384, False, 1),
    (4000, 8, 520, 128, True, 0), (2048, 1024, 96, 96, False, 0), (9, 3, 128, 1024, False, 9)])
@pytest.mark.parametrize("out", [BF16, F32])
def test_grouped(rows, experts, n, k, skew, behind, out):
    off = _offsets(rows, experts, rows + n, skew, behind)
    (a, sa), (b, sb) = random_i8((rows, k), 1), random_i8((experts, n, k), 2)
    bias = torch.randn(experts, n, generator=torch.Generator().manual_seed(3))
    size = fp4.fp4_gemm_i8_grouped_workspace_size(experts, rows, n, k)
    ws = torch.zeros(max(1, size), dtype=torch.uint8, device="cuda")
    dev = [t.cuda() for t in (off, a, sa, b, sb)]
    first = None
    for with_bias in (True, True, False):
        d = torch.full((rows, n), 7.0, dtype=out, device="cuda")
        fp4.fp4_gemm_i8_grouped(experts, *dev, rows, n, k, bias.cuda() if with_bias else None, fp4.ACT_NONE, d, CODE[out], ws,
                                ws.numel())
        torch.cuda.synchronize()
        assert fp4.fp4_get_status() == fp4.OK and not ws.any()
        assert (d[rows - behind:] == 7.0).all(), "rows behind the last expert"
        for e in range(experts):
            lo, hi = int(off[e]), int(off[e + 1])
            if lo < hi:
                want, err = product_i8(a[lo:hi], sa[lo:hi], b[e], sb[e], bias[e] if with_bias else None)
                assert_close(d[lo:hi], want, err, f"expert {e}")
        if with_bias:
            first = d if first is None else first
            assert torch.equal(d, first)


def test_two_captured_graphs_with_workspaces_of_their_own():
    m, n, k = 16, 2048, 4096
    w = fp4.quantize_i8(random_input(n, k, 1, BF16, std=0.02).cuda())
    xs = [random_input(m, k, s, BF16).cuda() for s in (2, 3)]
    want = [fp4.gemm_i8(fp4.quantize_i8(x), w) for x in xs]
    graphs = []
    for x in xs:
        ws = fp4.Workspace()
        fp4.gemm_i8(fp4.quantize_i8(x), w, workspace=ws)  # grows before the capture
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            d = fp4.gemm_i8(fp4.quantize_i8(x), w, workspace=ws)
        graphs.append((g, d, ws))
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(20):
        for (g, _, _), st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    for (_, d, ws), t in zip(graphs, want):
        assert torch.equal(d, t) and not ws.buf.any()


def test_on_another_stream():
    m, n, k = 100, 500, 1024
    w = fp4.quantize_i8(random_input(n, k, 1, BF16, std=0.02).cuda())
    x = random_input(m, k, 2, BF16).cuda()
    want = fp4.gemm_i8(fp4.quantize_i8(x), w, out_dtype=F32)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = fp4.gemm_i8(fp4.quantize_i8(x, stream=side), w, out_dtype=F32, stream=side)
    raw = torch.empty_like(want)
    codes, scales = torch.empty(m, k, dtype=torch.int8, device="cuda"), torch.empty(m, device="cuda")
    torch.cuda.synchronize()
    fp4.fp4_quantize_i8(x, m, k, fp4.BF16, codes, scales, None, side.cuda_stream)
    fp4.fp4_gemm_i8(codes, scales, w.codes, w.scales, m, n, k, None, fp4.ACT_NONE, raw, fp4.F32, stream=side)
    side.synchronize()
    assert torch.equal(got, want) and torch.equal(raw, want)


def test_quantize_stops_at_a_row_count_on_the_device():
    x = random_input(50, 256, 1, BF16)
    x[30:] = float("nan")
    q, s = i8_rows(x[:30])
    for valid in (0, 17, 30):
        codes, scales = torch.full((50, 256), 99, dtype=torch.int8, device="cuda"), torch.full((50,), -1.0, device="cuda")
        fp4.fp4_quantize_i8(x.cuda(), 50, 256, fp4.BF16, codes, scales, torch.tensor([valid], dtype=torch.int32, device="cuda"))
        assert fp4.fp4_get_status() == fp4.OK
        assert torch.equal(codes[:valid].cpu(), q[:valid]) and torch.equal(scales[:valid].cpu(), s[:valid])
        assert (codes[valid:] == 99).all() and (scales[valid:] == -1).all()


def test_weights_beyond_32_bit_offsets():
    """N K and M N beyond 2^31."""
    m, n, k = 40, 70000, 32768
    b = torch.zeros(n, k, dtype=torch.int8, device="cuda")
    sb = torch.ones(n, device="cuda")
    rows = torch.tensor([0, 65535, 65536, 69999])
    q, _ = random_i8((4, k), 1)
    b[rows] = q.cuda()
    a, sa = random_i8((m, k), 2)
    d = _gemm(a.cuda(), sa.cuda(), b, sb)
    want, err = product_i8(a, sa, q, torch.ones(4))
    assert_close(d[:, rows.cuda()], want, err)
    d[:, rows.cuda()] = 0
    assert not d.any()
    del b, d
    m, n, k = 33000, 66000, 16  # outputs beyond 2^31
    (a, sa), (b, sb) = random_i8((m, k), 3), random_i8((n, k), 4)
    d = torch.empty(m, n, dtype=BF16, device="cuda")
    fp4.fp4_gemm_i8(a.cuda(), sa.cuda(), b.cuda(), sb.cuda(), m, n, k, None, fp4.ACT_NONE, d, fp4.BF16)
    for r in (0, 32999, 32767, 16500):
        want, err = product_i8(a[r:r + 1], sa[r:r + 1], b, sb)
        assert_close(d[r:r + 1], want, err)
