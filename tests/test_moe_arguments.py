"""Refusals of the experts' and the 8-bit entry points on the host, before anything is enqueued (no
GPU needed), workspace sizes, and the conveniences' checks of their operands."""
import pytest
import torch

import block_scaled_fp4_04_b200 as fp4
from block_scaled_fp4_04_b200 import build as fp4_build


@pytest.fixture(scope="module", autouse=True)
def built():
    fp4_build.build()


def _call(name, base, **kw):
    a = dict(base)
    assert set(kw) <= set(a), set(kw) - set(a)
    a.update(kw)
    return getattr(fp4.lib(), name)(*a.values())


SORT = dict(ids=16, id_bytes=4, tokens=8, topk=2, E=4, off=16, row=16, srow=16, ws=None, wsb=0, stream=None)


@pytest.mark.parametrize("kw", [
    dict(ids=None), dict(off=None), dict(row=None), dict(id_bytes=2), dict(id_bytes=0), dict(tokens=0), dict(tokens=-1),
    dict(topk=0), dict(E=0), dict(E=1025), dict(ids=18), dict(ids=20, id_bytes=8), dict(off=2), dict(row=1), dict(srow=6),
    dict(tokens=20000), dict(tokens=20000, ws=16, wsb=64), dict(tokens=20000, ws=18, wsb=1 << 20)])
def test_sort_refuses(kw):
    assert _call("fp4_moe_sort", SORT, **kw) == fp4.ERR_INVALID_ARG


def test_sort_sizes():
    assert _call("fp4_moe_sort", SORT, tokens=1 << 30) == fp4.ERR_UNSUPPORTED
    assert _call("fp4_moe_sort", SORT, topk=1025) == fp4.ERR_UNSUPPORTED
    assert fp4.fp4_moe_sort_workspace_size(8192, 4, 32) == 0
    assert 0 < fp4.fp4_moe_sort_workspace_size(8193, 4, 32) <= 128 * 32 * 4
    assert fp4.fp4_moe_sort_workspace_size(1 << 27, 8, 1024) == 128 * 1024 * 4
    assert fp4.fp4_moe_sort_workspace_size(0, 4, 32) == 0


DISP = dict(x=16, tokens=8, cols=64, dt=fp4.F32, topk=2, row=16, y=32, out=fp4.BF16, stream=None)


@pytest.mark.parametrize("kw", [dict(x=None), dict(y=None), dict(row=None), dict(tokens=0), dict(cols=0), dict(topk=-1),
                                dict(dt=5), dict(out=2), dict(x=8), dict(y=24), dict(row=2), dict(y=16)])
def test_dispatch_refuses(kw):
    assert _call("fp4_moe_dispatch", DISP, **kw) == fp4.ERR_INVALID_ARG


def test_dispatch_sizes():
    assert _call("fp4_moe_dispatch", DISP, cols=(1 << 24) + 1) == fp4.ERR_UNSUPPORTED
    assert _call("fp4_moe_dispatch", DISP, tokens=(1 << 29) + 1) == fp4.ERR_UNSUPPORTED


CODES = dict(x=48, tokens=8, cols=64, dt=fp4.F32, topk=2, row=16, srow=16, E=4, off=16, fmt=fp4.NVFP4, codes=16, scales=32,
             g=16, stream=None)


@pytest.mark.parametrize("kw", [
    dict(x=None), dict(row=None), dict(srow=None), dict(off=None), dict(codes=None), dict(scales=None), dict(g=None),
    dict(E=0), dict(E=1025), dict(fmt=fp4.MXFP8), dict(fmt=7), dict(cols=48), dict(tokens=0), dict(dt=9), dict(x=8),
    dict(codes=8), dict(scales=8), dict(g=2), dict(srow=2), dict(off=1), dict(codes=48)])
def test_dispatch_codes_refuses(kw):
    assert _call("fp4_moe_dispatch_codes", CODES, **kw) == fp4.ERR_INVALID_ARG


I8D = dict(x=32, tokens=8, cols=64, dt=fp4.F32, topk=2, row=16, codes=16, scales=16, stream=None)


@pytest.mark.parametrize("kw", [dict(x=None), dict(row=None), dict(codes=None), dict(scales=None), dict(cols=40),
                                dict(tokens=0), dict(dt=3), dict(x=8), dict(codes=24), dict(scales=2), dict(codes=32)])
def test_dispatch_i8_refuses(kw):
    assert _call("fp4_moe_dispatch_i8", I8D, **kw) == fp4.ERR_INVALID_ARG


COMB = dict(y=16, dt=fp4.BF16, row=16, w=16, tokens=8, topk=2, cols=64, res=32, rdt=fp4.BF16, out=48, odt=fp4.BF16, stream=None)


@pytest.mark.parametrize("kw", [
    dict(y=None), dict(row=None), dict(out=None), dict(tokens=0), dict(cols=0), dict(topk=0), dict(dt=2), dict(odt=3),
    dict(rdt=4), dict(y=8), dict(res=40), dict(out=56), dict(w=2), dict(out=16), dict(out=32, odt=fp4.F32)])
def test_combine_refuses(kw):
    assert _call("fp4_moe_combine", COMB, **kw) == fp4.ERR_INVALID_ARG


GRAD = dict(dout=16, y=32, dt=fp4.BF16, row=16, w=16, tokens=8, topk=2, cols=64, dy=48, odt=fp4.BF16, dw=16, stream=None)


@pytest.mark.parametrize("kw", [
    dict(dout=None), dict(y=None), dict(row=None), dict(dy=None, dw=None), dict(tokens=0), dict(cols=-4), dict(topk=0),
    dict(dt=2), dict(odt=3), dict(dout=8), dict(y=40), dict(dy=56), dict(w=1), dict(dw=2), dict(dy=16),
    dict(dy=32, odt=fp4.F32)])
def test_combine_backward_refuses(kw):
    assert _call("fp4_moe_combine_backward", GRAD, **kw) == fp4.ERR_INVALID_ARG


Q8 = dict(x=32, rows=8, cols=64, dt=fp4.F32, codes=16, scales=16, valid=16, stream=None)


@pytest.mark.parametrize("kw", [dict(x=None), dict(codes=None), dict(scales=None), dict(rows=0), dict(cols=0), dict(cols=24),
                                dict(dt=2), dict(x=8), dict(codes=8), dict(scales=2), dict(valid=2), dict(codes=32)])
def test_quantize_i8_refuses(kw):
    assert _call("fp4_quantize_i8", Q8, **kw) == fp4.ERR_INVALID_ARG


def test_quantize_i8_sizes():
    assert _call("fp4_quantize_i8", Q8, rows=1 << 31) == fp4.ERR_UNSUPPORTED


G8 = dict(A=16, sA=16, B=32, sB=16, M=512, N=4096, K=64, bias=16, act=fp4.ACT_SILU, D=48, out=fp4.BF16, ws=None, wsb=0,
          flags=0, stream=None)


@pytest.mark.parametrize("kw", [
    dict(A=None), dict(sA=None), dict(B=None), dict(sB=None), dict(D=None), dict(M=0), dict(N=0), dict(K=0), dict(K=40),
    dict(act=5), dict(act=-1), dict(out=2), dict(A=8), dict(B=24), dict(D=56), dict(sA=2), dict(sB=1), dict(bias=3),
    dict(flags=2), dict(M=16, K=4096), dict(M=16, K=4096, ws=16, wsb=4096), dict(M=16, K=4096, ws=8, wsb=1 << 30)])
def test_gemm_i8_refuses(kw):
    assert _call("fp4_gemm_i8", G8, **kw) == fp4.ERR_INVALID_ARG


def test_gemm_i8_sizes():
    for kw in (dict(M=1 << 31), dict(N=1 << 31), dict(K=131072)):
        assert _call("fp4_gemm_i8", G8, **kw) == fp4.ERR_UNSUPPORTED
    assert fp4.fp4_gemm_i8_workspace_size(8192, 8192, 8192) == 0
    assert fp4.fp4_gemm_i8_workspace_size(16, 8192, 8192) >= 16 * 128 * 4
    assert fp4.fp4_gemm_i8_workspace_size(0, 8192, 8192) == 0
    assert fp4.fp4_gemm_i8_grouped_workspace_size(0, 64, 128, 128) == 0
    assert fp4.fp4_gemm_i8_grouped_workspace_size(32, 64, 5760, 2880) > 0


GG8 = dict(E=4, off=16, A=16, sA=16, B=32, sB=16, rows=4096, N=4096, K=64, bias=16, act=fp4.ACT_NONE, D=48, out=fp4.BF16,
           ws=None, wsb=0, stream=None)


@pytest.mark.parametrize("kw", [
    dict(E=0), dict(E=1025), dict(off=None), dict(off=2), dict(A=None), dict(D=None), dict(rows=0), dict(K=8), dict(act=9),
    dict(out=4), dict(rows=8, K=2880), dict(rows=8, K=2880, ws=16, wsb=100)])
def test_gemm_i8_grouped_refuses(kw):
    assert _call("fp4_gemm_i8_grouped", GG8, **kw) == fp4.ERR_INVALID_ARG


def test_gemm_i8_grouped_sizes():
    assert _call("fp4_gemm_i8_grouped", GG8, E=1024, N=1 << 21) == fp4.ERR_UNSUPPORTED


def test_conveniences_check_their_operands():
    ids = torch.zeros(4, 2, dtype=torch.int64)
    with pytest.raises(ValueError):      # not on a GPU
        fp4.moe_sort(ids, 4)
    with pytest.raises(ValueError):
        fp4.moe_sort(ids[0], 4)
    with pytest.raises(TypeError):
        fp4.moe_sort(ids.float(), 4)
    with pytest.raises(ValueError):      # a strided operand
        fp4.moe_sort(torch.zeros(4, 4, dtype=torch.int64)[:, ::2], 4)
    i32 = torch.zeros(4, 2, dtype=torch.int32)
    r = fp4.Routing(torch.zeros(5, dtype=torch.int32), i32, i32, 4)
    assert (r.tokens, r.topk) == (4, 2)
    x = torch.zeros(4, 64)
    with pytest.raises(ValueError):
        fp4.moe_dispatch(x, r)
    with pytest.raises(ValueError):      # another number of tokens
        fp4.moe_dispatch(x[:3], r)
    with pytest.raises(ValueError):      # rows of slots, not of tokens
        fp4.moe_combine(x, r)
    with pytest.raises(TypeError):
        fp4.moe_combine(torch.zeros(8, 64), r, torch.zeros(4, 2, dtype=torch.bfloat16))
    with pytest.raises(TypeError):
        fp4.moe_combine_backward(x.bfloat16(), torch.zeros(8, 64), r)
    with pytest.raises(ValueError):
        fp4.quantize_i8(x[0])
    q = fp4.Int8Rows(torch.zeros(4, 64, dtype=torch.int8), torch.zeros(4))
    with pytest.raises(ValueError):
        fp4.gemm_i8(q, fp4.Int8Rows(torch.zeros(4, 32, dtype=torch.int8), torch.zeros(4)))
    with pytest.raises(ValueError):      # experts' weights without offsets
        fp4.gemm_i8(q, fp4.Int8Rows(torch.zeros(2, 4, 64, dtype=torch.int8), torch.zeros(2, 4)))
    with pytest.raises(TypeError):
        fp4.gemm_i8(q, fp4.Int8Rows(torch.zeros(4, 64), torch.zeros(4)))
