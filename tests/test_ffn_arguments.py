"""Refusals of the feed-forward block's entry points on the host, before anything is enqueued
(no GPU needed), and the conveniences' checks of their operands."""
import pytest
import torch

import block_scaled_fp4_04_b200 as fp4
from block_scaled_fp4_04_b200 import build as fp4_build

INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module", autouse=True)
def built():
    fp4_build.build()


def _call(name, base, **kw):
    a = dict(base)
    assert set(kw) <= set(a), set(kw) - set(a)
    a.update(kw)
    return getattr(fp4.lib(), name)(*a.values())


LN = dict(x=16, rows=4, cols=64, dt=fp4.F32, w=16, b=16, eps=1e-5, y=32, out=fp4.F32, mean=16, rstd=16, fmt=fp4.NVFP4,
          codes=None, scales=None, g=None, amax=None, stream=None)


@pytest.mark.parametrize("kw", [
    dict(x=None), dict(y=None), dict(rows=0), dict(cols=0), dict(rows=-1), dict(x=8), dict(y=24), dict(dt=7), dict(out=2),
    dict(eps=-1.0), dict(eps=NAN), dict(eps=INF), dict(w=2), dict(b=6), dict(mean=1), dict(rstd=2), dict(amax=2),
    dict(codes=16, g=16), dict(codes=16, scales=16), dict(codes=16, scales=16, g=16, cols=48),
    dict(codes=8, scales=16, g=16), dict(codes=16, scales=24, g=16), dict(codes=16, scales=16, g=16, fmt=fp4.MXFP8),
    dict(codes=16, scales=16, g=16, w=20)])
def test_layernorm_refuses(kw):
    assert _call("fp4_layernorm", LN, **kw) == fp4.ERR_INVALID_ARG



def test_layernorm_in_place_needs_one_type():
    assert _call("fp4_layernorm", LN, y=16, out=fp4.BF16) == fp4.ERR_INVALID_ARG
    assert "x's place" in fp4.fp4_last_error()


LNB = dict(dy=16, x=32, rows=4, cols=64, dt=fp4.F32, w=16, mean=16, rstd=16, dres=48, dx=64, out=fp4.F32, dw=16, db=16,
           ws=16, wsb=1 << 20, stream=None)


@pytest.mark.parametrize("kw", [
    dict(dy=None), dict(x=None), dict(mean=None), dict(rstd=None), dict(dx=None), dict(rows=0), dict(cols=0), dict(dy=8),
    dict(dx=72), dict(dres=8), dict(dt=3), dict(out=9), dict(dx=32), dict(dx=16, out=fp4.BF16), dict(dx=48, out=fp4.BF16),
    dict(ws=None), dict(ws=8), dict(wsb=16), dict(dw=2), dict(db=1)])
def test_layernorm_backward_refuses(kw):
    assert _call("fp4_layernorm_backward", LNB, **kw) == fp4.ERR_INVALID_ARG


def test_layernorm_sizes_beyond_the_offsets():
    assert _call("fp4_layernorm", LN, rows=1 << 31) == fp4.ERR_UNSUPPORTED
    assert _call("fp4_layernorm", LN, cols=(1 << 30) + 1) == fp4.ERR_UNSUPPORTED
    assert _call("fp4_layernorm_backward", LNB, rows=1 << 31) == fp4.ERR_UNSUPPORTED


AG = dict(dh=16, g=32, u=48, rows=4, cols=64, dt=fp4.F32, act=fp4.ACT_SILU, dz=64, out=fp4.F32, db=16, fmt=fp4.NVFP4,
          codes=None, scales=None, gl=None, amax=None, ws=16, wsb=1 << 20, stream=None)


@pytest.mark.parametrize("kw", [
    dict(dh=None), dict(g=None), dict(dz=None), dict(rows=0), dict(cols=0), dict(act=5), dict(act=-1), dict(dt=4),
    dict(out=5), dict(dh=8), dict(g=8), dict(u=8), dict(dz=8), dict(dz=16), dict(dz=32), dict(dz=48), dict(ws=None),
    dict(wsb=8), dict(ws=24), dict(codes=16, gl=16), dict(codes=16, scales=16), dict(codes=16, scales=16, gl=16, cols=40),
    dict(amax=2), dict(db=2)])
def test_act_backward_refuses(kw):
    assert _call("fp4_act_backward", AG, **kw) == fp4.ERR_INVALID_ARG


GT = dict(fmt=fp4.NVFP4, A=16, sA=16, gA=16, Wg=16, sWg=16, gWg=16, Wu=16, sWu=16, gWu=16, M=128, F=256, K=256, bg=16,
          bu=16, act=fp4.ACT_SILU, H=16, out=fp4.BF16, G=32, U=48, codes=None, scales=None, gH=None, amax=None, ws=None,
          wsb=0, flags=0, stream=None)


@pytest.mark.parametrize("kw", [
    dict(fmt=fp4.MXFP8), dict(fmt=9), dict(A=None), dict(sA=None), dict(Wg=None), dict(sWg=None), dict(Wu=None),
    dict(sWu=None), dict(H=None), dict(G=None), dict(U=None), dict(G=16), dict(U=16), dict(G=48), dict(M=0), dict(F=0),
    dict(K=0), dict(K=48), dict(act=7), dict(out=3), dict(A=8), dict(Wg=8), dict(Wu=24), dict(sWu=8), dict(H=8), dict(G=8),
    dict(bg=2), dict(bu=3), dict(flags=2), dict(codes=16, gH=16), dict(codes=16, scales=16),
    dict(codes=16, scales=16, gH=16, F=48), dict(codes=24, scales=16, gH=16), dict(amax=2),
    dict(M=16, F=512, K=2048),                              # needs a workspace
    dict(M=16, F=512, K=2048, ws=16, wsb=1024),             # too small
    dict(M=16, F=512, K=2048, ws=8, wsb=1 << 30)])          # misaligned
def test_gemm_gated_refuses(kw):
    assert _call("fp4_gemm_gated", GT, **kw) == fp4.ERR_INVALID_ARG


def test_gemm_gated_sizes():
    assert _call("fp4_gemm_gated", GT, M=1 << 31) == fp4.ERR_UNSUPPORTED
    assert fp4.fp4_gemm_gated_workspace_size(8192, 8192, 8192, fp4.NVFP4, False) == 0
    assert fp4.fp4_gemm_gated_workspace_size(16, 4096, 8192, fp4.NVFP4, False) >= 2 * 16 * 4096 * 4
    assert fp4.fp4_gemm_gated_workspace_size(16, 4096, 8192, fp4.MXFP4, False) >= 2 * 16 * 4096 * 4
    assert fp4.fp4_gemm_gated_workspace_size(0, 4096, 8192, fp4.NVFP4, False) == 0
    assert fp4.fp4_gemm_gated_bf16a_workspace_size(16, 4096, 8192) > fp4.fp4_quantize_workspace_size()


GX = dict(X=16, Wg=16, sWg=16, gWg=16, Wu=16, sWu=16, gWu=16, M=16, F=256, K=256, bg=16, bu=16, act=fp4.ACT_SILU, H=16,
          out=fp4.BF16, G=32, U=48, Xc=16, Xs=16, gX=16, ws=16, wsb=1 << 30, flags=0, stream=None)


@pytest.mark.parametrize("kw", [
    dict(X=None), dict(Wg=None), dict(sWg=None), dict(Wu=None), dict(sWu=None), dict(H=None), dict(Xc=None), dict(Xs=None),
    dict(gX=None), dict(ws=None), dict(wsb=64), dict(M=0), dict(F=0), dict(K=40), dict(act=5), dict(out=8), dict(G=None),
    dict(U=16), dict(X=8), dict(Xc=8), dict(ws=8), dict(flags=4), dict(bg=2)])
def test_gemm_gated_bf16a_refuses(kw):
    assert _call("fp4_gemm_gated_bf16a", GX, **kw) == fp4.ERR_INVALID_ARG


GG = dict(fmt=fp4.MXFP4, E=4, off=16, A=16, sA=16, gA=None, Wg=16, sWg=16, gWg=None, Wu=16, sWu=16, gWu=None, rows=64,
          F=100, K=64, bg=None, bu=None, act=fp4.ACT_SILU, H=16, out=fp4.BF16, G=None, U=None, stream=None)


@pytest.mark.parametrize("kw", [dict(E=0), dict(E=1025), dict(off=None), dict(rows=0), dict(F=0), dict(K=33), dict(H=None),
                                dict(G=32), dict(Wu=None), dict(gWg=2), dict(fmt=4)])
def test_gemm_gated_grouped_refuses(kw):
    assert _call("fp4_gemm_gated_grouped", GG, **kw) == fp4.ERR_INVALID_ARG


EX = dict(fmt=fp4.NVFP4, A=16, sA=16, gA=16, B=16, sB=16, gB=16, M=128, N=256, K=256, bias=16, act=fp4.ACT_GELU, res=32,
          rdt=fp4.BF16, D=48, out=fp4.BF16, pre=64, codes=None, scales=None, gD=None, amax=None, ws=None, wsb=0, flags=0,
          stream=None)


@pytest.mark.parametrize("kw", [
    dict(A=None), dict(B=None), dict(D=None), dict(act=5), dict(rdt=6), dict(res=8), dict(pre=8), dict(pre=48),
    dict(pre=32), dict(D=32, out=fp4.F32), dict(flags=2), dict(K=40), dict(M=0), dict(out=4), dict(bias=2),
    dict(codes=16), dict(codes=16, scales=16, gD=16, N=272), dict(amax=2)])
def test_gemm_epilogue_ex_refuses(kw):
    assert _call("fp4_gemm_epilogue_ex", EX, **kw) == fp4.ERR_INVALID_ARG


def test_plain_epilogue_keeps_its_activations():
    L = fp4.lib()
    assert L.fp4_gemm_epilogue(fp4.NVFP4, 16, 16, 16, 16, 16, 16, 128, 128, 256, None, fp4.ACT_SILU, 16, fp4.BF16, None,
                               None, None, None, None, 0, None) == fp4.ERR_INVALID_ARG


def test_conveniences_check_their_operands():
    x = torch.zeros(4, 64)
    with pytest.raises(ValueError):      # not on a GPU
        fp4.layernorm(x)
    with pytest.raises(ValueError):
        fp4.layernorm(x[0])
    with pytest.raises(TypeError):
        fp4.layernorm(x, torch.zeros(64, dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        fp4.layernorm(x, torch.zeros(63))
    with pytest.raises(ValueError):      # a strided operand
        fp4.layernorm(torch.zeros(4, 128)[:, ::2])
    with pytest.raises(TypeError):
        fp4.act_backward(x, x.bfloat16())
    with pytest.raises(ValueError):
        fp4.act_backward(x, x, x[:2])
    with pytest.raises(ValueError):
        fp4.layernorm_backward(x, x, None, torch.zeros(5), torch.zeros(4))
    q = fp4.Quantized(torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(512, dtype=torch.uint8), torch.ones(1), 4, 64, 0)
    w = fp4.Quantized(torch.zeros(8, 16, dtype=torch.uint8), torch.zeros(512, dtype=torch.uint8), torch.ones(1), 8, 32, 0)
    with pytest.raises(ValueError):
        fp4.gemm_gated(q, w, w)
    with pytest.raises(ValueError):
        fp4.gemm_epilogue(q, w)
