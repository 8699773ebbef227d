"""Global scales, maxima and offsets that do not stand at 4 bytes are refused on the host, before
anything is enqueued (no GPU needed)."""
import pytest

import block_scaled_fp4_04_b200 as fp4
from block_scaled_fp4_04_b200 import build as fp4_build

NV, F32, BIG = fp4.NVFP4, fp4.F32, 1 << 30


@pytest.fixture(scope="module", autouse=True)
def built():
    fp4_build.build()


# calls with `bad` where a scalar's address goes
CALLS = {
    "amax out": lambda L, bad: L.fp4_amax(16, 64, F32, bad, 16, BIG, None),
    "quantize global out": lambda L, bad: L.fp4_quantize(16, 4, 64, F32, NV, 16, 16, 16, bad, None, None, None, 16, BIG, None),
    "quantize global in": lambda L, bad: L.fp4_quantize(16, 4, 64, F32, NV, 16, 16, 16, 16, None, None, bad, 16, BIG, None),
    "quantize offsets": lambda L, bad: L.fp4_quantize_grouped(16, 4, 64, F32, NV, 2, bad, 16, 16, 16, None, 16, BIG, None),
    "global scale in": lambda L, bad: L.fp4_global_scale(bad, 16, None),
    "global scale out": lambda L, bad: L.fp4_global_scale(16, bad, None),
    "dequantize global": lambda L, bad: L.fp4_dequantize(16, 16, bad, 4, 64, NV, 16, None),
    "gemm gA": lambda L, bad: L.fp4_gemm(NV, 16, 16, bad, 16, 16, 16, 128, 128, 64, 16, F32, None, 0, None),
    "gemm gB": lambda L, bad: L.fp4_gemm(NV, 16, 16, 16, 16, 16, bad, 128, 128, 64, 16, F32, None, 0, None),
    "grouped offsets": lambda L, bad: L.fp4_gemm_grouped(NV, 2, bad, 16, 16, 16, 16, 16, 16, 128, 128, 64, 16, F32, None, 0,
                                                         None),
    "epilogue gD": lambda L, bad: L.fp4_gemm_epilogue(NV, 16, 16, 16, 16, 16, 16, 128, 128, 64, None, 0, None, F32, 16, 16,
                                                      bad, None, None, 0, None),
    "bf16a gB": lambda L, bad: L.fp4_gemm_bf16a(16, 16, 16, bad, 16, 128, 64, 16, F32, 16, 16, 16, 16, BIG, 0, None),
    "bf16a gX": lambda L, bad: L.fp4_gemm_bf16a(16, 16, 16, 16, 16, 128, 64, 16, F32, 16, 16, bad, 16, BIG, 0, None),
    "gated gA": lambda L, bad: L.fp4_gemm_gated(NV, 16, 16, bad, 16, 16, 16, 16, 16, 16, 128, 128, 64, None, None, 2, 16, F32,
                                                None, None, None, None, None, None, None, 0, 0, None),
    "gated gWg": lambda L, bad: L.fp4_gemm_gated(NV, 16, 16, 16, 16, 16, bad, 16, 16, 16, 128, 128, 64, None, None, 2, 16, F32,
                                                 None, None, None, None, None, None, None, 0, 0, None),
    "gated gWu": lambda L, bad: L.fp4_gemm_gated(NV, 16, 16, 16, 16, 16, 16, 16, 16, bad, 128, 128, 64, None, None, 2, 16, F32,
                                                 None, None, None, None, None, None, None, 0, 0, None),
    "gated gH": lambda L, bad: L.fp4_gemm_gated(NV, 16, 16, 16, 16, 16, 16, 16, 16, 16, 128, 128, 64, None, None, 2, None, F32,
                                                None, None, 16, 16, bad, None, None, 0, 0, None),
    "gated bf16a gX": lambda L, bad: L.fp4_gemm_gated_bf16a(16, 16, 16, 16, 16, 16, 16, 16, 128, 64, None, None, 2, 16, F32,
                                                            None, None, 16, 16, bad, 16, BIG, 0, None),
    "gated bf16a gWu": lambda L, bad: L.fp4_gemm_gated_bf16a(16, 16, 16, 16, 16, 16, bad, 16, 128, 64, None, None, 2, 16, F32,
                                                             None, None, 16, 16, 16, 16, BIG, 0, None),
    "gated offsets": lambda L, bad: L.fp4_gemm_gated_grouped(NV, 2, bad, 16, 16, 16, 16, 16, 16, 16, 16, 16, 128, 128, 64, None,
                                                             None, 2, 16, F32, None, None, None),
    "norm global": lambda L, bad: L.fp4_layernorm(16, 4, 64, F32, None, None, 1e-5, None, F32, None, None, NV, 16, 16, bad,
                                                  None, None),
    "act backward global": lambda L, bad: L.fp4_act_backward(16, 16, None, 4, 64, F32, 2, None, F32, None, NV, 16, 16, bad,
                                                             None, None, 0, None),
}


@pytest.mark.parametrize("name", CALLS)
@pytest.mark.parametrize("bad", [1, 18, 35])
def test_refused(name, bad):
    assert CALLS[name](fp4.lib(), bad) == fp4.ERR_INVALID_ARG
    assert "alignment" in fp4.fp4_last_error()
