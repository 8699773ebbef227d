"""Sizes that the kernels' 32-bit counts do not hold are refused on the host, before anything is
enqueued (no GPU needed)."""
import pytest

import block_scaled_fp4_04_b200 as fp4
from block_scaled_fp4_04_b200 import build as fp4_build

NV, MX, F32, BIG = fp4.NVFP4, fp4.MXFP4, fp4.F32, 1 << 62
FAR = 1 << 31


@pytest.fixture(scope="module", autouse=True)
def built():
    fp4_build.build()


@pytest.mark.parametrize("m,n,k", [(FAR, 128, 128), (128, FAR, 128), (128, 128, FAR), (1, 1, 2 * FAR),
                                   (FAR - 128, 128, 128)])
def test_products(m, n, k):
    L, head = fp4.lib(), (NV, 16, 16, 16, 16, 16, 16, m, n, k)
    assert L.fp4_gemm(*head, 16, F32, 16, BIG, None) == fp4.ERR_UNSUPPORTED
    assert L.fp4_gemm_ex(*head, 16, F32, 16, BIG, 0, None) == fp4.ERR_UNSUPPORTED
    assert L.fp4_gemm_epilogue(*head, None, 0, 16, F32, None, None, None, None, 16, BIG, None) == fp4.ERR_UNSUPPORTED
    assert L.fp4_gemm_epilogue_ex(*head, None, 2, 32, F32, 48, F32, 64, None, None, None, None, 16, BIG, 0,
                                  None) == fp4.ERR_UNSUPPORTED
    assert L.fp4_gemm_mixed(MX, 32, 16, MX, 32, 16, m, n, k, 16, F32, None) == fp4.ERR_UNSUPPORTED
    assert L.fp4_gemm_bf16a(16, 16, 16, 16, m, n, k, 16, F32, 16, 16, 16, 16, BIG, 0, None) == fp4.ERR_UNSUPPORTED
    assert L.fp4_gemm_gated(NV, 16, 16, 16, 16, 16, 16, 16, 16, 16, m, n, k, None, None, 2, 16, F32, None, None, None, None,
                            None, None, 16, BIG, 0, None) == fp4.ERR_UNSUPPORTED
    assert L.fp4_gemm_gated_bf16a(16, 16, 16, 16, 16, 16, 16, m, n, k, None, None, 2, 16, F32, None, None, 16, 16, 16, 16, BIG,
                                  0, None) == fp4.ERR_UNSUPPORTED


def test_rows_of_all_experts():
    L = fp4.lib()
    n = 1 << 22  # 1024 experts of as many rows
    assert L.fp4_gemm_grouped(NV, 1024, 16, 16, 16, 16, 16, 16, 16, 128, n, 64, 16, F32, None, 0, None) == fp4.ERR_UNSUPPORTED
    assert L.fp4_gemm_gated_grouped(NV, 1024, 16, 16, 16, 16, 16, 16, 16, 16, 16, 16, 128, n, 64, None, None, 2, 16, F32, None,
                                    None, None) == fp4.ERR_UNSUPPORTED
