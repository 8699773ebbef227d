"""Workspaces that the entry points refuse on the host, before anything is enqueued, and the buffers
that a Workspace hands out (no GPU needed)."""
import pytest
import torch

import block_scaled_fp4_04_b200 as fp4
from block_scaled_fp4_04_b200 import build as fp4_build

ENOUGH = 1 << 30
SPLIT = [                     # m, n, k, fmt of products that need a workspace with 16-byte accesses
    (16, 512, 2048, fp4.NVFP4),   # decode kernel
    (16, 512, 2048, fp4.MXFP4),   # operands swapped
    (48, 640, 2048, fp4.NVFP4),   # the same, 64 columns
    (256, 256, 8192, fp4.NVFP4),  # in place
    (130, 260, 8192, fp4.MXFP4),
]


@pytest.fixture(scope="module", autouse=True)
def built():
    fp4_build.build()


@pytest.mark.parametrize("m,n,k,fmt", SPLIT)
@pytest.mark.parametrize("ws", [2, 4, 8, 24])
def test_products_refuse_a_misaligned_workspace(m, n, k, fmt, ws):
    L, head = fp4.lib(), (fmt, 16, 16, 16, 16, 16, 16, m, n, k)
    assert fp4.fp4_gemm_workspace_size(m, n, k, fmt) > 0
    assert L.fp4_gemm(*head, 16, fp4.F32, ws, ENOUGH, None) == fp4.ERR_INVALID_ARG
    assert L.fp4_gemm_ex(*head, 16, fp4.F32, ws, ENOUGH, 0, None) == fp4.ERR_INVALID_ARG
    assert L.fp4_gemm_epilogue(*head, None, fp4.ACT_RELU, 16, fp4.F32, None, None, None, None, ws, ENOUGH,
                               None) == fp4.ERR_INVALID_ARG
    assert "alignment" in fp4.fp4_last_error()
    for res, pre in ((None, None), (32, None), (None, 64)):
        assert L.fp4_gemm_epilogue_ex(*head, None, fp4.ACT_RELU, res, fp4.F32, 48, fp4.F32, pre, None, None, None, None, ws,
                                      ENOUGH, 0, None) == fp4.ERR_INVALID_ARG
        assert "alignment" in fp4.fp4_last_error()


@pytest.mark.parametrize("m,n,k", [(1, 512, 2048), (7, 640, 4096), (130, 257, 8192)])
def test_odd_products_refuse_less_than_their_words(m, n, k):
    """Partial sums that move one at a time need 4 bytes; the long epilogue pads them to 16."""
    L, head = fp4.lib(), (fp4.NVFP4, 16, 16, 16, 16, 16, 16, m, n, k)
    for ws in (1, 2, 18):
        assert L.fp4_gemm(*head, 16, fp4.F32, ws, ENOUGH, None) == fp4.ERR_INVALID_ARG
    for ws in (2, 4, 8):
        assert L.fp4_gemm_epilogue_ex(*head, None, fp4.ACT_SILU, None, fp4.F32, 48, fp4.F32, None, None, None, None, None, ws,
                                      ENOUGH, 0, None) == fp4.ERR_INVALID_ARG


def test_a_workspace_does_not_grow_into_a_capture(monkeypatch):
    """What a capture allocates is zero-filled when the graph replays, not before: calls outside the
    graph must not be given it."""
    ws = fp4.Workspace("cpu")
    first = ws.get(5000)
    monkeypatch.setattr(fp4, "_capturing", lambda device: True)
    assert ws.get(4000).data_ptr() == first.data_ptr()  # large enough: the one buffer
    inside = ws.get(9000)
    assert inside.numel() >= 9000 and not inside.any()
    assert ws.get(9000).data_ptr() != inside.data_ptr()
    monkeypatch.undo()
    assert ws.get(5000).data_ptr() == first.data_ptr()
    after = ws.get(9000)
    assert after.data_ptr() != inside.data_ptr() and ws.get(9000).data_ptr() == after.data_ptr()


def test_a_workspace_keeps_the_buffers_it_has_outgrown():
    ws = fp4.Workspace("cpu")
    held = [ws.get(n).data_ptr() for n in (5000, 50000, 500000)]
    assert len(set(held)) == 3 and [b.data_ptr() for b in ws._outgrown] == held[:2]


def test_what_a_workspace_keeps_stays_below_what_it_uses():
    ws = fp4.Workspace("cpu")
    for n in range(5000, 200000, 1000):
        assert ws.get(n).numel() >= n
    assert sum(b.numel() for b in ws._outgrown) < ws.buf.numel() < 2 * 200000


SLOTS = 512 * 128  # the decode kernel's workspace ends in these


def test_a_k_too_long_for_the_decode_kernel_takes_the_others():
    """A CTA holds one segment of at most 2048 elements of K; a grid has one CTA per SM (148 where
    there is no GPU to ask)."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count if torch.cuda.is_available() else 148
    last, n = 2048 * sms, 64
    for m in (1, 16):
        for size in (fp4.fp4_gemm_workspace_size, lambda *a: fp4.fp4_gemm_epilogue_workspace_size(*a, False),
                     lambda *a: fp4.fp4_gemm_gated_workspace_size(*a, False)):
            assert size(m, n, last, fp4.NVFP4) > SLOTS
            assert 0 < size(m, n, last + 32, fp4.NVFP4) < SLOTS
    # whatever the epilogue's plan is, one size serves it with and without its extras
    for m, n in ((1, 64), (16, 28672), (32, 40000)):
        assert (fp4.fp4_gemm_epilogue_workspace_size(m, n, last + 32, fp4.NVFP4, False)
                >= fp4.fp4_gemm_workspace_size(m, n, last + 32, fp4.NVFP4))
