"""Sizes whose products pass 64 bits, or a kernel's 32-bit offsets: refused on the host, no GPU."""
import ctypes

import pytest

import fp8_blockwise_scaled_b200 as fb
from fp8_blockwise_scaled_b200 import _lib

P = ctypes.c_void_p
A = P(0x10000)            # never dereferenced: every case below fails validation first
N0 = P(0)
LAST = (1 << 63) - 1


def test_padded_rows():
    f = fb.fp8blk_grouped_padded_rows
    assert f(LAST, 1) == -1 and f(LAST - 127 * 1024 + 1, fb.MAX_GROUPS) == -1
    assert f(1 << 40, fb.MAX_GROUPS) == (1 << 40) + 127 * 1024 // 128 * 128


def test_workspaces_and_scales():
    big = 1 << 33
    assert fb.fp8blk_linear_grouped_workspace_bytes(1, big, big) == -1
    assert fb.fp8blk_linear_grouped_workspace_bytes(1, (1 << 31) - 1, 128) == ((1 << 31) - 1) * 132
    for fmt in (fb.MXFP4, fb.NVFP4):
        assert fb.fp8blk_mx4_scale_bytes(fmt, LAST, 64) == -1 and fb.fp8blk_mx4_scale_bytes(fmt, 64, LAST) == -1
        assert fb.fp8blk_linear_mx4_workspace_bytes(fmt, big, 1 << 34) == -1
        assert fb.fp8blk_mx4_scale_bytes(fmt, (1 << 31) - 1, 128) == (1 << 24) * (1 if fmt == fb.MXFP4 else 2) * 512


@pytest.mark.parametrize("rows,cols", [(LAST, 128), (1 << 62, 128), (8, 1 << 30), (8, 1 << 62), (1, (1 << 29) + 128),
                                       (1 << 18, 1 << 59)])
@pytest.mark.parametrize("groups", [1, 1024])
def test_ragged_quantiser(rows, cols, groups):
    assert _lib.lib.fp8blk_quantize_act_1x128_grouped(A, rows, cols, cols, 1, A, groups, A, A, N0, N0, N0) == 2
    assert _lib.lib.fp8blk_linear_grouped(0, groups, A, rows, 128, cols, A, cols, A, A, A, LAST, A, 128, N0) == 2


@pytest.mark.parametrize("layout,m,n,k", [(0, 1 << 17, 1 << 60, 128), (0, 5, 128, 1 << 60), (1, 5, 128, 1 << 61),
                                          (0, LAST, 128, 128), (2, 1 << 60, 128, 128), (2, 1 << 60, 1 << 60, 128),
                                          (2, 128, 128, 1 << 62)])
@pytest.mark.parametrize("groups", [16, 1024])
def test_grouped_products(layout, m, n, k, groups):
    assert _lib.lib.fp8blk_gemm_grouped(layout, groups, A, m, n, k, A, A, A, A, A, n, N0) == 2
