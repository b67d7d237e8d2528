"""The 4-bit reference against the formats' definitions, and the entry points' refusals: host logic, no GPU."""
import ctypes

import numpy as np
import pytest
import torch

import fp8_blockwise_scaled_b200 as fb
from fp8_blockwise_scaled_b200 import _lib
from tests import mx4_reference as ref

P = ctypes.c_void_p
A = P(0x10000)            # never dereferenced: every case below fails validation first
M8 = P(0x10008)
ODD = P(0x10002)
N0 = P(0)


def test_reference_rounds_to_the_nearest_code_with_ties_to_even():
    v = np.array([0.0, -0.0, 0.25, 0.26, 0.75, 1.25, 1.75, 2.5, 2.6, 3.5, 5.0, 5.1, 7.0, -0.75, -6.5])
    assert ref.GRID[ref.round_e2m1(v) & 7].tolist() == [0, 0, 0, 0.5, 1, 1, 2, 2, 3, 4, 4, 6, 6, 1, 6]
    assert (ref.round_e2m1(np.array([-0.75, -0.0, 0.0])) >> 3).tolist() == [1, 1, 0]
    x = np.abs(np.random.default_rng(0).standard_normal(4000).astype(np.float32)) * 300
    want = torch.from_numpy(np.minimum(x, 448)).to(torch.float8_e4m3fn).float().numpy()
    assert np.array_equal(ref.e4m3_values()[ref.round_e4m3(x.astype(np.float64))], want.astype(np.float64))


def test_reference_layout():
    byte = np.arange(130 * 5).reshape(130, 5).astype(np.uint8)
    t = ref.tile(byte)
    assert t.shape == (2, 2, 512)
    assert t[0, 0, 33 % 32 * 16 + 1 * 4 + 2] == byte[33, 2] and t[1, 1, 16] == byte[129, 4]
    assert t[1, 1].sum() == int(byte[128, 4]) + int(byte[129, 4])
    codes = np.random.default_rng(1).integers(0, 16, size=(3, 32)).astype(np.uint8)
    assert np.array_equal(ref.unpack(ref.pack(codes)), codes)


def test_scale_bytes():
    f = fb.fp8blk_mx4_scale_bytes
    assert f(fb.MXFP4, 1, 32) == 512 and f(fb.NVFP4, 129, 80) == 2 * 2 * 512
    assert f(fb.MXFP4, 128, 1536) == 12 * 512 and f(fb.NVFP4, 0, 64) == 0
    assert f(2, 1, 32) == -1 and f(fb.MXFP4, -1, 32) == -1
    for fmt in (fb.MXFP4, fb.NVFP4):
        for rows, k in ((1, 32), (200, 1504)):
            assert f(fmt, rows, k) == int(np.prod(fb._mx4_scale_shape(fmt, rows, k)))


@pytest.mark.parametrize("args,code", [
    ((A, 5, 32, 32, 0, 0, N0, A, A, N0, N0, N0), 1),        # mode
    ((A, 5, 32, 32, 5, 0, N0, A, A, N0, N0, N0), 1),        # E5M2 has no 4-bit form
    ((A, 5, 32, 32, 1, 2, N0, A, A, N0, N0, N0), 1),        # format
    ((A, 5, 32, 32, 1, 0, A, A, A, N0, N0, N0), 1),         # a tensor scale with MXFP4
    ((A, 5, 32, 32, 1, 1, ODD, A, A, N0, N0, N0), 3),
    ((A, 5, 40, 40, 1, 0, N0, A, A, N0, N0, N0), 2),        # blocks along the columns: cols % 32
    ((A, -1, 32, 32, 1, 0, N0, A, A, N0, N0, N0), 2),
    ((A, 5, 0, 32, 2, 0, N0, N0, N0, A, A, N0), 2),
    ((A, 1 << 22, 1 << 22, 1 << 22, 1, 0, N0, A, A, N0, N0, N0), 2),   # tile count
    ((A, 5, 32, 24, 1, 0, N0, A, A, N0, N0, N0), 1),        # ldx < cols
    ((A, 5, 32, 36, 1, 0, N0, A, A, N0, N0, N0), 3),        # row stride
    ((M8, 5, 32, 32, 1, 0, N0, A, A, N0, N0, N0), 3),
    ((N0, 5, 32, 32, 1, 0, N0, A, A, N0, N0, N0), 1),
    ((A, 5, 32, 32, 1, 0, N0, A, N0, N0, N0, N0), 1),       # outputs
    ((A, 5, 32, 32, 3, 0, N0, A, A, A, N0, N0), 1),
    ((A, 5, 32, 32, 2, 0, N0, N0, N0, M8, A, N0), 3),
    ((N0, 0, 32, 32, 1, 0, N0, N0, N0, N0, N0, N0), 0),     # nothing to do
])
def test_quantiser_argument_errors(args, code):
    assert _lib.lib.fp8blk_quantize_mx4(*args) == code


@pytest.mark.parametrize("args,code", [
    ((A, A, 5, 32, 2, N0, A, 32, N0), 1),
    ((A, A, 5, 32, 0, A, A, 32, N0), 1),
    ((A, A, 5, 48, 0, N0, A, 48, N0), 2),
    ((A, A, 5, 32, 0, N0, A, 24, N0), 1),
    ((A, A, 5, 32, 0, N0, A, 36, N0), 3),
    ((A, N0, 5, 32, 0, N0, A, 32, N0), 1),
    ((A, A, 5, 32, 0, N0, M8, 32, N0), 3),
    ((N0, N0, 0, 32, 0, N0, N0, 32, N0), 0),
])
def test_dequantiser_argument_errors(args, code):
    assert _lib.lib.fp8blk_dequantize_mx4(*args) == code


@pytest.mark.parametrize("args,code", [
    ((2, 5, 8, 32, A, A, N0, A, A, N0, A, 8, N0), 1),       # format
    ((64, 5, 8, 32, A, A, N0, A, A, N0, A, 8, N0), 1),      # unknown flag
    ((0, 5, 8, 32, A, A, A, A, A, N0, A, 8, N0), 1),        # tensor scales with MXFP4
    ((0, 5, 8, 32, A, A, N0, A, A, A, A, 8, N0), 1),
    ((1, 5, 8, 32, A, A, N0, A, A, ODD, A, 8, N0), 3),
    ((0, -1, 8, 32, A, A, N0, A, A, N0, A, 8, N0), 2),
    ((0, 5, 0, 32, A, A, N0, A, A, N0, A, 8, N0), 2),
    ((0, 5, 8, 48, A, A, N0, A, A, N0, A, 8, N0), 2),
    ((0, 1 << 31, 8, 32, A, A, N0, A, A, N0, A, 8, N0), 2),
    ((0, 5, 8, 32, A, A, N0, A, A, N0, A, 4, N0), 1),       # ldd < N
    ((0, 5, 8, 32, A, A, N0, A, A, N0, A, 12, N0), 3),      # ldd % 8
    ((0 | 32, 5, 8, 32, A, A, N0, A, A, N0, A, 10, N0), 3), # fp32: ldd % 4
    ((0, 5, 8, 32, A, A, N0, A, A, N0, M8, 8, N0), 3),
    ((0, 5, 8, 32, A, N0, N0, A, A, N0, A, 8, N0), 1),
    ((0, 5, 8, 32, M8, A, N0, A, A, N0, A, 8, N0), 3),
    ((0, 5, 8, 0, N0, N0, N0, N0, N0, N0, N0, 8, N0), 1),   # no d
    ((0, 0, 8, 32, N0, N0, N0, A, A, N0, N0, 8, N0), 0),    # nothing to do
])
def test_gemm_argument_errors(args, code):
    assert _lib.lib.fp8blk_gemm_mx4(*args) == code


@pytest.mark.parametrize("args,code", [
    ((2, 5, 8, 32, A, 32, N0, A, A, N0, A, 1 << 20, A, 8, N0), 1),      # format
    ((0, 5, 8, 32, A, 32, A, A, A, N0, A, 1 << 20, A, 8, N0), 1),       # a tensor scale with MXFP4
    ((0, 5, 8, 48, A, 48, N0, A, A, N0, A, 1 << 20, A, 8, N0), 2),
    ((0, 5, 8, 32, A, 24, N0, A, A, N0, A, 1 << 20, A, 8, N0), 1),      # ldx < K
    ((0, 5, 8, 32, A, 36, N0, A, A, N0, A, 1 << 20, A, 8, N0), 3),
    ((0, 5, 8, 32, M8, 32, N0, A, A, N0, A, 1 << 20, A, 8, N0), 3),
    ((0, 5, 8, 32, N0, 32, N0, A, A, N0, A, 1 << 20, A, 8, N0), 1),
    ((0, 17, 8, 32, A, 32, N0, A, A, N0, N0, 1 << 20, A, 8, N0), 1),    # no workspace
    ((0, 5, 8, 32, A, 32, N0, A, A, N0, M8, 1 << 20, A, 8, N0), 3),
    ((0, 17, 8, 32, A, 32, N0, A, A, N0, A, 17 * 16 + 511, A, 8, N0), 1),   # too small
    ((0, 5, 8, 32, A, 32, N0, A, A, N0, A, 1 << 20, A, 4, N0), 1),      # ldd < N
    ((0, 0, 8, 32, N0, 32, N0, A, A, N0, N0, 0, N0, 8, N0), 0),         # nothing to do
])
def test_linear_argument_errors(args, code):
    assert _lib.lib.fp8blk_linear_mx4(*args) == code


def test_linear_workspace():
    f = fb.fp8blk_linear_mx4_workspace_bytes
    assert f(fb.MXFP4, 17, 32) == 17 * 16 + 512 and f(fb.MXFP4, 16, 32) == 0 and f(fb.NVFP4, 129, 96) == 129 * 48 + 2 * 2 * 512
    assert f(2, 5, 32) == -1 and f(fb.MXFP4, -1, 32) == -1 and f(fb.MXFP4, 5, 48) == -1 and f(fb.MXFP4, 0, 32) == 0


def test_binding_refuses():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    q, s = torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(1, 1, 512, dtype=torch.uint8)
    for call in (lambda: fb.fp8blk_quantize_mx4(x, fb.MXFP4), lambda: fb.fp8blk_quantize_mx4(x, 2),
                 lambda: fb.fp8blk_dequantize_mx4(q, s, fb.NVFP4),
                 lambda: fb.fp8blk_gemm_mx4(q, s, q, s, fb.NVFP4)):
        with pytest.raises(ValueError):
            call()
