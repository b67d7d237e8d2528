"""Refusals of the grouped entry points, and the padded layout's size: host logic, no GPU."""
import ctypes
import random

import pytest
import torch

import fp8_blockwise_scaled_b200 as fb
from fp8_blockwise_scaled_b200 import _lib

P = ctypes.c_void_p
A = P(0x10000)            # never dereferenced: every case below fails validation first
MISALIGNED = P(0x10008)
ODD = P(0x10002)
NULL = P(0)
S = NULL


def test_padded_rows_hold_every_split():
    rng = random.Random(1)
    for _ in range(2000):
        groups = rng.randrange(1, 40)
        counts = [rng.choice([0, 0, 1, rng.randrange(400)]) for _ in range(groups)]
        rows = sum(counts) + rng.choice([0, 0, rng.randrange(50)])
        padded = fb.fp8blk_grouped_padded_rows(rows, groups)
        assert padded % 128 == 0
        assert sum(-(-c // 128) * 128 for c in counts) <= padded <= rows + 127 * min(groups, rows)
    # and some split needs all of it
    assert fb.fp8blk_grouped_padded_rows(3, 8) == 3 * 128
    assert fb.fp8blk_grouped_padded_rows(129 + 1, 2) == 3 * 128
    assert fb.fp8blk_grouped_padded_rows(0, 4) == 0
    assert fb.fp8blk_grouped_padded_rows(-1, 4) == -1
    assert fb.fp8blk_grouped_padded_rows(5, 0) == -1 and fb.fp8blk_grouped_padded_rows(5, fb.MAX_GROUPS + 1) == -1


@pytest.mark.parametrize("args,code", [
    ((A, 5, 128, 128, 1, NULL, 2, A, A, NULL, NULL, S), 1),               # no offsets
    ((A, 5, 128, 128, 1, ODD, 2, A, A, NULL, NULL, S), 3),                # offsets not 4-byte aligned
    ((A, 5, 128, 128, 1, A, 0, A, A, NULL, NULL, S), 1),                  # no groups
    ((A, 5, 128, 128, 1, A, 1025, A, A, NULL, NULL, S), 1),               # too many
    ((A, -1, 128, 128, 1, A, 2, A, A, NULL, NULL, S), 2),                 # rows < 0
    ((A, 1 << 25, 128, 128, 1, A, 2, A, A, NULL, NULL, S), 2),            # too many rows
    ((A, 5, 100, 128, 1, A, 2, A, A, NULL, NULL, S), 2),                  # cols % 128
    ((A, 5, 128, 64, 1, A, 2, A, A, NULL, NULL, S), 1),                   # ldx < cols
    ((A, 5, 128, 132, 1, A, 2, A, A, NULL, NULL, S), 3),                  # row stride
    ((MISALIGNED, 5, 128, 128, 1, A, 2, A, A, NULL, NULL, S), 3),
    ((NULL, 5, 128, 128, 1, A, 2, A, A, NULL, NULL, S), 1),
    ((A, 5, 128, 128, 4, A, 2, A, A, NULL, NULL, S), 1),                  # E5M2 without a layout
    ((A, 0, 128, 128, 4, A, 2, A, A, NULL, NULL, S), 1),                  # also without rows
    ((A, 0, 128, 128, 9, A, 2, A, A, NULL, NULL, S), 1),
    ((A, 5, 128, 128, 2, A, 2, A, A, NULL, A, S), 1),                     # no q_colT
    ((A, 5, 128, 128, 3, A, 2, A, A, MISALIGNED, A, S), 3),
])
def test_quantiser_argument_errors(args, code):
    assert _lib.lib.fp8blk_quantize_act_1x128_grouped(*args) == code


@pytest.mark.parametrize("args,code", [
    ((3, 2, A, 5, 128, 128, A, A, A, A, A, 128, S), 1),                   # bad layout
    ((0, 2, NULL, 5, 128, 128, A, A, A, A, A, 128, S), 1),                # no offsets
    ((0, 0, A, 5, 128, 128, A, A, A, A, A, 128, S), 1),                   # groups
    ((0, 1025, A, 5, 128, 128, A, A, A, A, A, 128, S), 1),
    ((0, 2, ODD, 5, 128, 128, A, A, A, A, A, 128, S), 3),
    ((0, 2, A, -1, 128, 128, A, A, A, A, A, 128, S), 2),
    ((0, 2, A, 5, 100, 128, A, A, A, A, A, 128, S), 2),
    ((1, 2, A, 5, 128, 100, A, A, A, A, A, 128, S), 2),
    ((2, 2, A, 100, 128, 128, A, A, A, A, A, 128, S), 2),                 # WGRAD: M % 128
    ((2, 2, A, 128, 128, 100, A, A, A, A, A, 128, S), 2),                 # WGRAD: K not whole blocks
    ((0, 1024, A, 5, 1 << 21, 128, A, A, A, A, A, 1 << 21, S), 2),        # groups * N = 2^31
    ((0, 2, A, (1 << 31) - 1, 128, 128, A, A, A, A, A, 128, S), 2),
    ((0, 2, A, 5, 256, 128, A, A, A, A, A, 128, S), 1),                   # ldd < N
    ((0, 2, A, 5, 128, 128, A, A, A, A, A, 136, S), 3),
    ((0 | 32, 2, A, 5, 128, 128, A, A, A, A, A, 132, S), 3),
    ((0, 2, A, 5, 128, 128, A, A, A, A, P(0x10010), 128, S), 3),
    ((0, 2, A, 5, 128, 128, NULL, A, A, A, A, 128, S), 1),
    ((2, 2, A, 128, 128, 0, NULL, NULL, NULL, NULL, NULL, 128, S), 1),    # no d
    ((1, 2, A, 5, 128, 128, A, A, MISALIGNED, A, A, 128, S), 3),
])
def test_gemm_argument_errors(args, code):
    assert _lib.lib.fp8blk_gemm_grouped(*args) == code


@pytest.mark.parametrize("args,code", [
    ((1, 2, A, 5, 128, 128, A, 128, A, A, A, 1 << 20, A, 128, S), 1),      # format
    ((8, 2, A, 5, 128, 128, A, 128, A, A, A, 1 << 20, A, 128, S), 1),
    ((0, 2, NULL, 5, 128, 128, A, 128, A, A, A, 1 << 20, A, 128, S), 1),
    ((0, 2, A, 5, 100, 128, A, 128, A, A, A, 1 << 20, A, 128, S), 2),
    ((0, 2, A, 1 << 25, 128, 128, A, 128, A, A, A, 1 << 40, A, 128, S), 2),
    ((0, 2, A, 5, 128, 128, NULL, 128, A, A, A, 1 << 20, A, 128, S), 1),
    ((0, 2, A, 5, 128, 128, A, 64, A, A, A, 1 << 20, A, 128, S), 1),       # ldx < K
    ((0, 2, A, 5, 128, 128, A, 132, A, A, A, 1 << 20, A, 128, S), 3),
    ((0, 2, A, 5, 128, 128, MISALIGNED, 128, A, A, A, 1 << 20, A, 128, S), 3),
    ((0, 2, A, 17, 128, 128, A, 128, A, A, NULL, 1 << 20, A, 128, S), 1),  # no workspace
    ((0, 1, A, 13, 128, 128, A, 128, A, A, NULL, 1 << 20, A, 128, S), 1),
    ((0, 2, A, 5, 128, 128, A, 128, A, A, MISALIGNED, 1 << 20, A, 128, S), 3),
    ((0, 2, A, 25, 128, 128, A, 128, A, A, A, 25 * 132 - 1, A, 128, S), 1),  # too small
    ((0, 2, A, 5, 128, 128, A, 128, A, A, A, 1 << 20, A, 64, S), 1),       # ldd < N
    ((0, 2, A, 0, 128, 128, NULL, 128, A, A, NULL, 0, NULL, 128, S), 0),   # nothing to do
])
def test_linear_argument_errors(args, code):
    assert _lib.lib.fp8blk_linear_grouped(*args) == code


def test_linear_workspace():
    f = fb.fp8blk_linear_grouped_workspace_bytes
    assert f(2, 25, 256) == 25 * 256 + 25 * 2 * 4 and f(2, 0, 128) == 0 and f(2, 16, 128) == 0 and f(1, 12, 128) == 0
    assert f(1, 13, 128) == 13 * 132 and f(2, -1, 128) == -1 and f(2, 5, 100) == -1 and f(0, 5, 128) == -1


def test_calls_without_rows_need_no_gpu():
    assert _lib.lib.fp8blk_quantize_act_1x128_grouped(NULL, 0, 128, 128, 3, A, 2, NULL, NULL, NULL, NULL, S) == 0
    assert _lib.lib.fp8blk_gemm_grouped(0, 2, A, 0, 128, 128, NULL, NULL, A, A, NULL, 128, S) == 0


def test_binding_refuses():
    x = torch.zeros(5, 128, dtype=torch.bfloat16)
    off = torch.zeros(3, dtype=torch.int32)
    for bad in (off.long(), off[:1], off.reshape(1, 3), torch.zeros(fb.MAX_GROUPS + 2, dtype=torch.int32)):
        with pytest.raises(ValueError):
            fb.fp8blk_quantize_act_1x128_grouped(x, bad)
    with pytest.raises(ValueError):
        fb.fp8blk_quantize_act_1x128_grouped(x, off)               # not a CUDA tensor
    q = torch.zeros(5, 128, dtype=torch.uint8).view(torch.float8_e4m3fn)
    with pytest.raises(ValueError):
        fb.fp8blk_gemm_grouped(fb.FWD, q, x, q, x, off)
