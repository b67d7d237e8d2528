"""Grouped and 4-bit calls at their far ends: offsets beyond 32 bits, the most groups, and a row's result beside
other groups of any size.  Large results are compared with the same call on a part of the inputs, which the
other files check against their references."""
import numpy as np
import pytest
import torch

import fp8_blockwise_scaled_b200 as fb
from tests import test_gpu_grouped as grouped
from tests.gpu_helpers import require_cuda

pytestmark = pytest.mark.gpu

ROWS, COLS = 36000, 131072           # 4.7e9 elements
OFFSETS = [0, 100, 20000, 36000]


def _off(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _bits(t):
    return t.contiguous().view(torch.uint8)


@pytest.fixture
def large():
    """bf16 [ROWS, COLS] of the 4-bit grid's values, drawn anew everywhere."""
    require_cuda()
    gen = torch.Generator(device="cuda").manual_seed(1)
    grid = torch.tensor([0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.5, -1.0, -3.0, -6.0], device="cuda").bfloat16()
    x = torch.empty((ROWS, COLS), dtype=torch.bfloat16, device="cuda")
    for c in range(0, COLS, 8192):
        x[:, c:c + 8192] = grid[torch.randint(len(grid), (ROWS, 8192), generator=gen, device="cuda", dtype=torch.int32)]
    yield x
    del x
    torch.cuda.empty_cache()


def test_ragged_quantiser_beyond_32_bits(large):
    q, s, qT, sT = fb.fp8blk_quantize_act_1x128_grouped(large, _off(OFFSETS), fb.BOTH)
    assert fb.fp8blk_get_device_error() == 0
    a, b, _, _ = fb.fp8blk_quantize_act_1x128_grouped(large[-300:], _off([0, 300]))
    assert torch.equal(_bits(q[-300:]), _bits(a)) and torch.equal(s[:, -300:], b)
    _, _, a, b = fb.fp8blk_quantize_act_1x128_grouped(large[:, -256:], _off(OFFSETS), fb.COLWISE_T)
    blocks = sum(-(-(j - i) // 128) for i, j in zip(OFFSETS, OFFSETS[1:]))
    assert torch.equal(_bits(qT[-256:, :128 * blocks]), _bits(a[:, :128 * blocks]))
    assert torch.equal(sT[:blocks, -256:], b[:blocks])


@pytest.mark.parametrize("fmt", [fb.MXFP4, fb.NVFP4])
def test_mx4_quantiser_and_values_beyond_32_bits(large, fmt):
    q, s, qT, sT = fb.fp8blk_quantize_mx4(large, fmt, fb.BOTH)
    y = fb.fp8blk_dequantize_mx4(q, s, fmt)
    assert fb.fp8blk_get_device_error() == 0
    tail = ROWS // 128 * 128 - 128                                   # whole scale atoms
    a, b, _, _ = fb.fp8blk_quantize_mx4(large[tail:], fmt)
    assert torch.equal(q[tail:], a) and torch.equal(s[tail // 128:], b)
    assert torch.equal(y[tail:], fb.fp8blk_dequantize_mx4(a, b, fmt))
    del y, q, s
    _, _, a, b = fb.fp8blk_quantize_mx4(large[:, -256:], fmt, fb.COLWISE_T)
    assert torch.equal(qT[-256:], a) and torch.equal(sT[-2:], b)
    y = fb.fp8blk_dequantize_mx4(qT, sT, fmt)
    assert fb.fp8blk_get_device_error() == 0
    assert torch.equal(y[-256:], fb.fp8blk_dequantize_mx4(a, b, fmt))


def test_row_product_beyond_32_bits(large):
    """The last group's rows of 36000 x 131072 outputs."""
    k, groups = 128, 3
    w = large[:groups * 1024, :k].repeat(COLS // 1024, 1)            # [groups * COLS, k]
    qw, sw = fb.fp8blk_quantize_weight_128x128(w)
    x = large[:, :k]
    y = fb.grouped_linear_forward(x, qw, sw, _off(OFFSETS))
    part = fb.grouped_linear_forward(x[-200:], qw, sw, _off([0, 0, 0, 200]))
    assert fb.fp8blk_get_device_error() == 0
    assert torch.equal(y[-200:], part)


@pytest.mark.parametrize("fmt", [fb.MXFP4, fb.NVFP4])
def test_mx4_product_beyond_32_bits(large, fmt):
    """Every sum is exact, so every kernel gives the same."""
    k = 64
    a, sa, _, _ = fb.fp8blk_quantize_mx4(large[:, :k], fmt)
    b, sb, _, _ = fb.fp8blk_quantize_mx4(large[:, k:2 * k].repeat(4, 1)[:COLS], fmt)
    d = fb.fp8blk_gemm_mx4(a, sa, b, sb, fmt)
    row, col = ROWS // 128 * 128 - 128, COLS - 384
    part = fb.fp8blk_gemm_mx4(a[row:], sa[row // 128:], b[col:], sb[col // 128:], fmt)
    assert fb.fp8blk_get_device_error() == 0
    assert torch.equal(d[row:, col:], part)


def test_weight_gradient_beyond_32_bits():
    """300 groups of 4096 x 4096 from one token each: the last groups against a call of their own."""
    require_cuda()
    groups, n = 300, 4096
    x = torch.randn((groups, n), device="cuda").bfloat16()
    dy = torch.randn((groups, n), device="cuda").bfloat16()
    off = _off(list(range(groups + 1)))
    _, _, qa, sa = fb.fp8blk_quantize_act_1x128_grouped(dy, off, fb.COLWISE_T)
    _, _, qb, sb = fb.fp8blk_quantize_act_1x128_grouped(x, off, fb.COLWISE_T)
    dw = fb.fp8blk_gemm_grouped(fb.WGRAD, qa, sa, qb, sb, off)
    part = [t[:, -256:].contiguous() if i % 2 == 0 else t[-2:] for i, t in enumerate((qa, sa, qb, sb))]
    want = fb.fp8blk_gemm_grouped(fb.WGRAD, *part, _off([0, 1, 2]))
    assert fb.fp8blk_get_device_error() == 0
    assert torch.equal(dw[-2:], want) and bool(want.any())
    del dw
    torch.cuda.empty_cache()


def _many_groups():
    """1024 groups: most of no, one or two rows, some of more than a tile."""
    rng = np.random.default_rng(7)
    counts = rng.choice([0, 1, 2], size=fb.MAX_GROUPS)
    counts[[0, 500, 1023]] = 130, 17, 40
    return counts.tolist()


@pytest.mark.parametrize("e5m2", [False, True])
def test_most_groups_quantiser(e5m2, monkeypatch):
    monkeypatch.setitem(grouped.COUNTS, "most_groups", _many_groups())
    grouped.test_quantiser_matches_the_oracle_group_by_group("most_groups", fb.BOTH, e5m2)


@pytest.mark.parametrize("layout", [fb.FWD, fb.DGRAD])
@pytest.mark.parametrize("block_n", ["auto", "128", "256"])
def test_most_groups_row_products(layout, block_n, monkeypatch):
    monkeypatch.setitem(grouped.COUNTS, "most_groups", _many_groups())
    grouped.test_row_products("most_groups", layout, 256, 128, torch.bfloat16, block_n, monkeypatch)


def test_most_groups_weight_gradient(monkeypatch):
    monkeypatch.setitem(grouped.COUNTS, "most_groups", _many_groups())
    grouped.test_weight_gradient("most_groups", 128, 256, torch.float32, False)


@pytest.mark.parametrize("layout", [fb.FWD, fb.DGRAD])
@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
def test_a_rows_result_does_not_depend_on_the_other_groups(layout, out_dtype, monkeypatch):
    """Bit for bit, whichever kernel the number of rows, or the tile width, makes the library take."""
    require_cuda()
    n, k, groups, rows = 512, 1536, 4, 9
    gen = torch.Generator(device="cuda").manual_seed(3)
    w = torch.randn((groups * (n if layout == fb.FWD else k), k if layout == fb.FWD else n), generator=gen, device="cuda")
    qw, sw, qwT, swT = fb.fp8blk_quantize_weight_128x128_both(w.bfloat16())
    b, sb = (qw, sw) if layout == fb.FWD else (qwT, swT)
    mine = torch.randn((rows, k), generator=gen, device="cuda").bfloat16()
    results = []
    for counts in ([0, rows, 0, 0], [3, rows, 2, 1], [200, rows, 0, 70], [700, rows, 1000, 3]):
        for block_n in (None, "128", "256"):
            if block_n is None:
                monkeypatch.delenv("FP8BLK_GEMM_BLOCK_N", raising=False)
            else:
                monkeypatch.setenv("FP8BLK_GEMM_BLOCK_N", block_n)
            x = torch.randn((sum(counts), k), generator=gen, device="cuda").bfloat16()
            x[counts[0]:counts[0] + rows] = mine
            off = _off(np.concatenate([[0], np.cumsum(counts)]).tolist())
            a, sa, _, _ = fb.fp8blk_quantize_act_1x128_grouped(x, off)
            d = fb.fp8blk_gemm_grouped(layout, a, sa, b, sb, off, out_dtype=out_dtype)
            results.append(d[counts[0]:counts[0] + rows])
            if layout == fb.FWD:
                results.append(fb.fp8blk_linear_grouped(x, b, sb, off, out_dtype=out_dtype)[counts[0]:counts[0] + rows])
    assert fb.fp8blk_get_device_error() == 0
    for r in results[1:]:
        assert torch.equal(r, results[0])
