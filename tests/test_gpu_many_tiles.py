"""The grouped and 4-bit kernels with several tiles a CTA.

The kernels are persistent, and the cases of the other files have fewer tiles than
the GPU has SMs, so a CTA sees one or two of them.  Here the same cases run on a few
CTAs: rings of stages, scales, accumulators and tile places carry over from tile to
tile, staging areas are used again, groups are stepped over.  K = 128 has a tile in
every K-block; K = 4224 has 33 K-blocks, which read the weights' scales (32 at a
time) twice."""
import numpy as np
import pytest
import torch

import fp8_blockwise_scaled_b200 as fb
import workloads
from tests import test_gpu_grouped as grouped
from tests import test_gpu_mx4 as mx4
from tests.gpu_helpers import assert_gemm_close, f32, require_cuda, to_dev

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture
def few_ctas(monkeypatch):
    monkeypatch.setenv("FP8BLK_GEMM_MAX_CTAS", "3")
    monkeypatch.setenv("FP8BLK_QUANT_MAX_CTAS", "3")
    return monkeypatch


@pytest.mark.parametrize("counts", grouped.COUNTS, ids=str)
@pytest.mark.parametrize("mode", [fb.ROWWISE, fb.COLWISE_T, fb.BOTH])
@pytest.mark.parametrize("e5m2", [False, True])
def test_ragged_quantiser(counts, mode, e5m2, few_ctas):
    grouped.test_quantiser_matches_the_oracle_group_by_group(counts, mode, e5m2)


def test_ragged_quantiser_leaves_rows_outside_every_group_alone(few_ctas):
    grouped.test_quantiser_leaves_rows_outside_every_group_alone()


@pytest.mark.parametrize("counts", grouped.COUNTS, ids=str)
@pytest.mark.parametrize("layout", [fb.FWD, fb.DGRAD])
@pytest.mark.parametrize("n,k", [(1280, 128), (512, 4224)])
@pytest.mark.parametrize("out_dtype,block_n", [(BF16, "auto"), (BF16, "128"), (BF16, "256"), (F32, "auto"), (F32, "256")])
def test_row_products(counts, layout, n, k, out_dtype, block_n, few_ctas):
    grouped.test_row_products(counts, layout, n, k, out_dtype, block_n, few_ctas)


@pytest.mark.parametrize("block_n,counts", [("128", [70, 0, 129, 3]), ("256", [70, 0, 129, 3]), ("0", [3, 0, 7, 1, 2]),
                                            ("0", [3, 0, 70, 100, 2])])
def test_rows_outside_every_group_and_the_row_pitch_stay(block_n, counts, few_ctas):
    grouped.test_rows_outside_every_group_and_the_row_pitch_stay(block_n, counts, few_ctas)


@pytest.mark.parametrize("counts", ["edges", "single_rows", "most_empty", "uneven"])
@pytest.mark.parametrize("n_out,n_in", [(384, 256), (256, 640)])
@pytest.mark.parametrize("out_dtype", [BF16, F32])
@pytest.mark.parametrize("e5m2", [False, True])
def test_weight_gradient(counts, n_out, n_in, out_dtype, e5m2, few_ctas):
    grouped.test_weight_gradient(counts, n_out, n_in, out_dtype, e5m2)


@pytest.mark.parametrize("counts", [[1, 0, 3, 2, 0, 0, 4, 1], [16, 0], [1] * 16])
@pytest.mark.parametrize("k", [128, 4224])
@pytest.mark.parametrize("out_dtype", [BF16, F32])
def test_few_rows_quantised_on_the_way(counts, k, out_dtype, few_ctas):
    """One launch, against the formula in 64 bits on the oracle's codes."""
    require_cuda()
    n, rows = 640, sum(counts)
    x = workloads.activation_with_outliers(np.random.default_rng(k + rows), rows, k, frac=0.01)
    qa, sa = grouped._rowwise_ref(x, False)
    (qw, sw), _ = grouped._weights(len(counts), n, k, 3)
    assert fb.fp8blk_linear_grouped_workspace_bytes(len(counts), rows, k) == 0
    y = fb.fp8blk_linear_grouped(to_dev(x), grouped._f8(qw), grouped._dev(sw), grouped._offsets(counts),
                                 out_dtype=out_dtype)
    assert fb.fp8blk_get_device_error() == 0
    assert_gemm_close(f32(y), grouped._rows_ref(fb.FWD, qa, sa, qw, sw, counts, n, k), str(counts))


@pytest.mark.parametrize("rows,cols", [(300, 416), (257, 1536), (1300, 160)])
@pytest.mark.parametrize("mode", [fb.ROWWISE, fb.COLWISE_T, fb.BOTH])
@pytest.mark.parametrize("fmt,g", [("mxfp4", None), ("nvfp4", 0.0071)])
def test_mx4_quantiser(rows, cols, mode, fmt, g, few_ctas):
    mx4.test_quantiser(rows, cols, mode, fmt, g)


@pytest.mark.parametrize("m,n,k", [(16, 640, 256), (130, 264, 544), (257, 520, 800), (384, 1000, 1536), (700, 131, 288)])
@pytest.mark.parametrize("fmt,g", [("mxfp4", None), ("nvfp4", 0.0071)])
@pytest.mark.parametrize("out_dtype", [BF16, F32])
def test_mx4_product(m, n, k, fmt, g, out_dtype, few_ctas):
    mx4.test_product(m, n, k, fmt, g, g, out_dtype)


@pytest.mark.parametrize("m,n,k", [(2560, 2048, 512), (2500, 2100, 288), (256, 19000, 96)])
@pytest.mark.parametrize("fmt", mx4.FORMATS)
@pytest.mark.parametrize("out_dtype", [BF16, F32])
def test_mx4_product_on_pairs(m, n, k, fmt, out_dtype, monkeypatch):
    """Two pairs of CTAs, about 40 tiles each."""
    monkeypatch.setenv("FP8BLK_GEMM_MAX_CTAS", "4")
    mx4.test_large_product(m, n, k, fmt, out_dtype)
