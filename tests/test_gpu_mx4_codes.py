"""The 4-bit quantiser's codes with their signs, and what it makes of values that are not finite."""
import numpy as np
import pytest
import torch

import fp8_blockwise_scaled_b200 as fb
import workloads
from tests import mx4_reference as ref
from tests.gpu_helpers import require_cuda, to_dev

pytestmark = pytest.mark.gpu

FORMATS = {"mxfp4": fb.MXFP4, "nvfp4": fb.NVFP4}


def _scalar(g):
    return None if g is None else torch.tensor([g], dtype=torch.float32, device="cuda")


def _x(rows, cols, seed):
    """Both signs of zero, zero blocks, and blocks of both signs that are too small for any scale but zero."""
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((rows, cols)).astype(np.float32)
    x[rng.random((rows, cols)) < 0.1] = 0.0
    x[rng.random((rows, cols)) < 0.1] = -0.0
    tiny = rng.random((-(-rows // 32), cols // 16)) < 0.3
    tiny = np.repeat(np.repeat(tiny, 32, 0), 16, 1)[:rows]
    x[tiny] *= np.float32(1e-9)
    empty = np.repeat(np.repeat(rng.random((-(-rows // 32), cols // 16)) < 0.2, 32, 0), 16, 1)[:rows]
    x[empty] = np.where(rng.random(x[empty].shape) < 0.5, 0.0, -0.0)
    return workloads.f32_to_bf16(x)


@pytest.mark.parametrize("rows,cols", [(1, 32), (31, 160), (300, 416)])
@pytest.mark.parametrize("fmt,g", [("mxfp4", None), ("nvfp4", None), ("nvfp4", 0.0071)])
def test_codes_with_their_signs(rows, cols, fmt, g):
    """A block whose NVFP4 scale is zero has the codes 0, whatever its signs; elsewhere zeros keep theirs."""
    require_cuda()
    bits = _x(rows, cols, rows + cols)
    x = workloads.bf16_to_f32(bits).astype(np.float64)
    q, s, qT, sT = fb.fp8blk_quantize_mx4(to_dev(bits), FORMATS[fmt], fb.BOTH, _scalar(g))
    q1, _, _, _ = fb.fp8blk_quantize_mx4(to_dev(bits), FORMATS[fmt], fb.ROWWISE, _scalar(g))
    assert fb.fp8blk_get_device_error() == 0
    codes, byte = ref.quantize(x, fmt, g or 1.0)
    codesT, byteT = ref.quantize(np.ascontiguousarray(ref.pad_rows(x).T), fmt, g or 1.0)
    if fmt == "nvfp4" and rows > 1:
        assert (byte == 0).any() and (byteT == 0).any()
    assert np.array_equal(s.cpu().numpy(), ref.tile(byte)) and np.array_equal(sT.cpu().numpy(), ref.tile(byteT))
    assert np.array_equal(ref.unpack(q.cpu().numpy()), codes)
    assert np.array_equal(ref.unpack(q1.cpu().numpy()), codes)
    assert np.array_equal(ref.unpack(qT.cpu().numpy()), codesT)


def test_zeros_come_back_without_a_sign():
    require_cuda()
    x = torch.zeros((40, 96), dtype=torch.bfloat16, device="cuda")
    for fmt in FORMATS.values():
        q, s, qT, sT = fb.fp8blk_quantize_mx4(x, fmt, fb.BOTH)
        for a, b in ((q, s), (qT, sT)):
            assert not bool(a.any()) and not bool(fb.fp8blk_dequantize_mx4(a, b, fmt).view(torch.int16).any())


def test_few_rows_quantised_on_the_way_have_the_same_codes():
    """Rows of zero blocks and tiny values of both signs: bit for bit the product of the quantiser's codes."""
    require_cuda()
    x, w = to_dev(_x(16, 416, 1)), to_dev(_x(72, 416, 2))
    qw, sw, _, _ = fb.fp8blk_quantize_mx4(w, fb.NVFP4, tensor_scale=_scalar(0.0071))
    qx, sx, _, _ = fb.fp8blk_quantize_mx4(x, fb.NVFP4, tensor_scale=_scalar(0.0071))
    want = fb.fp8blk_gemm_mx4(qx, sx, qw, sw, fb.NVFP4, _scalar(0.0071), _scalar(0.0071), out_dtype=torch.float32)
    got = fb.fp8blk_linear_mx4(x, qw, sw, fb.NVFP4, _scalar(0.0071), _scalar(0.0071), out_dtype=torch.float32)
    assert fb.fp8blk_get_device_error() == 0
    assert torch.equal(got.view(torch.int32), want.view(torch.int32))


def _dev8(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def test_e8m0_byte_255_is_nan_in_the_values_and_in_the_product():
    """The format's NaN, whatever the codes below it; every other byte is its power of two."""
    require_cuda()
    codes = np.tile(np.arange(16, dtype=np.uint8), (256, 2))
    byte = np.arange(256, dtype=np.uint8)[:, None]
    y = fb.fp8blk_dequantize_mx4(_dev8(ref.pack(codes)), _dev8(ref.tile(byte)), fb.MXFP4).float().cpu().numpy()
    assert np.isnan(y[255]).all()
    with np.errstate(over="ignore"):
        want = ref.values(codes[:255], byte[:255], "mxfp4").astype(np.float32)
    assert np.array_equal(y[:255], torch.from_numpy(want).to(torch.bfloat16).float().numpy())
    for m in (5, 200):
        ones, scales = np.full((m, 64), 2, np.uint8), np.full((m, 2), 127, np.uint8)
        scales[3, 1] = 255
        a = _dev8(ref.pack(ones)), _dev8(ref.tile(scales))
        b = _dev8(ref.pack(ones[:2])), _dev8(ref.tile(np.full((2, 2), 127, np.uint8)))
        d = fb.fp8blk_gemm_mx4(*a, *b, fb.MXFP4, out_dtype=torch.float32).cpu().numpy()
        assert np.isnan(d[3]).all() and (np.delete(d, 3, 0) == 64.0).all()
    assert fb.fp8blk_get_device_error() == 0


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("m", [9, 200])
def test_a_value_that_is_not_finite_makes_its_block_nan(fmt, bad, m):
    """Its block's scale is the format's NaN in both directions, so its row of a product is NaN and its token's
    column of a weight gradient too; every other block is as without it."""
    require_cuda()
    f, b, k, n = FORMATS[fmt], ref.BLOCK[fmt], 160, 80
    row, col = m // 2, 70
    x = workloads.bf16_to_f32(_x(m, k, 3))
    x[row, col] = 1.0
    clean = to_dev(workloads.f32_to_bf16(x))
    x[row, col] = bad
    dirty = clean.clone()
    dirty[row, col] = bad
    nan = 255 if fmt == "mxfp4" else 0x7F
    q, s, qT, sT = fb.fp8blk_quantize_mx4(dirty, f, fb.BOTH)
    q1, s1, _, _ = fb.fp8blk_quantize_mx4(dirty, f, fb.ROWWISE)
    c, t, cT, tT = fb.fp8blk_quantize_mx4(clean, f, fb.BOTH)
    assert torch.equal(s, s1) and torch.equal(q, q1)
    for got, want, r, at, codes, clean_codes in ((s, t, row, col, q, c), (sT, tT, col, row, qT, cT)):
        place = (r // 128, at // b // 4, (r % 32) * 16 + (r % 128 // 32) * 4 + at // b % 4)
        assert int(got[place]) == nan
        got, want = got.clone(), want.clone()
        got[place] = want[place] = 0
        assert torch.equal(got, want)
        span = slice(at // b * b // 2, (at // b + 1) * b // 2)
        codes, clean_codes = codes.clone(), clean_codes.clone()
        codes[r, span] = clean_codes[r, span] = 0
        assert torch.equal(codes, clean_codes)
    y = fb.fp8blk_dequantize_mx4(q, s, f).float()
    inside = torch.zeros_like(y, dtype=torch.bool)
    inside[row, col // b * b:(col // b + 1) * b] = True
    assert torch.equal(torch.isnan(y), inside)
    w, dy = to_dev(_x(n, k, 4)), to_dev(_x(m, n, 5))
    qw, sw, _, _ = fb.fp8blk_quantize_mx4(w, f)
    d = fb.mx4_linear_forward(dirty, qw, sw, f)
    dw = fb.mx4_linear_wgrad(dirty, dy, f)
    assert fb.fp8blk_get_device_error() == 0
    assert bool(torch.isnan(d[row]).all()) and bool(torch.isnan(dw[:, col]).all())
    rest = torch.arange(m, device="cuda") != row
    assert bool(torch.isfinite(d[rest]).all()) and bool(torch.isfinite(dw[:, torch.arange(k, device="cuda") != col]).all())
    assert torch.equal(d[rest], fb.mx4_linear_forward(clean, qw, sw, f)[rest])


@pytest.mark.parametrize("cols", [10, 96])
def test_single_row_of_any_stride(cols):
    """A row without a pitch, in and out; what stands beside it stays."""
    require_cuda()
    k = 64
    x = _x(1, 96, 6)[:, :cols]
    around = torch.full((cols + 3,), 7.0, dtype=torch.bfloat16, device="cuda")
    row = around[:cols].reshape(1, cols)
    row.copy_(to_dev(x))
    _, _, qT, sT = fb.fp8blk_quantize_mx4(row, fb.MXFP4, fb.COLWISE_T)
    codes, byte = ref.quantize(np.ascontiguousarray(ref.pad_rows(workloads.bf16_to_f32(x).astype(np.float64)).T), "mxfp4")
    assert np.array_equal(sT.cpu().numpy(), ref.tile(byte)) and np.array_equal(ref.unpack(qT.cpu().numpy()), codes)
    w, v = to_dev(_x(cols, k, 7) if cols % 8 == 0 else _x(16, k, 7)[:cols]), to_dev(_x(1, k, 8))
    qw, sw, _, _ = fb.fp8blk_quantize_mx4(w, fb.MXFP4)
    want = fb.fp8blk_linear_mx4(v, qw, sw, fb.MXFP4)
    fb.fp8blk_linear_mx4(v, qw, sw, fb.MXFP4, d=row)
    assert fb.fp8blk_get_device_error() == 0
    assert torch.equal(row, want) and bool((around[cols:] == 7.0).all())


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("m", [64, 256])
def test_product_of_every_scale_byte(fmt, m):
    """1.0 in one place a row below every scale byte, the smallest and the subnormal ones among them: D is the
    product of two scales exactly, wherever fp32 holds it as a normal number."""
    require_cuda()
    k, n = 64, 4
    b = ref.BLOCK[fmt]
    one, none = np.array([56 if fmt == "nvfp4" else 127], np.uint8), np.uint8(0)
    last = 127 if fmt == "nvfp4" else 255
    for first in range(0, last, m):
        mine = (np.arange(first, first + m) % last).astype(np.uint8)
        ca, ba = np.zeros((m, k), np.uint8), np.full((m, k // b), none)
        place = (np.arange(m) * 7) % k
        ca[np.arange(m), place] = 2
        ba[np.arange(m), place // b] = mine
        bb = np.repeat(np.array([one[0], 1, last - 1, last // 3], np.uint8)[:, None], k // b, 1)
        d = fb.fp8blk_gemm_mx4(_dev8(ref.pack(ca)), _dev8(ref.tile(ba)), _dev8(ref.pack(np.full((n, k), 2, np.uint8))),
                               _dev8(ref.tile(bb)), FORMATS[fmt], out_dtype=torch.float32).cpu().numpy()
        want = ref.values(ca, ba, fmt) @ ref.values(np.full((n, k), 2, np.uint8), bb, fmt).T
        held = (want == 0) | ((want >= 2.0**-126) & (want < 2.0**128))
        assert held.any() and np.array_equal(d[held], want[held].astype(np.float32))
    assert fb.fp8blk_get_device_error() == 0
