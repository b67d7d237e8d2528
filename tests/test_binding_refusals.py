"""Calls of the layer functions that only the binding can refuse: host logic, no GPU."""
import pytest
import torch

import fp8_blockwise_scaled_b200 as fb


@pytest.fixture(autouse=True)
def no_library(monkeypatch):
    monkeypatch.setattr(fb, "_need_cuda", lambda *tensors: torch.device("cpu"))
    monkeypatch.setattr(fb, "_run", lambda *args: None)
    monkeypatch.setattr(fb, "_stream_handle", lambda stream, device=None: 0)


@pytest.mark.parametrize("tokens", [(33, 40), (5, 6), (128, 127)])
def test_backward_of_other_numbers_of_tokens(tokens):
    """Their padded operands may have the same size, which hid it."""
    x, dy = (torch.zeros((t, 128), dtype=torch.bfloat16) for t in tokens)
    off = torch.zeros(2, dtype=torch.int32)
    q8, s8 = torch.zeros((128, 128), dtype=torch.float8_e4m3fn), torch.zeros((1, 1))
    q4, s4 = torch.zeros((128, 64), dtype=torch.uint8), torch.zeros((1, 1, 512), dtype=torch.uint8)
    for call in (lambda: fb.grouped_linear_backward(x, dy, q8, s8, off),
                 lambda: fb.mx4_linear_backward(x, dy, q4, s4, fb.MXFP4),
                 lambda: fb.mx4_linear_wgrad(x, dy, fb.MXFP4)):
        with pytest.raises(ValueError, match="tokens"):
            call()
    same = torch.zeros((tokens[0], 128), dtype=torch.bfloat16)
    fb.grouped_linear_backward(x, same, q8, s8, off)
    fb.mx4_linear_backward(x, same, q4, s4, fb.MXFP4)
    fb.mx4_linear_wgrad(x, same, fb.MXFP4)


def test_single_row_of_any_stride(monkeypatch):
    """The stride of a matrix of one row says nothing: the library gets a pitch that it takes."""
    seen = []
    monkeypatch.setattr(fb, "_run", lambda device, fn, *args: seen.append(args))
    row = torch.zeros(1, 129, dtype=torch.bfloat16)[:, :128]                     # pitch 129
    odd = torch.zeros(1, 10, dtype=torch.bfloat16)                               # contiguous, 10 columns
    q8, s8 = torch.zeros((128, 128), dtype=torch.float8_e4m3fn), torch.zeros((1, 1))
    q4, s4 = torch.zeros((10, 64), dtype=torch.uint8), torch.zeros((1, 1, 512), dtype=torch.uint8)
    off = torch.zeros(2, dtype=torch.int32)
    fb.fp8blk_quantize_act_1x128_grouped(row, off)
    assert seen.pop()[3] == 128
    fb.fp8blk_quantize_mx4(row, fb.MXFP4)
    assert seen.pop()[3] == 128
    fb.fp8blk_quantize_mx4(odd, fb.MXFP4, fb.COLWISE_T)
    assert seen.pop()[3] == 16
    fb.fp8blk_linear_grouped(row, q8, s8, off, d=row)
    args = seen.pop()
    assert args[7] == 128 and args[-2] == 128
    fb.fp8blk_linear_mx4(row, q4, s4, fb.MXFP4, d=odd)
    args = seen.pop()
    assert args[5] == 128 and args[-2] == 16
    wide = torch.zeros(2, 136, dtype=torch.bfloat16)[:, :128]                    # two rows: their own pitch
    fb.fp8blk_quantize_mx4(wide, fb.MXFP4)
    assert seen.pop()[3] == 136


def test_per_tensor_calls_refuse_what_the_kernels_would_read_or_write_wrongly():
    """Shapes, types and strides that reach the kernel as bare pointers."""
    f8, f32 = torch.float8_e4m3fn, torch.float32
    q, one = torch.zeros((128, 128), dtype=f8), torch.ones(1)
    x = torch.zeros((128, 128), dtype=torch.bfloat16)
    fb.fp8blk_gemm_tensor_scaled(q, one, q, one, d=torch.zeros((128, 256), dtype=torch.bfloat16)[:, :128])
    fb.fp8blk_quantize_tensor(x, one)
    wide = torch.zeros((128, 256), dtype=f8)[:, :128]
    for call in (lambda: fb.fp8blk_gemm_tensor_scaled(wide, one, q, one), lambda: fb.fp8blk_gemm_tensor_scaled(q, one, wide, one),
                 lambda: fb.fp8blk_gemm_tensor_scaled(q, one.half(), q, one),
                 lambda: fb.fp8blk_gemm_tensor_scaled(q, one, q, torch.ones(0)),
                 lambda: fb.fp8blk_gemm_tensor_scaled(q, one, q, one, d=torch.zeros((128, 64), dtype=torch.bfloat16)),
                 lambda: fb.fp8blk_gemm_tensor_scaled(q, one, q, one, d=torch.zeros((128, 128))),
                 lambda: fb.fp8blk_gemm_tensor_scaled(q, one, q, one, d=x.t()),
                 lambda: fb.fp8blk_quantize_tensor(x, one.half()), lambda: fb.fp8blk_quantize_tensor(x, torch.ones(0)),
                 lambda: fb.fp8blk_gemm(fb.FWD, q, torch.ones(1, 128).half(), q, torch.ones(1, 1)),
                 lambda: fb.fp8blk_gemm(fb.FWD, q, torch.ones(1, 128), q, torch.ones(1, 1).half())):
        with pytest.raises(ValueError):
            call()
