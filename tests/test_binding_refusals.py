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
