"""Calls with a `stream` argument: order on the stream that is named, and memory that belongs to it."""
import numpy as np
import pytest
import torch

import fp8_blockwise_scaled_b200 as fb
import workloads
from tests.gpu_helpers import require_cuda, to_dev

pytestmark = pytest.mark.gpu

T, K, N, GROUPS = 256, 256, 384, 2


def _x(rows, cols, seed):
    return to_dev(workloads.activation(np.random.default_rng(seed), rows, cols))


class Case:
    """Inputs of every entry point that takes a stream, and those calls."""

    def __init__(self):
        self.x, self.dy, self.w = _x(T, K, 1), _x(T, N, 2), _x(N, K, 3)
        self.off = torch.tensor([0, 100, T], dtype=torch.int32, device="cuda")
        self.few = self.off.clamp(max=9)
        self.one = torch.tensor([0.01], device="cuda")
        self.amax = [self.one.clone() for _ in range(8)]         # one for every call that updates it
        w2 = torch.cat([self.w, self.w])
        self.qw, self.sw, self.qwT, self.swT = fb.fp8blk_quantize_weight_128x128_both(w2)
        self.q4, self.s4, self.q4T, self.s4T = fb.fp8blk_quantize_mx4(self.w, fb.MXFP4, fb.BOTH)
        self.qx, self.sx, _, _ = fb.fp8blk_quantize_act_1x128(self.x)
        self.q1, self.s1 = fb.fp8blk_quantize_weight_128x128(self.w)
        self.qx4, self.sx4, _, _ = fb.fp8blk_quantize_mx4(self.x, fb.MXFP4)

    def layer(self, **k):
        """The layer functions: forward, few rows and backward over groups, then in 4 bits."""
        return (fb.grouped_linear_forward(self.x, self.qw, self.sw, self.off, **k),
                fb.grouped_linear_forward(self.x[:9], self.qw, self.sw, self.few, **k),
                *fb.grouped_linear_backward(self.x, self.dy, self.qwT, self.swT, self.off, **k),
                fb.mx4_linear_forward(self.x, self.q4, self.s4, fb.MXFP4, **k),
                fb.mx4_linear_forward(self.x[:9], self.q4, self.s4, fb.MXFP4, **k),
                fb.mx4_linear_wgrad(self.x, self.dy, fb.MXFP4, **k),
                *fb.mx4_linear_backward(self.x, self.dy, self.q4T, self.s4T, fb.MXFP4, **k))


@pytest.mark.parametrize("handle", ["0", "1", "current"])
def test_handle_of_the_default_stream_keeps_its_order(handle):
    """x and dy are written late on the default stream, and the results read on it at once: the calls wait for
    the one and the reads for the calls."""
    require_cuda()
    c = Case()
    x, dy = c.x.clone(), c.dy.clone()
    want = c.layer()
    torch.cuda.synchronize()
    handle = torch.cuda.current_stream().cuda_stream if handle == "current" else int(handle)
    c.x.zero_()
    c.dy.zero_()
    torch.cuda.synchronize()
    torch.cuda._sleep(300_000_000)
    c.x.copy_(x)
    c.dy.copy_(dy)
    got = [t.clone() for t in c.layer(stream=handle)]
    torch.cuda.synchronize()
    assert fb.fp8blk_get_device_error() == 0
    for a, b in zip(got, want):
        assert torch.equal(a, b)


PRIMITIVES = {
    "quantize_grouped": lambda c, **k: fb.fp8blk_quantize_act_1x128_grouped(c.x, c.off, fb.BOTH, **k),
    "gemm_grouped": lambda c, **k: fb.fp8blk_gemm_grouped(fb.FWD, c.qx, c.sx, c.qw, c.sw, c.off, **k),
    "quantize_mx4": lambda c, **k: fb.fp8blk_quantize_mx4(c.x, fb.MXFP4, fb.BOTH, **k),
    "dequantize_mx4": lambda c, **k: fb.fp8blk_dequantize_mx4(c.q4, c.s4, fb.MXFP4, **k),
    "gemm_mx4": lambda c, **k: fb.fp8blk_gemm_mx4(c.qx4, c.sx4, c.q4, c.s4, fb.MXFP4, **k),
}

BLOCKWISE = {
    "quantize_act": lambda c, **k: fb.fp8blk_quantize_act_1x128(c.x, fb.BOTH, **k),
    "quantize_weight": lambda c, **k: fb.fp8blk_quantize_weight_128x128(c.w, **k),
    "quantize_weight_t": lambda c, **k: fb.fp8blk_quantize_weight_128x128_t(c.w, **k),
    "quantize_weight_both": lambda c, **k: fb.fp8blk_quantize_weight_128x128_both(c.w, **k),
    "quantize_weights": lambda c, **k: tuple(t for o in fb.fp8blk_quantize_weights_128x128_both([c.w, c.w], **k) for t in o),
    "gemm": lambda c, **k: fb.fp8blk_gemm(fb.FWD, c.qx, c.sx, c.q1, c.s1, **k),
    "gemm_splitk": lambda c, **k: fb.fp8blk_gemm_splitk(fb.FWD, c.qx, c.sx, c.q1, c.s1, 2, **k),
    "amax_ema": lambda c, **k: fb.fp8blk_amax_ema(c.x, c.amax.pop(), **k)[1],
    "quantize_tensor": lambda c, **k: fb.fp8blk_quantize_tensor(c.x, c.one, **k),
    "gemm_tensor_scaled": lambda c, **k: fb.fp8blk_gemm_tensor_scaled(c.qx, c.one, c.q1, c.one, **k),
    "linear_forward": lambda c, **k: fb.linear_forward(c.x, c.w, **k),
    "linear_backward": lambda c, **k: fb.linear_backward(c.x, c.w, c.dy, **k),
    "linear_delayed": lambda c, **k: fb.fp8_linear_delayed_forward(c.x, c.w, c.amax.pop(), c.amax.pop(), **k),
}


def _bits(t):
    return t.contiguous().view(torch.uint8)


def _check_allocation(call):
    """Blocks of every size, freed behind a long queue of writes of NaN on the current stream, are not handed to a
    call on another stream."""
    want = call()
    want = want if isinstance(want, tuple) else (want,)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for stream in (side, side.cuda_stream):
        blocks = [torch.empty(1 << b, dtype=torch.uint8, device="cuda") for b in range(9, 24) for _ in range(3)]
        for _ in range(40):
            for b in blocks:
                b.fill_(255)
        taken = [(b.data_ptr(), b.data_ptr() + b.numel()) for b in blocks]
        del blocks, b
        got = call(stream=stream)
        got = got if isinstance(got, tuple) else (got,)
        torch.cuda.synchronize()
        assert fb.fp8blk_get_device_error() == 0
        for g, w in zip(got, want):
            if w is None:
                assert g is None
                continue
            assert not any(lo <= g.data_ptr() < hi for lo, hi in taken)
            assert g.shape == w.shape and g.dtype == w.dtype
            assert torch.equal(_bits(g), _bits(w))
        del got, g


@pytest.mark.parametrize("name", PRIMITIVES)
def test_primitives_allocate_from_the_named_stream(name):
    require_cuda()
    c = Case()
    _check_allocation(lambda **k: PRIMITIVES[name](c, **k))


@pytest.mark.parametrize("name", BLOCKWISE)
def test_blockwise_calls_allocate_from_the_named_stream(name):
    require_cuda()
    c = Case()
    torch.cuda.synchronize()
    _check_allocation(lambda **k: BLOCKWISE[name](c, **k))
