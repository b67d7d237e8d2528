"""The `stream` argument of the binding: which stream a handle names, and where missing outputs come from.  Host
logic, no GPU: torch's stream calls and the library's entry points are replaced."""
import contextlib

import pytest
import torch

import fp8_blockwise_scaled_b200 as fb

CPU = torch.device("cpu")


class FakeStream:
    def __init__(self, name):
        self.name, self.device = name, CPU


@pytest.fixture
def streams(monkeypatch):
    """The stream that is current, as torch.cuda.stream sets it; ExternalStream(h) is named by its handle."""
    now = [FakeStream("caller")]

    @contextlib.contextmanager
    def current(stream):
        now.append(stream)
        yield
        now.pop()

    monkeypatch.setattr(torch.cuda, "stream", current)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: now[-1])
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: FakeStream("default"))
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device=None: FakeStream(handle))
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda self, stream: None, raising=False)
    return now


@pytest.mark.parametrize("handle,name", [(0, "default"), (1, "default"), (2, 2), (0x7F00, 0x7F00)])
def test_handle_of_the_default_stream_is_that_stream(streams, handle, name):
    seen = []

    def call():
        seen.append(streams[-1].name)
        return torch.zeros(1)

    fb._on_stream(handle, CPU, call)
    assert seen == [name] and streams[-1].name == "caller"


def _args():
    """Tensors that pass the binding's checks, on the CPU."""
    f8, u8, f32 = torch.float8_e4m3fn, torch.uint8, torch.float32
    z = lambda *shape, t=torch.bfloat16: torch.zeros(shape, dtype=t)  # noqa: E731
    return {"x": z(128, 128), "off": torch.zeros(2, dtype=torch.int32), "q": z(128, 128, t=f8), "s": z(1, 128, t=f32),
            "sw": z(1, 1, t=f32), "q4": z(128, 64, t=u8), "s4": z(1, 1, 512, t=u8), "d": z(128, 128), "one": torch.ones(1)}


GROUPED_AND_MX4 = {
    "quantize_grouped": lambda a, **k: fb.fp8blk_quantize_act_1x128_grouped(a["x"], a["off"], fb.BOTH, **k),
    "quantize_grouped_some_given": lambda a, **k: fb.fp8blk_quantize_act_1x128_grouped(
        a["x"], a["off"], fb.BOTH, q_row=a["q"], s_row=a["s"], **k),
    "gemm_grouped": lambda a, **k: fb.fp8blk_gemm_grouped(fb.FWD, a["q"], a["s"], a["q"], a["sw"], a["off"], **k),
    "linear_grouped": lambda a, **k: fb.fp8blk_linear_grouped(a["x"], a["q"], a["sw"], a["off"], **k),
    "quantize_mx4": lambda a, **k: fb.fp8blk_quantize_mx4(a["x"], fb.MXFP4, fb.COLWISE_T, **k),
    "dequantize_mx4": lambda a, **k: fb.fp8blk_dequantize_mx4(a["q4"], a["s4"], fb.MXFP4, **k),
    "gemm_mx4": lambda a, **k: fb.fp8blk_gemm_mx4(a["q4"], a["s4"], a["q4"], a["s4"], fb.MXFP4, **k),
    "linear_mx4": lambda a, **k: fb.fp8blk_linear_mx4(a["x"], a["q4"], a["s4"], fb.MXFP4, **k),
}


@pytest.fixture
def made(streams, monkeypatch):
    """(shape, name of the current stream) of every tensor that a call makes; the library is not called."""
    seen = []
    real = torch.empty, torch.empty_strided

    def note(make):
        def made_by(shape, *args, **kwargs):
            seen.append((tuple(shape) if not isinstance(shape, int) else (shape,), streams[-1].name))
            return make(shape, *args, **kwargs)
        return made_by

    monkeypatch.setattr(torch, "empty", note(real[0]))
    monkeypatch.setattr(torch, "empty_strided", note(real[1]))
    monkeypatch.setattr(fb, "_need_cuda", lambda *tensors: CPU)
    monkeypatch.setattr(fb, "_run", lambda *args: None)
    monkeypatch.setattr(fb, "_stream_handle", lambda stream, device=None: 0)
    monkeypatch.setattr(fb, "fp8blk_gemm_splitk_workspace_bytes", lambda *args: 128 * 128 * 4)
    monkeypatch.setattr(torch.cuda, "device", lambda device: contextlib.nullcontext())
    return seen


BLOCKWISE = {
    "quantize_act": lambda a, **k: fb.fp8blk_quantize_act_1x128(a["x"], fb.BOTH, **k),
    "quantize_act_some_given": lambda a, **k: fb.fp8blk_quantize_act_1x128(a["x"], q_row=a["q"], **k),
    "quantize_weight": lambda a, **k: fb.fp8blk_quantize_weight_128x128(a["x"], q=a["q"], **k),
    "quantize_weight_t": lambda a, **k: fb.fp8blk_quantize_weight_128x128_t(a["x"], **k),
    "quantize_weight_both": lambda a, **k: fb.fp8blk_quantize_weight_128x128_both(a["x"], **k),
    "quantize_weights": lambda a, **k: fb.fp8blk_quantize_weights_128x128_both([a["x"], a["x"]], **k),
    "gemm": lambda a, **k: fb.fp8blk_gemm(fb.FWD, a["q"], a["s"], a["q"], a["sw"], **k),
    "gemm_splitk_workspace": lambda a, **k: fb.fp8blk_gemm_splitk(fb.FWD, a["q"], a["s"], a["q"], a["sw"], 2, d=a["d"], **k),
    "round": lambda a, **k: fb.fp8blk_round_f32_to_bf16(a["s"], **k),
    "amax_ema": lambda a, **k: fb.fp8blk_amax_ema(a["x"], a["one"], scale=a["one"], **k),
    "quantize_tensor": lambda a, **k: fb.fp8blk_quantize_tensor(a["x"], a["one"], **k),
    "gemm_tensor_scaled": lambda a, **k: fb.fp8blk_gemm_tensor_scaled(a["q"], a["one"], a["q"], a["one"], **k),
    "linear_forward": lambda a, **k: fb.linear_forward(a["x"], a["x"], **k),
    "linear_backward": lambda a, **k: fb.linear_backward(a["x"], a["x"], a["x"], **k),
    "linear_delayed": lambda a, **k: fb.fp8_linear_delayed_forward(a["x"], a["x"], a["one"], a["one"], **k),
}
EVERY = {**GROUPED_AND_MX4, **BLOCKWISE}


@pytest.mark.parametrize("name", EVERY)
def test_missing_outputs_come_from_the_named_stream(made, name):
    """Memory of the caller's current stream may still be written by that stream's earlier work."""
    EVERY[name](_args(), stream=0x7F00)
    assert made and {where for _, where in made} == {0x7F00}
    made.clear()
    EVERY[name](_args())
    assert made and {where for _, where in made} == {"caller"}


def test_nothing_is_made_where_every_output_is_given(made):
    a = _args()
    for call in (lambda **k: fb.fp8blk_quantize_act_1x128_grouped(a["x"], a["off"], q_row=a["q"], s_row=a["s"], **k),
                 lambda **k: fb.fp8blk_gemm_grouped(fb.FWD, a["q"], a["s"], a["q"], a["sw"], a["off"], d=a["d"], **k),
                 lambda **k: fb.fp8blk_quantize_mx4(a["x"], fb.MXFP4, q_row=a["q4"], s_row=a["s4"], **k),
                 lambda **k: fb.fp8blk_dequantize_mx4(a["q4"], a["s4"], fb.MXFP4, y=a["d"], **k),
                 lambda **k: fb.fp8blk_gemm_mx4(a["q4"], a["s4"], a["q4"], a["s4"], fb.MXFP4, d=a["d"], **k)):
        call(stream=0x7F00)
    assert not made


def test_outputs_of_another_device_are_refused():
    """A host pointer, or another GPU's, would reach the kernel."""
    t = torch.zeros(4, 8)
    assert fb._out(t, (4, 8), torch.float32, CPU) is t
    with pytest.raises(ValueError, match="on cuda:0"):
        fb._out(t, (4, 8), torch.float32, torch.device("cuda", 0))
