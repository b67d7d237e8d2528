"""The binding asks the library how much workspace a call needs: host logic, no GPU."""
import random

import pytest
import torch

import fp8_blockwise_scaled_b200 as fb


@pytest.fixture
def calls(monkeypatch):
    """Arguments of the library's entry points, which are not called; tensors on the CPU."""
    seen = []
    monkeypatch.setattr(fb, "_need_cuda", lambda *tensors: torch.device("cpu"))
    monkeypatch.setattr(fb, "_run", lambda device, fn, *args: seen.append(args))
    monkeypatch.setattr(fb, "_stream_handle", lambda stream, device=None: 0)
    return seen


def _grouped(rows):
    q, s = torch.zeros((128, 128), dtype=torch.float8_e4m3fn), torch.zeros((1, 1))
    fb.fp8blk_linear_grouped(torch.zeros((rows, 128), dtype=torch.bfloat16), q, s, torch.zeros(2, dtype=torch.int32))


def _mx4(rows):
    q, s = torch.zeros((8, 64), dtype=torch.uint8), torch.zeros((1, 1, 512), dtype=torch.uint8)
    fb.fp8blk_linear_mx4(torch.zeros((rows, 128), dtype=torch.bfloat16), q, s, fb.MXFP4)


@pytest.mark.parametrize("call,size", [(_grouped, "fp8blk_linear_grouped_workspace_bytes"),
                                       (_mx4, "fp8blk_linear_mx4_workspace_bytes")])
@pytest.mark.parametrize("rows,need", [(3, 4096), (40, 0), (41, 12345)])
def test_size_is_the_librarys(calls, monkeypatch, call, size, rows, need):
    """Another rule in the library (here: the other way round) needs no change of the binding."""
    monkeypatch.setattr(fb, size, lambda *args: need)
    call(rows)
    (args,) = calls
    work, given = args[-5:-3]
    assert given == need and (work is None) == (need == 0)


def test_sizes_are_those_of_each_call(calls):
    rng = random.Random(3)
    for _ in range(200):
        rows = rng.choice([1, 12, 13, 16, 17, rng.randrange(300)])
        calls.clear()
        _grouped(rows)
        _mx4(rows)
        assert calls[0][-4] == fb.fp8blk_linear_grouped_workspace_bytes(1, rows, 128)
        assert calls[1][-4] == fb.fp8blk_linear_mx4_workspace_bytes(fb.MXFP4, rows, 128)
