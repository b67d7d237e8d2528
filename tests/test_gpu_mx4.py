"""4-bit microscaled quantisation and products on the GPU against numpy in 64 bits.

Quantiser: scale bytes and code values equal to the definition's, bit for bit
(a zero's sign apart), padding included.  Products: operands quantised by the
reference, so the GEMM is checked on its own.  Its fp32 result is a sum of K
products that are exact in fp32 (codes of 2 bits, scales of 1 or 4 bits), so
what differs from 64 bits is the accumulation: at most K roundings, each at
most half a step of a partial sum, which the sum of magnitudes S bounds:
|error| <= K 2^-24 S for sums kept in fp32.  The tensor cores keep a few bits
less below the largest addend of a step (64 values), 2^-21 of it or better is
asked here once a step and addend: |error| <= (K / 64) 2^-21 S + K 2^-24 S.
bf16 adds its half step, 2^-8 |D| (2^-9 rounded up for the product by the tensor
scales)."""
import numpy as np
import pytest
import torch

import fp8_blockwise_scaled_b200 as fb
import workloads
from tests import mx4_reference as ref
from tests.gpu_helpers import require_cuda, to_dev

pytestmark = pytest.mark.gpu

FORMATS = {"mxfp4": fb.MXFP4, "nvfp4": fb.NVFP4}


def _x(rows, cols, seed, spread=True):
    """Values over many binades, with zero blocks, exact ties and the largest magnitudes of a block repeated."""
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((rows, cols)).astype(np.float32)
    if spread:
        x *= np.exp2(rng.integers(-12, 8, size=(rows, 1))).astype(np.float32)
        x[rng.random((rows, cols)) < 0.05] = 0.0
        x[rows // 3] = 0.0
        x[:, cols // 3] = -0.0
        x[rows // 2] = rng.choice([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, -5.0], size=cols)
    return workloads.f32_to_bf16(x)


def _f64(bits):
    return workloads.bf16_to_f32(bits).astype(np.float64)


def _dev8(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def _scalar(g):
    return None if g is None else torch.tensor([g], dtype=torch.float32, device="cuda")


def _same_codes(q, codes, what):
    got = ref.unpack(q.cpu().numpy())
    got = np.where(got == 8, 0, got)
    want = np.where(codes == 8, 0, codes)
    bad = np.argwhere(got != want)
    assert bad.size == 0, f"{what}: {len(bad)} codes differ, first at {bad[0]}: {got[tuple(bad[0])]} {want[tuple(bad[0])]}"


SHAPES = [(1, 32), (3, 96), (31, 160), (128, 128), (129, 224), (300, 416), (257, 1536)]


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("mode", [fb.ROWWISE, fb.COLWISE_T, fb.BOTH])
@pytest.mark.parametrize("fmt,g", [("mxfp4", None), ("nvfp4", None), ("nvfp4", 0.0071), ("nvfp4", 1e-5)])
def test_quantiser(rows, cols, mode, fmt, g):
    require_cuda()
    pad = 8                                        # row pitch above the columns
    bits = _x(rows, cols + pad, rows + cols)
    x = _f64(bits)[:, :cols]
    q, s, qT, sT = fb.fp8blk_quantize_mx4(to_dev(bits)[:, :cols], FORMATS[fmt], mode, _scalar(g))
    assert fb.fp8blk_get_device_error() == 0
    if mode & fb.ROWWISE:
        codes, byte = ref.quantize(x, fmt, g or 1.0)
        assert np.array_equal(s.cpu().numpy(), ref.tile(byte)), "row scales"
        _same_codes(q, codes, "row codes")
    else:
        assert q is None and s is None
    if mode & fb.COLWISE_T:
        codes, byte = ref.quantize(np.ascontiguousarray(ref.pad_rows(x).T), fmt, g or 1.0)
        assert np.array_equal(sT.cpu().numpy(), ref.tile(byte)), "column scales"
        _same_codes(qT, codes, "column codes")
    else:
        assert qT is None and sT is None


@pytest.mark.parametrize("rows,cols", [(70, 1), (33, 13), (260, 130)])
@pytest.mark.parametrize("fmt", FORMATS)
def test_columns_of_any_number_along_the_rows(rows, cols, fmt):
    require_cuda()
    wide = -(-cols // 8) * 8
    bits = _x(rows, wide, rows)
    _, _, qT, sT = fb.fp8blk_quantize_mx4(to_dev(bits)[:, :cols], FORMATS[fmt], fb.COLWISE_T)
    assert fb.fp8blk_get_device_error() == 0
    codes, byte = ref.quantize(np.ascontiguousarray(ref.pad_rows(_f64(bits)[:, :cols]).T), fmt)
    assert np.array_equal(sT.cpu().numpy(), ref.tile(byte))
    _same_codes(qT, codes, "column codes")


def test_largest_and_smallest_values():
    """The ends of bf16: scales that saturate or vanish, subnormal inputs."""
    require_cuda()
    x = np.zeros((4, 64), np.float32)
    x[0, :32] = np.linspace(1.0, 3.3e38, 32)
    x[1, :32] = 2.0**-130
    x[1, 32:] = 2.0**-126 * np.arange(32)
    x[2] = 1e-3 * np.arange(64)
    x[3, 5] = -2.0**-133
    bits = workloads.f32_to_bf16(x)
    for fmt, g in (("mxfp4", None), ("nvfp4", 1e33), ("nvfp4", 1e-3)):
        v = _f64(bits)
        if g == 1e-3:
            v = v[1:]
        b = bits[1:] if g == 1e-3 else bits
        q, s, _, _ = fb.fp8blk_quantize_mx4(to_dev(b), FORMATS[fmt], tensor_scale=_scalar(g))
        codes, byte = ref.quantize(v, fmt, g or 1.0)
        assert np.array_equal(s.cpu().numpy(), ref.tile(byte)), (fmt, g)
        _same_codes(q, codes, f"{fmt} {g}")


@pytest.mark.parametrize("rows,cols", [(1, 32), (129, 224), (300, 1536)])
@pytest.mark.parametrize("fmt,g", [("mxfp4", None), ("nvfp4", None), ("nvfp4", 0.0071)])
def test_dequantised_values(rows, cols, fmt, g):
    require_cuda()
    codes, byte = ref.quantize(_f64(_x(rows, cols, 3)), fmt, g or 1.0)
    wide = torch.full((rows, cols + 8), 7.0, dtype=torch.bfloat16, device="cuda")
    fb.fp8blk_dequantize_mx4(_dev8(ref.pack(codes)), _dev8(ref.tile(byte)), FORMATS[fmt], _scalar(g), y=wide[:, :cols])
    assert fb.fp8blk_get_device_error() == 0
    v = np.where(codes & 8, -1.0, 1.0) * ref.GRID[codes & 7]
    if fmt == "mxfp4":
        want = ref.values(codes, byte, fmt).astype(np.float32)
    else:
        d = (ref.e4m3_values()[byte] * np.float64(np.float32(g or 1.0))).astype(np.float32)
        want = (v * np.repeat(d.astype(np.float64), 16, axis=1)).astype(np.float32)
    want = torch.from_numpy(want).to(torch.bfloat16)
    assert torch.equal(wide[:, :cols].cpu(), want)
    assert bool((wide[:, cols:] == 7.0).all())


def _operand(rows, k, fmt, seed, g=None):
    codes, byte = ref.quantize(_f64(_x(rows, k, seed, spread=False)), fmt, g or 1.0)
    return (_dev8(ref.pack(codes)), _dev8(ref.tile(byte))), ref.values(codes, byte, fmt)


def _assert_product(d, a, b, alpha, k, bf16, what):
    exact = alpha * (a @ b.T)
    s = abs(alpha) * (np.abs(a) @ np.abs(b).T)
    err = np.abs(d.double().cpu().numpy() - exact)
    bound = (np.ceil(k / 64) * 2.0**-21 + k * 2.0**-24) * s + (2.0**-8 * np.abs(exact) if bf16 else 2.0**-22 * np.abs(exact))
    worst = np.max(err - bound)
    assert np.all(np.isfinite(err)) and worst <= 0, f"{what}: {np.argwhere(err > bound)[:4]} of {err.shape}, by {worst}"


GEMM_SHAPES = [(1, 1, 32), (1, 200, 96), (5, 136, 512), (16, 128, 256), (17, 300, 224), (33, 129, 1504), (64, 64, 64),
               (65, 72, 320), (128, 128, 256), (130, 264, 544), (257, 520, 800), (384, 1000, 1536), (700, 131, 288),
               (2, 264, 4128), (20, 130, 2592), (50, 1000, 8960), (64, 4000, 1056)]


@pytest.mark.parametrize("m,n,k", GEMM_SHAPES)
@pytest.mark.parametrize("fmt,ga,gb", [("mxfp4", None, None), ("nvfp4", None, None), ("nvfp4", 0.0071, 3.0)])
@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
def test_product(m, n, k, fmt, ga, gb, out_dtype):
    require_cuda()
    (qa, sa), a = _operand(m, k, fmt, m + k, ga)
    (qb, sb), b = _operand(n, k, fmt, n + 7 * k, gb)
    d = fb.fp8blk_gemm_mx4(qa, sa, qb, sb, FORMATS[fmt], _scalar(ga), _scalar(gb), out_dtype=out_dtype)
    assert fb.fp8blk_get_device_error() == 0
    assert d.shape == (m, n) and d.dtype == out_dtype
    alpha = np.float64(np.float32(ga or 1.0) * np.float32(gb or 1.0))
    _assert_product(d, a, b, alpha, k, out_dtype == torch.bfloat16, f"{m} {n} {k} {fmt}")


@pytest.mark.parametrize("m", [7, 150, 400])
@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
def test_nothing_but_the_product_is_written(m, out_dtype):
    """Row pitch and rows around d stay; columns that are no multiple of anything."""
    require_cuda()
    n, k = 203, 352
    (qa, sa), a = _operand(m, k, "mxfp4", 1)
    (qb, sb), b = _operand(n, k, "mxfp4", 2)
    wide = torch.full((m + 3, n + 21), 7.0, dtype=out_dtype, device="cuda")
    fb.fp8blk_gemm_mx4(qa, sa, qb, sb, fb.MXFP4, d=wide[:m, :n])
    assert fb.fp8blk_get_device_error() == 0
    _assert_product(wide[:m, :n], a, b, 1.0, k, out_dtype == torch.bfloat16, "pitched")
    assert bool((wide[m:] == 7.0).all()) and bool((wide[:, n:] == 7.0).all())


def test_scales_of_every_row_and_block_reach_their_products():
    """One code a row (1.0) at a moving place, every scale another power of two: D shows which scale was taken."""
    require_cuda()
    m, n, k = 256, 256, 512
    rng = np.random.default_rng(4)
    for fmt in FORMATS:
        b = ref.BLOCK[fmt]
        ca, cb = np.zeros((m, k), np.uint8), np.full((n, k), 2, np.uint8)
        ca[np.arange(m), (np.arange(m) * 37) % k] = 2
        if fmt == "mxfp4":
            ba, bb = rng.integers(120, 134, size=(m, k // b)), rng.integers(120, 134, size=(n, k // b))
        else:
            ba, bb = 8 * rng.integers(2, 13, size=(m, k // b)), 8 * rng.integers(2, 13, size=(n, k // b))
        ba, bb = ba.astype(np.uint8), bb.astype(np.uint8)
        d = fb.fp8blk_gemm_mx4(_dev8(ref.pack(ca)), _dev8(ref.tile(ba)), _dev8(ref.pack(cb)), _dev8(ref.tile(bb)),
                               FORMATS[fmt], out_dtype=torch.float32)
        want = ref.values(ca, ba, fmt) @ ref.values(cb, bb, fmt).T
        assert np.array_equal(d.cpu().numpy(), want.astype(np.float32)), fmt


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("tokens", [1, 45, 300])
def test_layer_forward_and_backward(fmt, tokens):
    """The passes of a linear layer through the public entry points, against the definition in 64 bits."""
    require_cuda()
    n, k = 160, 224
    xb, wb = _x(tokens, k, 1, False), _x(n, k, 2, False)
    dyb = workloads.grad_output(np.random.default_rng(3), tokens, n)
    x, w, dy = _f64(xb), _f64(wb), _f64(dyb)
    g = [None if fmt == "mxfp4" else float(np.float32(np.abs(v).max() / 2688)) for v in (x, w, dy)]
    gx, gw, gdy = (_scalar(v) for v in g)
    f = FORMATS[fmt]
    qw, sw, qwT, swT = fb.fp8blk_quantize_mx4(to_dev(wb), f, fb.BOTH, gw)
    y = fb.mx4_linear_forward(to_dev(xb), qw, sw, f, gx, gw)
    dx, dw = fb.mx4_linear_backward(to_dev(xb), to_dev(dyb), qwT, swT, f, gx, gdy, gw, out_dtype=torch.float32)
    dw2 = fb.mx4_linear_wgrad(to_dev(xb), to_dev(dyb), f, gx, gdy, out_dtype=torch.float32)
    assert fb.fp8blk_get_device_error() == 0
    assert torch.equal(dw, dw2)

    def rows(v, i):
        return ref.values(*ref.quantize(np.ascontiguousarray(v), fmt, g[i] or 1.0), fmt)

    def alpha(i, j):
        return 1.0 if fmt == "mxfp4" else np.float64(np.float32(g[i]) * np.float32(g[j]))

    _assert_product(y, rows(x, 0), rows(w, 1), alpha(0, 1), k, True, "forward")
    _assert_product(dx, rows(dy, 2), rows(w.T, 1), alpha(2, 1), n, True, "dx")
    _assert_product(dw, rows(ref.pad_rows(dy).T, 2), rows(ref.pad_rows(x).T, 0), alpha(2, 0), tokens, False, "dw")


def test_no_tokens():
    require_cuda()
    n, k = 96, 64
    x = torch.empty((0, k), dtype=torch.bfloat16, device="cuda")
    dy = torch.empty((0, n), dtype=torch.bfloat16, device="cuda")
    qw, sw, _, _ = fb.fp8blk_quantize_mx4(to_dev(_x(n, k, 1)), fb.MXFP4)
    assert fb.mx4_linear_forward(x, qw, sw, fb.MXFP4).shape == (0, n)
    dw = fb.mx4_linear_wgrad(x, dy, fb.MXFP4)
    assert dw.shape == (n, k) and bool((dw == 0).all())
    assert fb.fp8blk_dequantize_mx4(*fb.fp8blk_quantize_mx4(x, fb.NVFP4)[:2], fb.NVFP4).shape == (0, k)


def test_captured_graph_on_a_side_stream():
    require_cuda()
    m, n, k = 9, 256, 512
    w = to_dev(_x(n, k, 5, False))
    qw, sw, _, _ = fb.fp8blk_quantize_mx4(w, fb.NVFP4)
    X = torch.zeros((m, k), dtype=torch.bfloat16, device="cuda")
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(stream):
        fb.mx4_linear_forward(X, qw, sw, fb.NVFP4)
        stream.synchronize()
        with torch.cuda.graph(graph, stream=stream):
            Y = fb.mx4_linear_forward(X, qw, sw, fb.NVFP4)
    torch.cuda.synchronize()
    for seed in (1, 2):
        X.copy_(to_dev(_x(m, k, seed, False)))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(Y, fb.mx4_linear_forward(X, qw, sw, fb.NVFP4))
    assert fb.fp8blk_get_device_error() == 0
    del graph


@pytest.mark.parametrize("m", [4, 256, 19000])
def test_stalled_product_reports_timeout_and_recovers(m, monkeypatch):
    require_cuda()
    n, k = 256, 512
    (qa, sa), a = _operand(m, k, "nvfp4", 1)
    (qb, sb), b = _operand(n, k, "nvfp4", 2)
    assert fb.fp8blk_get_device_error() == 0
    monkeypatch.setenv("FP8BLK_TEST_INJECT_STALL", "1")
    monkeypatch.setenv("FP8BLK_WAIT_TIMEOUT_MS", "200")
    fb.fp8blk_gemm_mx4(qa, sa, qb, sb, fb.NVFP4)
    assert fb.fp8blk_get_device_error() == 6
    assert fb.fp8blk_get_device_error() == 0
    monkeypatch.delenv("FP8BLK_TEST_INJECT_STALL")
    d = fb.fp8blk_gemm_mx4(qa, sa, qb, sb, fb.NVFP4)
    assert fb.fp8blk_get_device_error() == 0
    _assert_product(d, a, b, 1.0, k, True, "after timeout")


@pytest.mark.parametrize("m,n,k", [(2560, 2048, 512), (2500, 2100, 288), (256, 19000, 96)])
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
def test_large_product(m, n, k, fmt, out_dtype):
    """Enough 256 x 256 tiles for every pair of SMs, the last ones cut in both directions and along K."""
    require_cuda()
    g = None if fmt == "mxfp4" else 0.02
    (qa, sa), a = _operand(m, k, fmt, 1, g)
    (qb, sb), b = _operand(n, k, fmt, 2, g)
    d = fb.fp8blk_gemm_mx4(qa, sa, qb, sb, FORMATS[fmt], _scalar(g), _scalar(g), out_dtype=out_dtype)
    assert fb.fp8blk_get_device_error() == 0
    alpha = 1.0 if g is None else np.float64(np.float32(g) * np.float32(g))
    _assert_product(d, a, b, alpha, k, out_dtype == torch.bfloat16, f"{m} {n} {k} {fmt}")


@pytest.mark.parametrize("m", [3, 300])
def test_layer_on_a_stream_that_is_passed_in(m):
    require_cuda()
    n, k = 203, 352
    X, W, DY = to_dev(_x(m, k, 1, False)), to_dev(_x(n, k, 2, False)), to_dev(_x(m, 208, 3, False))[:, :n]
    qw, sw, _, _ = fb.fp8blk_quantize_mx4(W, fb.MXFP4)
    want = fb.mx4_linear_forward(X, qw, sw, fb.MXFP4), fb.mx4_linear_wgrad(X, DY, fb.MXFP4)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream):
        with torch.cuda.stream(side):
            torch.cuda._sleep(2_000_000)
        got = fb.mx4_linear_forward(X, qw, sw, fb.MXFP4, stream=stream), fb.mx4_linear_wgrad(X, DY, fb.MXFP4, stream=stream)
        junk = [torch.full((1 << 20,), 0x7F, dtype=torch.uint8, device="cuda") for _ in range(8)]
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
        del junk
    assert fb.fp8blk_get_device_error() == 0


@pytest.mark.parametrize("m,n,k", [(1, 1, 32), (1, 1536, 8960), (3, 200, 4128), (7, 136, 96), (16, 264, 1504),
                                   (16, 130, 288), (17, 264, 544), (200, 72, 320)])
@pytest.mark.parametrize("fmt,gx,gw", [("mxfp4", None, None), ("nvfp4", None, None), ("nvfp4", 0.0071, 0.5)])
@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
def test_quantised_on_the_way_is_the_two_calls(m, n, k, fmt, gx, gw, out_dtype):
    """Bit for bit the result of the quantiser and the product; rows of x with a pitch."""
    require_cuda()
    f = FORMATS[fmt]
    x = to_dev(_x(max(m, 3), k + 8, m + n))[:m, :k]
    qw, sw, _, _ = fb.fp8blk_quantize_mx4(to_dev(_x(n, k, 5, False)), f, fb.ROWWISE, _scalar(gw))
    qx, sx, _, _ = fb.fp8blk_quantize_mx4(x, f, fb.ROWWISE, _scalar(gx))
    want = fb.fp8blk_gemm_mx4(qx, sx, qw, sw, f, _scalar(gx), _scalar(gw), out_dtype=out_dtype)
    size = fb.fp8blk_linear_mx4_workspace_bytes(f, m, k)
    work = torch.full((size + 64,), 0x55, dtype=torch.uint8, device="cuda")
    wide = torch.full((m + 1, -(-n // 8) * 8 + 8), 7.0, dtype=out_dtype, device="cuda")
    got = fb.fp8blk_linear_mx4(x, qw, sw, f, _scalar(gx), _scalar(gw), d=wide[:m, :n], workspace=work[:size])
    assert fb.fp8blk_get_device_error() == 0
    assert torch.equal(got, want)
    assert torch.equal(fb.fp8blk_linear_mx4(x, qw, sw, f, _scalar(gx), _scalar(gw), out_dtype=out_dtype), want)
    assert bool((work[size:] == 0x55).all()) and bool((wide[m:] == 7.0).all()) and bool((wide[:, n:] == 7.0).all())


def test_few_rows_under_a_cap_on_the_ctas(monkeypatch):
    """With few CTAs allowed another kernel runs; the same values but for the order of the sums."""
    require_cuda()
    x, w = to_dev(_x(5, 1536, 1, False)), to_dev(_x(640, 1536, 2, False))
    (qx, sx, _, _), (qw, sw, _, _) = fb.fp8blk_quantize_mx4(x, fb.NVFP4), fb.fp8blk_quantize_mx4(w, fb.NVFP4)
    want = fb.fp8blk_gemm_mx4(qx, sx, qw, sw, fb.NVFP4, out_dtype=torch.float32)
    monkeypatch.setenv("FP8BLK_GEMM_MAX_CTAS", "3")
    got = fb.fp8blk_gemm_mx4(qx, sx, qw, sw, fb.NVFP4, out_dtype=torch.float32)
    assert fb.fp8blk_get_device_error() == 0
    # Sums of 1536 exact products in fp32, in two orders: each within 1536 2^-24 and 24 steps' 2^-21 of the sum of magnitudes.
    a, b = (fb.fp8blk_dequantize_mx4(*t, fb.NVFP4).double().abs() for t in ((qx, sx), (qw, sw)))
    bound = 2 * (24 * 2.0**-21 + 1536 * 2.0**-24) * (a @ b.t())
    assert bool(((got.double() - want.double()).abs() <= bound).all())


@pytest.mark.parametrize("fmt", FORMATS)
def test_stalled_product_that_quantises_reports_timeout_and_recovers(fmt, monkeypatch):
    require_cuda()
    x, w = to_dev(_x(5, 1536, 1, False)), to_dev(_x(200, 1536, 2, False))
    qw, sw, _, _ = fb.fp8blk_quantize_mx4(w, FORMATS[fmt])
    want = fb.fp8blk_linear_mx4(x, qw, sw, FORMATS[fmt])
    assert fb.fp8blk_get_device_error() == 0
    monkeypatch.setenv("FP8BLK_TEST_INJECT_STALL", "1")
    monkeypatch.setenv("FP8BLK_WAIT_TIMEOUT_MS", "200")
    fb.fp8blk_linear_mx4(x, qw, sw, FORMATS[fmt])
    assert fb.fp8blk_get_device_error() == 6
    monkeypatch.delenv("FP8BLK_TEST_INJECT_STALL")
    assert torch.equal(fb.fp8blk_linear_mx4(x, qw, sw, FORMATS[fmt]), want)
    assert fb.fp8blk_get_device_error() == 0


@pytest.mark.parametrize("g", [-1.0, -0.0, 0.0, float("nan"), float("inf"), -float("inf")])
def test_tensor_scales_that_are_not_positive_give_bytes_in_range(g):
    """The device holds the scalar, so the host cannot refuse it: codes are unspecified, scale bytes have no sign."""
    require_cuda()
    x = torch.linspace(-3, 3, 160 * 96, device="cuda").reshape(160, 96).bfloat16()
    _, s, _, sT = fb.fp8blk_quantize_mx4(x, fb.NVFP4, fb.BOTH, tensor_scale=_scalar(g))
    _, s1, _, _ = fb.fp8blk_quantize_mx4(x, fb.NVFP4, fb.ROWWISE, tensor_scale=_scalar(g))
    assert int(s.max()) < 128 and int(sT.max()) < 128 and torch.equal(s, s1)
    assert fb.fp8blk_get_device_error() == 0
