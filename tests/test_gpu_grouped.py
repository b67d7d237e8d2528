"""Rows sorted by group (tokens sorted by expert): the ragged quantiser and the grouped GEMMs.

The reference is the CPU oracle run group by group: a group's rows padded with
zeros to whole 128-row blocks give the same codes and scales for the rows that
exist (a zero row changes no maximum) and the same sums, in 64 bits.  Codes and
scales are compared bit for bit, GEMM outputs with the library's tolerance
(tests/gpu_helpers.py)."""
import numpy as np
import pytest
import torch

import fp8_blockwise_scaled_b200 as fb
import oracle
import workloads
from tests.gpu_helpers import assert_bits_equal, assert_gemm_close, f32, require_cuda, to_dev, u8

pytestmark = pytest.mark.gpu

# Rows per group: empty groups first, last and between, groups that end inside a
# 32-row quarter, at a block's end and one row behind it.
COUNTS = {
    "one_row": [1],
    "one_group": [300],
    "edges": [0, 1, 127, 0, 128, 129, 31, 32, 33, 0],
    "single_rows": [1] * 17,
    "most_empty": [0] * 40 + [5] + [0] * 60 + [260] + [0] * 27,
    "uneven": [513, 2, 64, 0, 255, 384, 7],
    "tiny": [3, 0, 5, 2],
    "few": [12, 0, 16, 33, 5],
    "some": [40, 0, 65, 20, 1],
}


def _offsets(counts, start=0):
    return torch.tensor(np.concatenate([[start], start + np.cumsum(counts)]).astype(np.int32)).cuda()


def _pad(x, rows=128):
    """x padded with zero rows to a multiple of `rows`, at least one block."""
    want = max(rows, -(-x.shape[0] // rows) * rows)
    return np.concatenate([x, np.zeros((want - x.shape[0], x.shape[1]), x.dtype)])


def _spans(counts, start=0):
    ends = np.concatenate([[start], start + np.cumsum(counts)])
    return [slice(int(a), int(b)) for a, b in zip(ends, ends[1:])]


def _rowwise_ref(x, e5m2):
    q, s = oracle.quantize_act_rowwise(_pad(x), oracle.E5M2 if e5m2 else oracle.E4M3)
    return q[:x.shape[0]], s[:, :x.shape[0]]


def _colwise_ref(x, counts, padded, e5m2, start=0):
    """q [cols, padded] and s [padded/128, cols] of the groups' blocks, and the number of blocks."""
    q, s, at = np.zeros((x.shape[1], padded), np.uint8), np.zeros((padded // 128, x.shape[1]), np.float32), 0
    for span in _spans(counts, start):
        if span.stop > span.start:
            qe, se = oracle.quantize_act_colwise_t(_pad(x[span]), oracle.E5M2 if e5m2 else oracle.E4M3)
            q[:, 128 * at:128 * at + qe.shape[1]] = qe
            s[at:at + se.shape[0]] = se
            at += se.shape[0]
    return q, s, at


@pytest.mark.parametrize("counts", COUNTS, ids=str)
@pytest.mark.parametrize("mode", [fb.ROWWISE, fb.COLWISE_T, fb.BOTH])
@pytest.mark.parametrize("e5m2", [False, True])
def test_quantiser_matches_the_oracle_group_by_group(counts, mode, e5m2):
    require_cuda()
    counts = COUNTS[counts]
    rows, cols, pad = sum(counts), 384, 64
    x = workloads.activation_with_outliers(np.random.default_rng(rows + mode), rows, cols + pad, frac=0.01)
    X = to_dev(x)[:, :cols]
    x = x[:, :cols]
    q, s, qT, sT = fb.fp8blk_quantize_act_1x128_grouped(X, _offsets(counts), mode | (fb.E5M2 if e5m2 else 0))
    assert fb.fp8blk_get_device_error() == 0
    if mode & fb.ROWWISE:
        rq, rs = _rowwise_ref(x, e5m2)
        assert_bits_equal(u8(q), rq, "row codes")
        assert_bits_equal(f32(s), rs, "row scales")
    else:
        assert q is None and s is None
    if mode & fb.COLWISE_T:
        padded = fb.fp8blk_grouped_padded_rows(rows, len(counts))
        rq, rs, blocks = _colwise_ref(x, counts, padded, e5m2)
        assert_bits_equal(u8(qT)[:, :128 * blocks], rq[:, :128 * blocks], "column codes")
        assert_bits_equal(f32(sT)[:blocks], rs[:blocks], "column scales")
    else:
        assert qT is None and sT is None


def test_quantiser_leaves_rows_outside_every_group_alone():
    require_cuda()
    counts, start, rows, cols = [100, 0, 45], 10, 200, 256
    x = workloads.activation(np.random.default_rng(5), rows, cols)
    padded = fb.fp8blk_grouped_padded_rows(rows, len(counts))
    q = torch.full((rows, cols), 0x55, dtype=torch.uint8, device="cuda")
    s = torch.full((cols // 128, rows), -7.0, device="cuda")
    qT = torch.full((cols, padded), 0x55, dtype=torch.uint8, device="cuda")
    sT = torch.full((padded // 128, cols), -7.0, device="cuda")
    f8 = torch.float8_e4m3fn
    fb.fp8blk_quantize_act_1x128_grouped(to_dev(x), _offsets(counts, start), fb.BOTH, q.view(f8), s, qT.view(f8), sT)
    assert fb.fp8blk_get_device_error() == 0
    stop = start + sum(counts)
    rq, rs = _rowwise_ref(x, False)
    assert_bits_equal(u8(q)[start:stop], rq[start:stop], "row codes")
    assert_bits_equal(f32(s)[:, start:stop], rs[:, start:stop], "row scales")
    for part in (q[:start], q[stop:]):
        assert bool((part == 0x55).all())
    for part in (s[:, :start], s[:, stop:]):
        assert bool((part == -7.0).all())
    rq, rs, blocks = _colwise_ref(x, counts, padded, False, start)
    assert_bits_equal(u8(qT)[:, :128 * blocks], rq[:, :128 * blocks], "column codes")
    assert bool((qT[:, 128 * blocks:] == 0x55).all()) and bool((sT[blocks:] == -7.0).all())


def _f8(a, e5m2=False):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda().view(torch.float8_e5m2 if e5m2 else torch.float8_e4m3fn)


def _dev(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).cuda()


def _weights(groups, n, k, seed):
    """W [groups, n, k] as one weight of groups * n rows: (q, s) and (qT, sT)."""
    w = workloads.weight(np.random.default_rng(seed), groups * n, k)
    return oracle.quantize_weight(w), oracle.quantize_weight_t(w)


def _rows_ref(layout, qa, sa, qb, sb, counts, n, k, fmt=0, start=0):
    """FWD / DGRAD in 64 bits, group by group; rows of qa that no group owns give NaN."""
    out = np.full((qa.shape[0], n), np.nan)
    groups = len(counts)
    for e, span in enumerate(_spans(counts, start)):
        if span.stop == span.start:
            continue
        a = _pad(qa[span])
        s = np.ones((k // 128, a.shape[0]), np.float32)
        s[:, :span.stop - span.start] = sa[:, span]
        if layout == oracle.FWD:
            b, t = qb[e * n:(e + 1) * n], sb[e * n // 128:(e + 1) * n // 128]
        else:
            b, t = qb[:, e * k:(e + 1) * k], sb[:, e * k // 128:(e + 1) * k // 128]
        d = oracle.gemm(layout, a, s, np.ascontiguousarray(b), np.ascontiguousarray(t), a_fmt=fmt)
        out[span] = d[:span.stop - span.start]
    return out


@pytest.mark.parametrize("counts", COUNTS, ids=str)
@pytest.mark.parametrize("layout", [fb.FWD, fb.DGRAD])
@pytest.mark.parametrize("n,k", [(256, 384), (640, 128)])
@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("block_n", ["auto", "128", "256"])
def test_row_products(counts, layout, n, k, out_dtype, block_n, monkeypatch):
    """Every number of rows through the kernel that the library takes and through the wide-tile ones."""
    require_cuda()
    if block_n == "256" and n % 256:
        pytest.skip("N not a multiple of 256")
    if block_n != "auto":
        monkeypatch.setenv("FP8BLK_GEMM_BLOCK_N", block_n)
    counts = COUNTS[counts]
    rows = sum(counts)
    rng = np.random.default_rng(rows + n)
    x = workloads.activation_with_outliers(rng, rows, k, frac=0.01)
    qa, sa = _rowwise_ref(x, False)
    # FWD: W [groups, n, k];  DGRAD: W [groups, k (out), n (in)], its transpose is the operand
    (qb, sb), (qbT, sbT) = _weights(len(counts), n if layout == fb.FWD else k, k if layout == fb.FWD else n, 3)
    if layout == fb.DGRAD:
        qb, sb = qbT, sbT
    d = fb.fp8blk_gemm_grouped(layout, _f8(qa), _dev(sa), _f8(qb), _dev(sb), _offsets(counts), out_dtype=out_dtype)
    assert fb.fp8blk_get_device_error() == 0
    assert d.dtype == out_dtype
    assert_gemm_close(f32(d), _rows_ref(layout, qa, sa, qb, sb, counts, n, k), f"{counts} layout {layout}")


@pytest.mark.parametrize("counts", ["edges", "few", "some", "single_rows"])
def test_input_gradient_of_e5m2_rows(counts):
    require_cuda()
    counts, n, k = COUNTS[counts], 256, 384
    dy = workloads.grad_output(np.random.default_rng(3), sum(counts), k)
    qa, sa = _rowwise_ref(dy, True)
    _, (qb, sb) = _weights(len(counts), k, n, 3)
    d = fb.fp8blk_gemm_grouped(fb.DGRAD, _f8(qa, True), _dev(sa), _f8(qb), _dev(sb), _offsets(counts))
    assert fb.fp8blk_get_device_error() == 0
    assert_gemm_close(f32(d), _rows_ref(fb.DGRAD, qa, sa, qb, sb, counts, n, k, oracle.E5M2), str(counts))


@pytest.mark.parametrize("block_n,counts", [("128", [70, 0, 129, 3]), ("256", [70, 0, 129, 3]), ("0", [3, 0, 7, 1, 2]),
                                            ("0", [3, 0, 40, 1, 2]), ("0", [3, 0, 70, 100, 2])])
def test_rows_outside_every_group_and_the_row_pitch_stay(block_n, counts, monkeypatch):
    require_cuda()
    monkeypatch.setenv("FP8BLK_GEMM_BLOCK_N", block_n)
    start, n, k = 6, 256, 256
    rows = start + sum(counts) + 5
    x = workloads.activation(np.random.default_rng(8), rows, k)
    qa, sa = _rowwise_ref(x, False)
    (qb, sb), _ = _weights(len(counts), n, k, 4)
    wide = torch.full((rows, n + 32), 7.0, dtype=torch.bfloat16, device="cuda")
    fb.fp8blk_gemm_grouped(fb.FWD, _f8(qa), _dev(sa), _f8(qb), _dev(sb), _offsets(counts, start), d=wide[:, :n])
    assert fb.fp8blk_get_device_error() == 0
    stop = start + sum(counts)
    ref = _rows_ref(fb.FWD, qa, sa, qb, sb, counts, n, k, start=start)
    assert_gemm_close(f32(wide[start:stop, :n]), ref[start:stop], "rows of the groups")
    for part in (wide[:start], wide[stop:], wide[:, n:]):
        assert bool((part == 7.0).all())


def _wgrad_ref(dy, x, counts, e5m2):
    out = np.zeros((len(counts), dy.shape[1], x.shape[1]))
    for e, span in enumerate(_spans(counts)):
        if span.stop > span.start:
            qa, sa = oracle.quantize_act_colwise_t(_pad(dy[span]), oracle.E5M2 if e5m2 else oracle.E4M3)
            qb, sb = oracle.quantize_act_colwise_t(_pad(x[span]))
            out[e] = oracle.gemm(oracle.WGRAD, qa, sa, qb, sb, a_fmt=oracle.E5M2 if e5m2 else oracle.E4M3)
    return out


@pytest.mark.parametrize("counts", ["one_row", "edges", "uneven"])
@pytest.mark.parametrize("n_out,n_in", [(128, 384), (384, 256)])
@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("e5m2", [False, True])
def test_weight_gradient(counts, n_out, n_in, out_dtype, e5m2):
    """Each group's own sum, zeros for a group without rows; the operands from the ragged quantiser."""
    require_cuda()
    counts = COUNTS[counts]
    rng = np.random.default_rng(sum(counts) + n_out)
    dy = workloads.grad_output(rng, sum(counts), n_out)
    x = workloads.swiglu_like(rng, sum(counts), n_in)
    off = _offsets(counts)
    _, _, qa, sa = fb.fp8blk_quantize_act_1x128_grouped(to_dev(dy), off, fb.COLWISE_T | (fb.E5M2 if e5m2 else 0))
    _, _, qb, sb = fb.fp8blk_quantize_act_1x128_grouped(to_dev(x), off, fb.COLWISE_T)
    d = fb.fp8blk_gemm_grouped(fb.WGRAD, qa, sa, qb, sb, off, out_dtype=out_dtype)
    assert fb.fp8blk_get_device_error() == 0
    ref = _wgrad_ref(dy, x, counts, e5m2)
    for e, c in enumerate(counts):
        if c == 0:
            assert bool((d[e] == 0).all()), f"group {e} has no rows"
        else:
            assert_gemm_close(f32(d[e]), ref[e], f"group {e}")


def test_layer_forward_and_backward_with_no_rows():
    require_cuda()
    g, n, k = 3, 256, 128
    (qw, sw), (qwT, swT) = _weights(g, n, k, 6)
    off = torch.zeros(g + 1, dtype=torch.int32, device="cuda")
    x = torch.empty((0, k), dtype=torch.bfloat16, device="cuda")
    dy = torch.empty((0, n), dtype=torch.bfloat16, device="cuda")
    y = fb.grouped_linear_forward(x, _f8(qw), _dev(sw), off)
    dx, dw = fb.grouped_linear_backward(x, dy, _f8(qwT), _dev(swT), off)
    assert fb.fp8blk_get_device_error() == 0
    assert y.shape == (0, n) and dx.shape == (0, k)
    assert dw.shape == (g, n, k) and bool((dw == 0).all())


def test_layer_in_a_captured_graph_follows_new_offsets():
    """One graph of forward and backward, replayed with other rows and other groups; on a side stream."""
    require_cuda()
    g, n, k, rows = 6, 256, 384, 700
    (qw, sw), (qwT, swT) = _weights(g, n, k, 9)
    QW, SW, QWT, SWT = _f8(qw), _dev(sw), _f8(qwT), _dev(swT)
    X = torch.zeros((rows, k), dtype=torch.bfloat16, device="cuda")
    DY = torch.zeros((rows, n), dtype=torch.bfloat16, device="cuda")
    off = torch.zeros(g + 1, dtype=torch.int32, device="cuda")
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(stream):
        fb.grouped_linear_forward(X, QW, SW, off)
        fb.grouped_linear_backward(X, DY, QWT, SWT, off)
        stream.synchronize()
        with torch.cuda.graph(graph, stream=stream):
            Y = fb.grouped_linear_forward(X, QW, SW, off)
            DX, DW = fb.grouped_linear_backward(X, DY, QWT, SWT, off)
    torch.cuda.synchronize()
    for counts in ([700, 0, 0, 0, 0, 0], [1, 130, 0, 256, 64, 200]):
        rng = np.random.default_rng(counts[1] + 2)
        x, dy = workloads.activation(rng, rows, k), workloads.grad_output(rng, rows, n)
        X.copy_(to_dev(x))
        DY.copy_(to_dev(dy))
        off.copy_(_offsets(counts))
        graph.replay()
        assert fb.fp8blk_get_device_error() == 0
        used = sum(counts)
        qx, sx = _rowwise_ref(x, False)
        qd, sd = _rowwise_ref(dy, False)
        assert_gemm_close(f32(Y[:used]), _rows_ref(fb.FWD, qx, sx, qw, sw, counts, n, k)[:used], "forward")
        assert_gemm_close(f32(DX[:used]), _rows_ref(fb.DGRAD, qd, sd, qwT, swT, counts, k, n)[:used], "dx")
        ref = _wgrad_ref(dy, x, counts, False)
        for e, c in enumerate(counts):
            if c:
                assert_gemm_close(f32(DW[e]), ref[e], f"dw of group {e}")
            else:
                assert bool((DW[e] == 0).all())
    del graph


def test_offsets_that_break_the_rules_write_nothing_out_of_range():
    """Decreasing, negative and too large offsets: ranges are clamped, buffers around the outputs stay."""
    require_cuda()
    rows, n, k, guard = 150, 128, 256, 64
    off = torch.tensor([-5, 90, 20, 100000, 3, 160], dtype=torch.int32, device="cuda")
    g = off.numel() - 1
    (qw, sw), _ = _weights(g, n, k, 2)
    x = to_dev(workloads.activation(np.random.default_rng(1), rows, k))
    padded = fb.fp8blk_grouped_padded_rows(rows, g)
    qT = torch.full((k + 1, padded), 0x55, dtype=torch.uint8, device="cuda")
    sT = torch.full((padded // 128 + 1, k), -7.0, device="cuda")
    q, s, _, _ = fb.fp8blk_quantize_act_1x128_grouped(x, off, fb.BOTH, None, None, qT[:k].view(torch.float8_e4m3fn),
                                                      sT[:-1])
    y = torch.full((rows + guard, n), 7.0, dtype=torch.bfloat16, device="cuda")
    fb.fp8blk_gemm_grouped(fb.FWD, q, s, _f8(qw), _dev(sw), off, d=y[:rows])
    dw = torch.full((g + 1, k, k), 7.0, dtype=torch.bfloat16, device="cuda")
    f8T = qT[:k].view(torch.float8_e4m3fn)
    fb.fp8blk_gemm_grouped(fb.WGRAD, f8T, sT[:-1], f8T, sT[:-1], off, d=dw[:g])
    assert fb.fp8blk_get_device_error() == 0
    assert bool((y[rows:] == 7.0).all()) and bool((dw[g] == 7.0).all())
    assert bool((qT[k] == 0x55).all()) and bool((sT[-1] == -7.0).all())


@pytest.mark.parametrize("layout,counts", [(fb.FWD, [200, 56]), (fb.FWD, [20, 6]), (fb.WGRAD, [200, 56])])
def test_stalled_grouped_gemm_reports_timeout_and_recovers(layout, counts, monkeypatch):
    """As tests/test_gpu_timeout.py: a wait that nothing completes ends by its limit."""
    require_cuda()
    n, k = 256, 256
    rng = np.random.default_rng(3)
    x, dy = workloads.activation(rng, sum(counts), k), workloads.grad_output(rng, sum(counts), n)
    off = _offsets(counts)
    (qw, sw), _ = _weights(2, n, k, 5)
    if layout == fb.FWD:
        a, sa, _, _ = fb.fp8blk_quantize_act_1x128_grouped(to_dev(x), off)
        b, sb = _f8(qw), _dev(sw)
    else:
        _, _, a, sa = fb.fp8blk_quantize_act_1x128_grouped(to_dev(dy), off, fb.COLWISE_T)
        _, _, b, sb = fb.fp8blk_quantize_act_1x128_grouped(to_dev(x), off, fb.COLWISE_T)
    assert fb.fp8blk_get_device_error() == 0
    monkeypatch.setenv("FP8BLK_TEST_INJECT_STALL", "1")
    monkeypatch.setenv("FP8BLK_WAIT_TIMEOUT_MS", "200")
    fb.fp8blk_gemm_grouped(layout, a, sa, b, sb, off)
    assert fb.fp8blk_get_device_error() == 6
    assert fb.fp8blk_get_device_error() == 0
    monkeypatch.delenv("FP8BLK_TEST_INJECT_STALL")
    d = fb.fp8blk_gemm_grouped(layout, a, sa, b, sb, off)
    assert fb.fp8blk_get_device_error() == 0
    if layout == fb.FWD:
        qx, sx = _rowwise_ref(x, False)
        assert_gemm_close(f32(d), _rows_ref(fb.FWD, qx, sx, qw, sw, counts, n, k), "after timeout")
    else:
        ref = _wgrad_ref(dy, x, counts, False)
        for e in range(2):
            assert_gemm_close(f32(d[e]), ref[e], "after timeout")


def test_layer_on_a_stream_that_is_passed_in():
    """A stream other than the current one, as an object and as a handle, with allocations after the call
    that would take the memory of the codes if it were given out again."""
    require_cuda()
    g, n, k, counts = 3, 256, 384, [200, 0, 129]
    (qw, sw), (qwT, swT) = _weights(g, n, k, 9)
    rng = np.random.default_rng(4)
    X = to_dev(workloads.activation(rng, sum(counts), k))
    DY = to_dev(workloads.grad_output(rng, sum(counts), n))
    QW, SW, QWT, SWT, off = _f8(qw), _dev(sw), _f8(qwT), _dev(swT), _offsets(counts)
    want = (fb.grouped_linear_forward(X, QW, SW, off), *fb.grouped_linear_backward(X, DY, QWT, SWT, off))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream):
        with torch.cuda.stream(side):
            torch.cuda._sleep(2_000_000)                   # the calls below are queued behind it
        y = fb.grouped_linear_forward(X, QW, SW, off, stream=stream)
        dx, dw = fb.grouped_linear_backward(X, DY, QWT, SWT, off, stream=stream)
        junk = [torch.full((1 << 20,), 0x7F, dtype=torch.uint8, device="cuda") for _ in range(8)]
        torch.cuda.synchronize()
        for a, b in zip((y, dx, dw), want):
            assert torch.equal(a, b)
        del junk
    assert fb.fp8blk_get_device_error() == 0


def test_forward_refuses_what_does_not_match():
    require_cuda()
    x = torch.zeros((5, 256), dtype=torch.bfloat16, device="cuda")
    off = _offsets([2, 3])
    q = torch.zeros((256, 256), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    s = torch.ones((2, 2), device="cuda")
    for bad in (lambda: fb.grouped_linear_forward(x[:, :128], q, s, off), lambda: fb.grouped_linear_forward(x, q, s[:1], off),
                lambda: fb.grouped_linear_forward(x, q.view(torch.float8_e5m2), s, off),
                lambda: fb.grouped_linear_forward(x, q.t(), s, off), lambda: fb.grouped_linear_forward(x, q, s.t(), off[:2])):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(fb.Fp8BlkError):                  # 64 output columns a group: not a multiple of 128
        fb.grouped_linear_forward(x, q[:128].contiguous(), s[:1].contiguous(), off)


@pytest.mark.parametrize("counts", COUNTS, ids=str)
@pytest.mark.parametrize("n,k", [(128, 384), (384, 1536)])
@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
def test_quantised_on_the_way_is_the_two_calls(counts, n, k, out_dtype):
    """Bit for bit the result of the quantiser and the product; x and d with a row pitch, rows outside every group."""
    require_cuda()
    counts, start = COUNTS[counts], 3
    rows = start + sum(counts) + 2
    (qw, sw), _ = _weights(len(counts), n, k, 3)
    QW, SW, off = _f8(qw), _dev(sw), _offsets(counts, start)
    x = to_dev(workloads.activation_with_outliers(np.random.default_rng(rows), rows, k + 8, frac=0.01))[:, :k]
    want = torch.full((rows, n), 7.0, dtype=out_dtype, device="cuda")
    q, s, _, _ = fb.fp8blk_quantize_act_1x128_grouped(x, off)
    fb.fp8blk_gemm_grouped(fb.FWD, q, s, QW, SW, off, d=want)
    size = fb.fp8blk_linear_grouped_workspace_bytes(len(counts), rows, k)
    work = torch.full((size + 64,), 0x55, dtype=torch.uint8, device="cuda")
    wide = torch.full((rows, n + 32), 7.0, dtype=out_dtype, device="cuda")
    got = fb.fp8blk_linear_grouped(x, QW, SW, off, d=wide[:, :n], workspace=work[:size])
    assert fb.fp8blk_get_device_error() == 0
    assert torch.equal(got, want)
    assert bool((work[size:] == 0x55).all()) and bool((wide[:, n:] == 7.0).all())


def test_stalled_product_that_quantises_reports_timeout_and_recovers(monkeypatch):
    require_cuda()
    counts, n, k = [7, 0, 3], 256, 384
    (qw, sw), _ = _weights(3, n, k, 3)
    x, QW, SW, off = to_dev(workloads.activation(np.random.default_rng(1), 10, k)), _f8(qw), _dev(sw), _offsets(counts)
    want = fb.fp8blk_linear_grouped(x, QW, SW, off)
    assert fb.fp8blk_get_device_error() == 0
    monkeypatch.setenv("FP8BLK_TEST_INJECT_STALL", "1")
    monkeypatch.setenv("FP8BLK_WAIT_TIMEOUT_MS", "200")
    fb.fp8blk_linear_grouped(x, QW, SW, off)
    assert fb.fp8blk_get_device_error() == 6
    monkeypatch.delenv("FP8BLK_TEST_INJECT_STALL")
    assert torch.equal(fb.fp8blk_linear_grouped(x, QW, SW, off), want)
    assert fb.fp8blk_get_device_error() == 0
