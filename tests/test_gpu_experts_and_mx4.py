"""The grouped products and the 4-bit products as a mixture-of-experts block uses them, forward and backward.

Tokens are routed, sorted by expert and taken through the experts' layer with
FP8 blockwise operands; a layer that all tokens share runs in 4 bits.  The
results are compared with the block's formula in 64 bits on the values that the
quantisers' codes stand for; gradients also with differences of the layer's own
outputs, on integers that every code format holds exactly (so that the layer is
exactly linear and the difference quotient has no error of its own)."""
import numpy as np
import pytest
import torch

import fp8_blockwise_scaled_b200 as fb
import oracle
import workloads
from tests import mx4_reference as ref
from tests.gpu_helpers import assert_gemm_close, f32, require_cuda, to_dev, u8

pytestmark = pytest.mark.gpu

TOKENS, CHOICES, EXPERTS, K, N = 150, 2, 8, 384, 256


def _route(seed, skip):
    """Expert of each (token, choice) and the order that sorts them; experts in `skip` get nothing."""
    rng = np.random.default_rng(seed)
    allowed = [e for e in range(EXPERTS) if e not in skip]
    expert = np.stack([rng.choice(allowed, CHOICES, replace=False) for _ in range(TOKENS)]).ravel()
    order = np.argsort(expert, kind="stable")
    counts = np.bincount(expert, minlength=EXPERTS)
    return order, counts, np.concatenate([[0], np.cumsum(counts)])


def _values(q, s, block):
    """64-bit values of E4M3 codes with scales [groups, rows] (128 along the columns)."""
    v = oracle.e4m3_decode(q)
    return v * np.repeat(s.astype(np.float64).T, block, axis=1)


def _weight_values(q, s):
    return oracle.e4m3_decode(q) * np.repeat(np.repeat(s.astype(np.float64), 128, 0), 128, 1)


class Block:
    """y[t] = sum over the token's choices of x[t] . W[e]^T, plus x . V^T with V shared and in 4 bits."""

    def __init__(self, seed, fmt):
        rng = np.random.default_rng(seed)
        self.fmt = fmt
        self.w, self.v = workloads.weight(rng, EXPERTS * N, K), workloads.weight(rng, N, K)
        self.x, self.dy = workloads.activation(rng, TOKENS, K), workloads.grad_output(rng, TOKENS, N)
        self.qw, self.sw, self.qwT, self.swT = fb.fp8blk_quantize_weight_128x128_both(to_dev(self.w))
        self.scale = {n: self._tensor_scale(a) for n, a in (("x", self.x), ("v", self.v), ("dy", self.dy))}
        self.qv, self.sv, self.qvT, self.svT = fb.fp8blk_quantize_mx4(to_dev(self.v), fmt, fb.BOTH, self.scale["v"])

    def _tensor_scale(self, bits):
        if self.fmt == fb.MXFP4:
            return None
        return torch.tensor([np.abs(workloads.bf16_to_f32(bits)).max() / 2688], dtype=torch.float32, device="cuda")

    def run(self, order, offsets, x, dy):
        """Forward and backward on the current stream: the experts' and the shared layer's parts of y and of dx
        (the experts' by sorted row), dW, dV, and the sums y and dx."""
        token = order // CHOICES
        xs, dys = x[token], dy[token]
        ys = fb.grouped_linear_forward(xs, self.qw, self.sw, offsets)
        shared = fb.mx4_linear_forward(x, self.qv, self.sv, self.fmt, self.scale["x"], self.scale["v"])
        y = shared.float().index_add(0, token, ys.float())
        dxs, dw = fb.grouped_linear_backward(xs, dys, self.qwT, self.swT, offsets, out_dtype=torch.float32)
        dx, dv = fb.mx4_linear_backward(x, dy, self.qvT, self.svT, self.fmt, self.scale["x"], self.scale["dy"],
                                        self.scale["v"], out_dtype=torch.float32)
        return ys, shared, dxs, dx, dw, dv, y, dx.float().index_add(0, token, dxs.float())

    def exact(self, order, offsets):
        """The same in 64 bits on the quantised values, without the sums."""
        token = order // CHOICES
        f = "mxfp4" if self.fmt == fb.MXFP4 else "nvfp4"

        def pad(a):
            want = max(128, -(-a.shape[0] // 128) * 128)
            return np.concatenate([a, np.zeros((want - a.shape[0], a.shape[1]), a.dtype)])

        def rows(bits):
            q, s = oracle.quantize_act_rowwise(pad(bits))
            return _values(q, s, 128)[:bits.shape[0]]

        def columns(bits):                       # groups of 128 tokens: values of the transpose, transposed back
            q, s = oracle.quantize_act_colwise_t(pad(bits))
            return _values(q, s, 128).T[:bits.shape[0]]

        def four(bits, g, along_rows=False):
            a = workloads.bf16_to_f32(bits).astype(np.float64)
            a = ref.pad_rows(a).T.copy() if along_rows else a
            g = 1.0 if g is None else float(g.item())
            v = ref.values(*ref.quantize(a, f, g), f) * g
            return v.T[:bits.shape[0]] if along_rows else v

        w = _weight_values(*oracle.quantize_weight(self.w)).reshape(EXPERTS, N, K)
        shared = four(self.x, self.scale["x"]) @ four(self.v, self.scale["v"]).T
        dx = four(self.dy, self.scale["dy"]) @ four(self.v, self.scale["v"], along_rows=True)
        dv = four(self.dy, self.scale["dy"], along_rows=True).T @ four(self.x, self.scale["x"], along_rows=True)
        dw = np.zeros((EXPERTS, N, K))
        xs, dys = self.x[token], self.dy[token]
        ys, dxs = np.zeros((len(order), N)), np.zeros((len(order), K))
        for e in range(EXPERTS):
            span = slice(offsets[e], offsets[e + 1])
            if span.stop == span.start:
                continue
            ys[span], dxs[span] = rows(xs[span]) @ w[e].T, rows(dys[span]) @ w[e]
            dw[e] = columns(dys[span]).T @ columns(xs[span])
        return ys, shared, dxs, dx, dw, dv


@pytest.mark.parametrize("fmt", [fb.MXFP4, fb.NVFP4])
@pytest.mark.parametrize("skip", [(), (0, 3, 7)])
def test_block_forward_and_backward(fmt, skip):
    require_cuda()
    block = Block(1, fmt)
    order, counts, ends = _route(2, skip)
    off = torch.from_numpy(ends.astype(np.int32)).cuda()
    got = block.run(torch.from_numpy(order).cuda(), off, to_dev(block.x), to_dev(block.dy))
    assert fb.fp8blk_get_device_error() == 0
    want = block.exact(order, ends)
    for g, w, what in zip(got, want, ("experts' y", "shared y", "experts' dx", "shared dx", "dW", "dV")):
        g = f32(g)
        if what == "dW":
            assert np.array_equal(g[counts == 0], np.zeros_like(g[counts == 0]))
            g, w = g[counts > 0].reshape(-1, K), w[counts > 0].reshape(-1, K)
        assert_gemm_close(g, w, what)


def _run_all(block, order, off, x, dy, stream):
    with torch.cuda.stream(stream):
        return block.run(order, off, x, dy)


def test_two_blocks_on_two_streams_at_once():
    """Interleaved launches of two blocks share the library but no memory: each gives what it gives alone."""
    require_cuda()
    blocks = [Block(1, fb.MXFP4), Block(5, fb.NVFP4)]
    args = []
    for i, b in enumerate(blocks):
        order, _, ends = _route(7 + i, (1,))
        args.append((torch.from_numpy(order).cuda(), torch.from_numpy(ends.astype(np.int32)).cuda(), to_dev(b.x), to_dev(b.dy)))
    alone = [b.run(*a) for b, a in zip(blocks, args)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    both = []
    for _ in range(3):
        both = [_run_all(b, *a, s) for b, a, s in zip(blocks, args, streams)]
    torch.cuda.synchronize()
    assert fb.fp8blk_get_device_error() == 0
    for i in range(2):
        for a, b in zip(both[i][:6], alone[i][:6]):     # index_add's order of additions may change the sums
            assert torch.equal(a, b)


def test_block_with_dependent_launch_is_bitwise_equal(monkeypatch):
    """FP8BLK_PDL=1 changes only how the launches overlap."""
    require_cuda()
    block = Block(3, fb.NVFP4)
    order, _, ends = _route(4, (2,))
    token = torch.from_numpy(order // CHOICES).cuda()
    off = torch.from_numpy(ends.astype(np.int32)).cuda()
    x, dy = to_dev(block.x), to_dev(block.dy)

    def outputs():
        out = [fb.grouped_linear_forward(x[token], block.qw, block.sw, off),
               *fb.grouped_linear_backward(x[token], dy[token], block.qwT, block.swT, off),
               fb.mx4_linear_forward(x, block.qv, block.sv, block.fmt, block.scale["x"], block.scale["v"]),
               *fb.mx4_linear_backward(x, dy, block.qvT, block.svT, block.fmt, block.scale["x"], block.scale["dy"],
                                       block.scale["v"])]
        tiny = off.clamp(max=9)
        out.append(fb.grouped_linear_forward(x[:9], block.qw, block.sw, tiny))
        out.append(fb.mx4_linear_forward(x[:9], block.qv, block.sv, block.fmt, block.scale["x"], block.scale["v"]))
        q, s, _, _ = fb.fp8blk_quantize_mx4(x, block.fmt)
        out.append(fb.fp8blk_dequantize_mx4(q, s, block.fmt))
        return out

    monkeypatch.delenv("FP8BLK_PDL", raising=False)
    plain = outputs()
    monkeypatch.setenv("FP8BLK_PDL", "1")
    for _ in range(3):
        for a, b in zip(outputs(), plain):
            assert torch.equal(a, b)
    assert fb.fp8blk_get_device_error() == 0


def _bits(a):
    return to_dev(workloads.f32_to_bf16(a.astype(np.float32)))


def test_grouped_gradients_against_differences():
    """Integers up to 7 with a 7 in every group of 128 (scale 1/64): E4M3 holds them all, Y is exactly linear."""
    require_cuda()
    rng = np.random.default_rng(6)
    counts, n, k = [130, 0, 5], 128, 256
    groups, rows = len(counts), sum(counts)
    off = torch.tensor(np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)).cuda()

    def ints(r, c):
        a = rng.integers(-5, 6, size=(r, c))
        a[:, ::128] = 7                          # a 7 in every row group ...
        a[::128] = 7                             # ... every block of rows ...
        return a

    x, w, g = ints(rows, k), ints(groups * n, k), ints(rows, n)
    x[130], g[130] = 7, 7                        # ... and every token group
    dx_step, dw_step = rng.integers(-2, 3, size=x.shape), rng.integers(-2, 3, size=w.shape)
    dx_step[np.abs(x) == 7] = 0
    dw_step[np.abs(w) == 7] = 0

    def loss(xv, wv):
        q, s = fb.fp8blk_quantize_weight_128x128(_bits(wv))
        y = fb.fp8blk_linear_grouped(_bits(xv), q, s, off, out_dtype=torch.float32)
        return float((y.double().cpu().numpy() * g).sum())

    _, _, qwT, swT = fb.fp8blk_quantize_weight_128x128_both(_bits(w))
    gq, gs, gqT, gsT = fb.fp8blk_quantize_act_1x128_grouped(_bits(g), off, fb.BOTH)
    _, _, xqT, xsT = fb.fp8blk_quantize_act_1x128_grouped(_bits(x), off, fb.COLWISE_T)
    dx = fb.fp8blk_gemm_grouped(fb.DGRAD, gq, gs, qwT, swT, off, out_dtype=torch.float32).double().cpu().numpy()
    dw = fb.fp8blk_gemm_grouped(fb.WGRAD, gqT, gsT, xqT, xsT, off, out_dtype=torch.float32).double().cpu().numpy()
    assert fb.fp8blk_get_device_error() == 0
    by_x = (loss(x + dx_step, w) - loss(x - dx_step, w)) / 2
    by_w = (loss(x, w + dw_step) - loss(x, w - dw_step)) / 2
    # Scales 1/64 are fl32(7/448) exactly and every partial sum is an integer / 4096 below 2^24: no rounding at all.
    assert (dx * dx_step).sum() == by_x
    assert (dw.reshape(w.shape) * dw_step).sum() == by_w


@pytest.mark.parametrize("fmt", [fb.MXFP4, fb.NVFP4])
def test_mx4_gradients_against_differences(fmt):
    """Values of the grid with a 6 in every block (scale 1): 4 bits hold them all, Y is exactly linear."""
    require_cuda()
    rng = np.random.default_rng(8)
    m, n, k = 70, 96, 160

    def grid(r, c):
        a = rng.choice([-3, -2, -1, 1, 2, 3], size=(r, c))
        a[:, ::16] = 6
        a[::16] = 6
        return a

    x, w, g = grid(m, k), grid(n, k), grid(m, n)
    x[64], g[64] = 6, 6
    dx_step, dw_step = rng.integers(-1, 2, size=x.shape), rng.integers(-1, 2, size=w.shape)
    dx_step[x == 6] = 0
    dw_step[w == 6] = 0

    def loss(xv, wv):
        q, s, _, _ = fb.fp8blk_quantize_mx4(_bits(wv), fmt)
        y = fb.fp8blk_linear_mx4(_bits(xv), q, s, fmt, out_dtype=torch.float32)
        return float((y.double().cpu().numpy() * g).sum())

    _, _, qwT, swT = fb.fp8blk_quantize_mx4(_bits(w), fmt, fb.BOTH)
    gq, gs, gqT, gsT = fb.fp8blk_quantize_mx4(_bits(g), fmt, fb.BOTH)
    dx = fb.fp8blk_gemm_mx4(gq, gs, qwT, swT, fmt, out_dtype=torch.float32).double().cpu().numpy()
    dw = fb.mx4_linear_wgrad(_bits(x), _bits(g), fmt, out_dtype=torch.float32).double().cpu().numpy()
    assert fb.fp8blk_get_device_error() == 0
    assert (dx * dx_step).sum() == (loss(x + dx_step, w) - loss(x - dx_step, w)) / 2
    assert (dw * dw_step).sum() == (loss(x, w + dw_step) - loss(x, w - dw_step)) / 2


def test_tensors_that_alias_their_rows_are_refused():
    """An expanded row (stride 0) is no matrix of that many rows."""
    require_cuda()
    off = torch.tensor([0, 5], dtype=torch.int32, device="cuda")
    x = torch.zeros((1, 256), dtype=torch.bfloat16, device="cuda").expand(5, 256)
    q, s = fb.fp8blk_quantize_weight_128x128(torch.zeros((128, 256), dtype=torch.bfloat16, device="cuda"))
    q4, s4, _, _ = fb.fp8blk_quantize_mx4(torch.zeros((128, 256), dtype=torch.bfloat16, device="cuda"), fb.MXFP4)
    d = torch.zeros((1, 128), dtype=torch.bfloat16, device="cuda").expand(5, 128)
    real = torch.zeros((5, 256), dtype=torch.bfloat16, device="cuda")
    for call in (lambda: fb.fp8blk_quantize_act_1x128_grouped(x, off), lambda: fb.fp8blk_linear_grouped(x, q, s, off),
                 lambda: fb.fp8blk_linear_grouped(real, q, s, off, d=d), lambda: fb.fp8blk_quantize_mx4(x, fb.MXFP4),
                 lambda: fb.fp8blk_linear_mx4(x, q4, s4, fb.MXFP4), lambda: fb.fp8blk_linear_mx4(real, q4, s4, fb.MXFP4, d=d)):
        with pytest.raises(fb.Fp8BlkError) as err:
            call()
        assert err.value.status == 1


def test_block_codes_match_the_quantisers_used_apart():
    """The block's expert codes are those of the 128-row quantiser where a group is whole blocks."""
    require_cuda()
    x = workloads.activation(np.random.default_rng(1), 256, K)
    off = torch.tensor([0, 128, 128, 256], dtype=torch.int32, device="cuda")
    a = fb.fp8blk_quantize_act_1x128(to_dev(x), fb.BOTH)
    b = fb.fp8blk_quantize_act_1x128_grouped(to_dev(x), off, fb.BOTH)
    for s, t in zip(a, b):
        s, t = u8(s), u8(t)
        assert np.array_equal(s, t[tuple(slice(0, n) for n in s.shape)])


@pytest.mark.parametrize("name", ["grouped_forward", "grouped_few", "grouped_backward", "mx4_forward", "mx4_few",
                                  "mx4_wgrad", "mx4_backward"])
@pytest.mark.parametrize("as_handle", [False, True])
def test_stream_argument_allocates_from_that_stream(name, as_handle):
    """With `stream` given, nothing that the call allocates may be memory that earlier work of the current
    stream still writes: blocks of every size, freed behind a long queue of writes of NaN, are not handed to it."""
    require_cuda()
    block = Block(3, fb.NVFP4)
    order, _, ends = _route(4, (2,))
    token = torch.from_numpy(order // CHOICES).cuda()
    off = torch.from_numpy(ends.astype(np.int32)).cuda()
    x, dy = to_dev(block.x), to_dev(block.dy)
    xs, dys, few = x[token].contiguous(), dy[token].contiguous(), off.clamp(max=9)
    sc = block.scale
    call = {
        "grouped_forward": lambda **k: fb.grouped_linear_forward(xs, block.qw, block.sw, off, **k),
        "grouped_few": lambda **k: fb.grouped_linear_forward(xs[:9], block.qw, block.sw, few, **k),
        "grouped_backward": lambda **k: fb.grouped_linear_backward(xs, dys, block.qwT, block.swT, off, **k),
        "mx4_forward": lambda **k: fb.mx4_linear_forward(x, block.qv, block.sv, block.fmt, sc["x"], sc["v"], **k),
        "mx4_few": lambda **k: fb.mx4_linear_forward(x[:9], block.qv, block.sv, block.fmt, sc["x"], sc["v"], **k),
        "mx4_wgrad": lambda **k: fb.mx4_linear_wgrad(x, dy, block.fmt, sc["x"], sc["dy"], **k),
        "mx4_backward": lambda **k: fb.mx4_linear_backward(x, dy, block.qvT, block.svT, block.fmt, sc["x"], sc["dy"],
                                                           sc["v"], **k),
    }[name]
    want = call()
    want = want if isinstance(want, tuple) else (want,)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    blocks = [torch.empty(1 << b, dtype=torch.uint8, device="cuda") for b in range(9, 24) for _ in range(3)]
    for _ in range(40):
        for b in blocks:
            b.fill_(255)
    taken = [(b.data_ptr(), b.data_ptr() + b.numel()) for b in blocks]
    del blocks, b
    got = call(stream=side.cuda_stream if as_handle else side)
    got = got if isinstance(got, tuple) else (got,)
    torch.cuda.synchronize()
    assert fb.fp8blk_get_device_error() == 0
    for g, w in zip(got, want):
        assert torch.equal(g, w)
        assert not any(lo <= g.data_ptr() < hi for lo, hi in taken)


def test_stream_argument_inside_a_capture():
    """A side stream that joins a capture, given as an argument: the graph replays with new inputs."""
    require_cuda()
    block = Block(3, fb.MXFP4)
    order, _, ends = _route(4, (2,))
    token = torch.from_numpy(order // CHOICES).cuda()
    off = torch.from_numpy(ends.astype(np.int32)).cuda()
    x, dy = to_dev(block.x)[token].contiguous(), to_dev(block.dy)[token].contiguous()
    xf = to_dev(block.x)

    def run(**k):
        return (fb.grouped_linear_forward(x, block.qw, block.sw, off, **k),
                *fb.grouped_linear_backward(x, dy, block.qwT, block.swT, off, **k),
                fb.mx4_linear_forward(xf, block.qv, block.sv, block.fmt, **k),
                fb.mx4_linear_wgrad(x, dy, block.fmt, **k))

    run()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        out = run(stream=side)
        torch.cuda.current_stream().wait_stream(side)
    for scale in (1.0, -0.5):
        x.mul_(scale)
        dy.mul_(scale)
        xf.mul_(scale)
        graph.replay()
        torch.cuda.synchronize()
        for got, want in zip(out, run()):
            assert torch.equal(got, want)
    assert fb.fp8blk_get_device_error() == 0
