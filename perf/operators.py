"""The block-scaled products over experts and in 4 bits: inputs, plain forms and definitions of what is timed.

Each case is one pass of an operator as a program calls it.

  experts_forward    tokens sorted by expert, y = x . w[e]^T with FP8 blockwise operands: the tokens are
                     quantised in 1x128 groups and multiplied with weights quantised ahead (128x128 blocks)
  experts_backward   dx and dw of the same layer: dy quantised along features and along each expert's
                     tokens, x along each expert's tokens, then the data- and weight-gradient products
  mx4_roundtrip      4-bit quantisation (one scale for 32 or 16 values) and the values back in bf16
  mx4_forward        y = x . w^T in 4 bits: x quantised in the call, w ahead
  mx4_wgrad          dw = dy^T . x in 4 bits: both quantised along the tokens in the call, fp32 result

Formats: "mxfp4" is E2M1 with one power-of-two scale (E8M0) for 32 values; "nvfp4" is E2M1 with one E4M3
scale for 16 values below one fp32 scale for the tensor.
"""
import math

import torch

own = False

HIDDEN, MLP_WIDTH, QKV_OUT = 1536, 8960, 2048    # the decoder layer's widths
EXPERT_WIDTH = MLP_WIDTH // 7                    # one expert's share of the MLP


def listed():
    return [
        # one token of a decoding step, routed to 8 of 64 experts: latency and the chosen experts' weights
        {"name": "experts_forward_one_token", "op": "experts_forward", "tokens": 8, "experts": 64, "k": HIDDEN,
         "n": 2 * EXPERT_WIDTH, "skew": 0.0, "idle": 56},
        # a decoding batch over all experts, a few tokens each, some idle
        {"name": "experts_forward_batch", "op": "experts_forward", "tokens": 509, "experts": 64, "k": HIDDEN,
         "n": 2 * EXPERT_WIDTH, "skew": 0.7, "idle": 5},
        # a prompt through the experts' second product, unevenly routed
        {"name": "experts_forward_prompt", "op": "experts_forward", "tokens": 16385, "experts": 64, "k": EXPERT_WIDTH,
         "n": HIDDEN, "skew": 0.5, "idle": 0},
        # training: few wide experts, many tokens
        {"name": "experts_forward_large", "op": "experts_forward", "tokens": 65536, "experts": 8, "k": HIDDEN,
         "n": MLP_WIDTH, "skew": 0.2, "idle": 0},
        # the smallest training step: about 60 tokens an expert, one expert without any
        {"name": "experts_backward_short", "op": "experts_backward", "tokens": 1003, "experts": 16, "k": HIDDEN,
         "n": 2 * EXPERT_WIDTH, "skew": 0.6, "idle": 1},
        # an ordinary training step
        {"name": "experts_backward_long", "op": "experts_backward", "tokens": 32768, "experts": 32, "k": HIDDEN,
         "n": 2 * EXPERT_WIDTH, "skew": 0.4, "idle": 0},
        # a short batch's activations
        {"name": "mx4_roundtrip_short", "op": "mx4_roundtrip", "rows": 77, "cols": HIDDEN, "format": "mxfp4",
         "both": False},
        # a training batch's activations along both directions
        {"name": "mx4_roundtrip_long", "op": "mx4_roundtrip", "rows": 16384, "cols": MLP_WIDTH, "format": "nvfp4",
         "both": True},
        # one decoding token through the MLP's second product
        {"name": "mx4_forward_one_token", "op": "mx4_forward", "m": 1, "k": MLP_WIDTH, "n": HIDDEN,
         "format": "nvfp4"},
        # a ragged prompt through the attention's input product
        {"name": "mx4_forward_odd", "op": "mx4_forward", "m": 333, "k": HIDDEN, "n": QKV_OUT, "format": "mxfp4"},
        # a training batch through the MLP's first product
        {"name": "mx4_forward_long", "op": "mx4_forward", "m": 16384, "k": HIDDEN, "n": 2 * MLP_WIDTH,
         "format": "nvfp4"},
        # that batch's weight gradient of the MLP's second product: a long sum, fp32 result
        {"name": "mx4_wgrad_long", "op": "mx4_wgrad", "tokens": 16384, "k": MLP_WIDTH, "n": HIDDEN,
         "format": "mxfp4"},
    ]


def draw(rng):
    def spread(low, high):
        return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))

    def width(low, high, step):
        return max(low, spread(low, high) // step * step)

    op = rng.choice(["experts_forward", "experts_backward", "mx4_roundtrip", "mx4_forward", "mx4_wgrad"])
    most = max(c["flops"] for c in (work(case) for case in listed() if case["op"] == op))
    while True:
        if op.startswith("experts"):
            tokens = spread(1, 65536) if op == "experts_forward" else spread(16, 32768)
            experts = spread(2, 128)
            case = {"op": op, "tokens": tokens, "experts": experts, "k": width(256, 4096, 128),
                    "n": width(256, MLP_WIDTH, 128), "skew": round(rng.uniform(0.0, 1.2), 2),
                    "idle": rng.randrange(experts // 2 + 1)}
            if case["experts"] * case["n"] * case["k"] > 1 << 29:
                continue
        elif op == "mx4_roundtrip":
            case = {"op": op, "rows": spread(1, 16384), "cols": width(64, MLP_WIDTH, 32),
                    "format": rng.choice(["mxfp4", "nvfp4"]), "both": rng.random() < 0.5}
        elif op == "mx4_forward":
            case = {"op": op, "m": spread(1, 16384), "k": width(64, MLP_WIDTH, 32), "n": width(64, 2 * MLP_WIDTH, 8),
                    "format": rng.choice(["mxfp4", "nvfp4"])}
        else:
            case = {"op": op, "tokens": spread(32, 16384), "k": width(64, MLP_WIDTH, 8), "n": width(64, 4096, 8),
                    "format": rng.choice(["mxfp4", "nvfp4"])}
        if work(case)["flops"] <= most:
            return case


def expert_counts(case):
    """Tokens of each expert: shares fall as rank^-skew over the experts that are not idle (largest remainders)."""
    active = max(1, case["experts"] - case["idle"])
    shares = [(i + 1.0) ** -case["skew"] for i in range(active)]
    total = sum(shares)
    exact_counts = [case["tokens"] * s / total for s in shares]
    counts = [int(c) for c in exact_counts]
    order = sorted(range(active), key=lambda i: (counts[i] - exact_counts[i], i))
    for i in order[:case["tokens"] - sum(counts)]:
        counts[i] += 1
    return counts + [0] * (case["experts"] - active)


def work(case):
    op = case["op"]
    if op == "mx4_roundtrip":
        rows, cols = case["rows"], case["cols"]
        ways = 2 if case["both"] else 1
        code = 0.5 + 1.0 / BLOCK[case["format"]]
        return {"bytes": int(rows * cols * (2 + ways * (2 + 2 * code))), "flops": 4 * ways * rows * cols}
    if op == "mx4_forward":
        m, n, k = case["m"], case["n"], case["k"]
        code = 0.5 + 1.0 / BLOCK[case["format"]]
        return {"bytes": int(2 * m * k + code * n * k + 2 * m * n), "flops": 2 * m * n * k}
    t, n, k = case["tokens"], case["n"], case["k"]
    if op == "mx4_wgrad":
        return {"bytes": 2 * t * (n + k) + 4 * n * k, "flops": 2 * t * n * k}
    weights = sum(c > 0 for c in expert_counts(case)) * n * k
    if op == "experts_forward":
        return {"bytes": 2 * t * (k + n) + weights, "flops": 2 * t * n * k}
    return {"bytes": 2 * t * (n + 2 * k) + weights + 2 * case["experts"] * n * k, "flops": 4 * t * n * k}


# ------------------------------------------------------------------ plain forms (32 bits)

BLOCK = {"mxfp4": 32, "nvfp4": 16}
MX4_VALUES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def by(x, divisor):
    """x / divisor, correctly rounded (a division by a Python number is a product with its reciprocal)."""
    return x / torch.full_like(x, divisor)


def fp8_values(x):
    """E4M3 codes and scales of the groups x [.., width]: one scale a group, amax / 448."""
    s = by(x.abs().amax(dim=-1, keepdim=True), 448.0).clamp_min(1e-12)
    return (x / s).clamp(-448.0, 448.0).to(torch.float8_e4m3fn), s


def fp8_rows(x):
    """x as the values its 1x128 groups along the columns stand for."""
    r, c = x.shape
    q, s = fp8_values(x.float().reshape(r, c // 128, 128))
    return (q.float() * s).reshape(r, c)


def fp8_columns(x):
    """x as the values its groups of 128 rows (the last one shorter) stand for."""
    r, c = x.shape
    padded = torch.zeros((-(-r // 128) * 128, c), dtype=torch.float32, device=x.device)
    padded[:r] = x.float()
    q, s = fp8_values(padded.reshape(-1, 128, c).transpose(1, 2))
    return (q.float() * s).transpose(1, 2).reshape(-1, c)[:r]


def fp8_weight(w):
    """Codes [n, k] and scales [n/128, k/128] of a weight in 128x128 blocks."""
    n, k = w.shape
    blocks = w.float().reshape(n // 128, 128, k // 128, 128).transpose(1, 2).reshape(n // 128, k // 128, 128 * 128)
    q, s = fp8_values(blocks)
    q = q.view(torch.uint8).reshape(n // 128, k // 128, 128, 128).transpose(1, 2).reshape(n, k)
    return q.contiguous().view(torch.float8_e4m3fn), s.squeeze(-1).contiguous()


def weight_values(q, s):
    return q.float() * s.repeat_interleave(128, 0).repeat_interleave(128, 1)


def power_of_two(byte):
    """2^(byte - 127) in float32, byte 0 .. 254 (the lowest one is not a normal number)."""
    byte = byte.to(torch.int32)
    return torch.where(byte == 0, 1 << 22, byte << 23).to(torch.int32).view(torch.float32)


def mx4_code(v):
    """The 4-bit code of v (float32): nearest of +-MX4_VALUES, ties to the even code."""
    a = v.abs()
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    return code.to(torch.uint8) | (torch.signbit(v).to(torch.uint8) << 3)


def mx4_quantize(x, fmt, g):
    """Packed codes [r, c/2] and scales (bytes, tiled as [r/128, c/(4 block), 512]) of x [r, c]."""
    r, c = x.shape
    b = BLOCK[fmt]
    blocks = x.float().reshape(r, c // b, b)
    amax = blocks.abs().amax(dim=-1)
    if fmt == "mxfp4":
        byte = ((amax.view(torch.int32) >> 23) - 2).clamp(0, 254).to(torch.uint8)
        v = blocks / power_of_two(byte)[..., None]
    else:
        sf = (by(amax, 6.0) / g).clamp_max(448.0).to(torch.float8_e4m3fn)
        byte, d = sf.view(torch.uint8), sf.float() * g
        v = torch.where((d > 0)[..., None], blocks / d[..., None], torch.zeros_like(blocks))
    code = mx4_code(v).reshape(r, c)
    rb, ka = -(-r // 128), -(-(c // b) // 4)
    tiled = torch.zeros((rb * 128, ka * 4), dtype=torch.uint8, device=x.device)
    tiled[:r, :c // b] = byte
    tiled = tiled.reshape(rb, 4, 32, ka, 4).permute(0, 3, 2, 1, 4).reshape(rb, ka, 512)
    return code[:, 0::2] | (code[:, 1::2] << 4), tiled


def mx4_values(q, s, fmt):
    """Values of the codes [r, c] and of the scales [r, c/block] (without the tensor's scale)."""
    r, c = q.shape[0], 2 * q.shape[1]
    table = torch.tensor(MX4_VALUES + tuple(-v for v in MX4_VALUES), dtype=torch.float32, device=q.device)
    codes = torch.stack((q & 15, q >> 4), dim=-1).reshape(r, c)
    rb, ka = s.shape[:2]
    byte = s.reshape(rb, ka, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(rb * 128, ka * 4)[:r, :c // BLOCK[fmt]].contiguous()
    scale = power_of_two(byte) if fmt == "mxfp4" else byte.view(torch.float8_e4m3fn).float()
    return table[codes.int()], scale


def mx4_dequantize(q, s, fmt, g):
    v, scale = mx4_values(q, s, fmt)
    d = scale if g is None else scale * g
    return (v * d.repeat_interleave(BLOCK[fmt], 1)).to(torch.bfloat16)


def mx4_operand(q, s, fmt):
    v, scale = mx4_values(q, s, fmt)
    return v * scale.repeat_interleave(BLOCK[fmt], 1)


def along_rows(x):
    """x^T with the contraction padded to a multiple of 32."""
    r, c = x.shape
    padded = torch.zeros((c, -(-r // 32) * 32), dtype=x.dtype, device=x.device)
    padded[:, :r] = x.t()
    return padded


# ------------------------------------------------------------------ inputs

def normal(rows, cols, std, gen):
    return (torch.randn((rows, cols), generator=gen, device="cuda") * std).to(torch.bfloat16)


def activation(rows, cols, gen):
    """N(0, 1) with two channels of the same large values for every token."""
    x = torch.randn((rows, cols), generator=gen, device="cuda")
    x[:, torch.randint(cols, (2,), generator=gen, device="cuda")] *= 20.0
    return x.to(torch.bfloat16)


def tensor_scale(x, fmt):
    return by(x.float().abs().amax(), 6.0 * 448.0).clamp_min(1e-12).reshape(1) if fmt == "nvfp4" else None


def inputs(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]
    if op.startswith("experts"):
        counts = expert_counts(case)
        places = torch.randperm(len(counts), generator=torch.Generator().manual_seed(seed)).tolist()
        counts = [counts[p] for p in places]
        t, n, k, e = case["tokens"], case["n"], case["k"], case["experts"]
        state = {"counts": counts, "x": activation(t, k, gen), "w": normal(e * n, k, 0.02, gen)}
        if op == "experts_backward":
            state["dy"] = normal(t, n, 1e-3, gen)
        return state
    fmt = case["format"]
    if op == "mx4_roundtrip":
        x = activation(case["rows"], case["cols"], gen)
        return {"x": x, "gx": tensor_scale(x, fmt)}
    if op == "mx4_forward":
        x, w = activation(case["m"], case["k"], gen), normal(case["n"], case["k"], 0.02, gen)
        return {"x": x, "w": w, "gx": tensor_scale(x, fmt), "gw": tensor_scale(w, fmt)}
    x, dy = activation(case["tokens"], case["k"], gen), normal(case["tokens"], case["n"], 1e-3, gen)
    return {"x": x, "dy": dy, "gx": tensor_scale(x, fmt), "gdy": tensor_scale(dy, fmt)}


def prepare(case, seed):
    state = {**case, **inputs(case, seed)}
    op = case["op"]
    if op.startswith("experts"):
        ends = torch.tensor([0] + state["counts"]).cumsum(0)
        state["offsets"] = ends.to(torch.int32).cuda()
        w = state.pop("w")
        q, s = fp8_weight(w)
        if op == "experts_forward":
            state["qw"], state["sw"] = q, s
        else:
            state["qwT"] = q.view(torch.uint8).t().contiguous().view(torch.float8_e4m3fn)
            state["swT"] = s.t().contiguous()
    elif op == "mx4_forward":
        state["qw"], state["sw"] = mx4_quantize(state.pop("w"), state["format"], state["gw"])
    return state


# ------------------------------------------------------------------ one pass

def run(state):
    return RUN[state["op"]](state)


def run_experts_forward(s):
    if own:
        import fp8_blockwise_scaled_b200 as fb
        return fb.grouped_linear_forward(s["x"], s["qw"], s["sw"], s["offsets"])
    w = weight_values(s["qw"], s["sw"]).reshape(s["experts"], s["n"], s["k"])
    x = fp8_rows(s["x"]).split(s["counts"])
    return torch.cat([x[e] @ w[e].t() for e in range(s["experts"])]).to(torch.bfloat16)


def run_experts_backward(s):
    if own:
        import fp8_blockwise_scaled_b200 as fb
        return fb.grouped_linear_backward(s["x"], s["dy"], s["qwT"], s["swT"], s["offsets"])
    w = weight_values(s["qwT"], s["swT"]).reshape(s["k"], s["experts"], s["n"])
    dy, x, counts = s["dy"].split(s["counts"]), s["x"].split(s["counts"]), range(s["experts"])
    rows = fp8_rows(s["dy"]).split(s["counts"])
    dx = torch.cat([rows[e] @ w[:, e].t() for e in counts]).to(torch.bfloat16)
    dw = torch.stack([(fp8_columns(dy[e]).t() @ fp8_columns(x[e])).to(torch.bfloat16) for e in counts])
    return dx, dw


def run_mx4_roundtrip(s):
    fmt, g = s["format"], s["gx"]
    if own:
        import fp8_blockwise_scaled_b200 as fb
        f = fb.MXFP4 if fmt == "mxfp4" else fb.NVFP4
        q, sf, qT, sfT = fb.fp8blk_quantize_mx4(s["x"], f, fb.BOTH if s["both"] else fb.ROWWISE, tensor_scale=g)
        y = fb.fp8blk_dequantize_mx4(q, sf, f, tensor_scale=g)
        return (y, fb.fp8blk_dequantize_mx4(qT, sfT, f, tensor_scale=g)) if s["both"] else (y,)
    y = mx4_dequantize(*mx4_quantize(s["x"], fmt, g), fmt, g)
    if not s["both"]:
        return (y,)
    return y, mx4_dequantize(*mx4_quantize(along_rows(s["x"]), fmt, g), fmt, g)


def run_mx4_forward(s):
    fmt, gx, gw = s["format"], s["gx"], s["gw"]
    if own:
        import fp8_blockwise_scaled_b200 as fb
        return fb.mx4_linear_forward(s["x"], s["qw"], s["sw"], fb.MXFP4 if fmt == "mxfp4" else fb.NVFP4, gx, gw)
    x = mx4_operand(*mx4_quantize(s["x"], fmt, gx), fmt)
    y = x @ mx4_operand(s["qw"], s["sw"], fmt).t()
    return (y if gx is None else y * (gx * gw)).to(torch.bfloat16)


def run_mx4_wgrad(s):
    fmt, gx, gdy = s["format"], s["gx"], s["gdy"]
    if own:
        import fp8_blockwise_scaled_b200 as fb
        return fb.mx4_linear_wgrad(s["x"], s["dy"], fb.MXFP4 if fmt == "mxfp4" else fb.NVFP4, gx, gdy,
                                   out_dtype=torch.float32)
    dy = mx4_operand(*mx4_quantize(along_rows(s["dy"]), fmt, gdy), fmt)
    dw = dy @ mx4_operand(*mx4_quantize(along_rows(s["x"]), fmt, gx), fmt).t()
    return dw if gx is None else dw * (gx * gdy)


RUN = {"experts_forward": run_experts_forward, "experts_backward": run_experts_backward,
       "mx4_roundtrip": run_mx4_roundtrip, "mx4_forward": run_mx4_forward, "mx4_wgrad": run_mx4_wgrad}


# ------------------------------------------------------------------ the definitions in 64 bits

def to_grid(v, mantissa, lowest, top):
    """v rounded to `mantissa` bits below the leading one (ties to even), exponents from `lowest`, saturating."""
    e = torch.frexp(v).exponent.clamp_min(lowest + 1) - 1
    step = torch.ldexp(torch.ones_like(v), e - mantissa)
    return (torch.round(v / step) * step).clamp(-top, top)


def quotient(x, s):
    """The 32-bit quotient that the definition rounds (53 bits hold enough of it to round it once more)."""
    return (x / s).float().double()


def exact_fp8(x, dim):
    """x [.., 128 along dim, ..] (64 bits) as the values of its E4M3 groups."""
    s = by(x.abs().amax(dim=dim, keepdim=True), 448.0).float().clamp_min(1e-12).double()
    return to_grid(quotient(x, s).clamp(-448.0, 448.0), 3, -6, 448.0) * s


def exact_fp8_rows(x):
    return exact_fp8(x.double().unflatten(1, (-1, 128)), 2).flatten(1, 2)


def exact_fp8_tokens(x):
    """Groups of 128 rows, the last one shorter."""
    whole = x.shape[0] // 128 * 128
    parts = [exact_fp8(x[:whole].double().unflatten(0, (-1, 128)), 1).flatten(0, 1)] if whole else []
    return torch.cat(parts + ([exact_fp8(x[whole:].double(), 0)] if whole < x.shape[0] else []))


def exact_fp8_weight(w):
    blocks = w.double().unflatten(1, (-1, 128)).unflatten(0, (-1, 128))
    s = by(blocks.abs().amax(dim=(1, 3), keepdim=True), 448.0).float().clamp_min(1e-12).double()
    return (to_grid(quotient(blocks, s).clamp(-448.0, 448.0), 3, -6, 448.0) * s).flatten(2, 3).flatten(0, 1)


def exact_mx4(x, fmt, g):
    """Codes and scales (both as values, 64 bits) of x [r, c]: [r, c/block, block] and [r, c/block, 1]."""
    v = x.double().unflatten(1, (-1, BLOCK[fmt]))
    amax = v.abs().amax(dim=2, keepdim=True)
    if fmt == "mxfp4":
        e = (torch.frexp(amax).exponent - 1 - 2).clamp(-127, 127)
        scale = torch.ldexp(torch.ones_like(amax), torch.where(amax > 0, e, -127))
        return to_grid((v / scale).clamp(-6.0, 6.0), 1, 0, 6.0), scale
    scale = to_grid((by(amax, 6.0).float().double() / g.double()).float().double().clamp_max(448.0), 3, -6, 448.0)
    d = (scale * g.double()).float().double()
    codes = to_grid(quotient(v, torch.where(d > 0, d, 1.0)).clamp(-6.0, 6.0), 1, 0, 6.0)
    return torch.where(d > 0, codes, 0.0), scale


def exact_mx4_values(x, fmt, g):
    codes, scale = exact_mx4(x, fmt, g)
    return (codes * (scale if g is None else scale * g.double())).flatten(1, 2)


def exact(case, seed):
    s, op = inputs(case, seed), case["op"]
    if op.startswith("experts"):
        w = exact_fp8_weight(s["w"]).unflatten(0, (case["experts"], case["n"]))
        ends = torch.tensor([0] + s["counts"]).cumsum(0).tolist()
        spans = [slice(a, b) for a, b in zip(ends, ends[1:])]
        if op == "experts_forward":
            return torch.cat([exact_fp8_rows(s["x"][span]) @ w[e].t() for e, span in enumerate(spans)])
        dx = torch.cat([exact_fp8_rows(s["dy"][span]) @ w[e] for e, span in enumerate(spans)])
        zero = torch.zeros((case["n"], case["k"]), dtype=torch.float64, device="cuda")
        dw = [exact_fp8_tokens(s["dy"][a]).t() @ exact_fp8_tokens(s["x"][a]) if a.stop > a.start else zero for a in spans]
        return dx, torch.stack(dw)
    fmt = case["format"]
    if op == "mx4_roundtrip":
        out = (exact_mx4_values(s["x"], fmt, s["gx"]),)
        return out + (exact_mx4_values(along_rows(s["x"]), fmt, s["gx"]),) if case["both"] else out
    if op == "mx4_forward":
        return exact_mx4_values(s["x"], fmt, s["gx"]) @ exact_mx4_values(s["w"], fmt, s["gw"]).t()
    dy = exact_mx4_values(along_rows(s["dy"]), fmt, s["gdy"])
    return dy @ exact_mx4_values(along_rows(s["x"]), fmt, s["gx"]).t()
