"""The 4-bit floating-point operators: their cases, plain forms and 64-bit definitions.

A 4-bit matrix holds E2M1 codes (the values 0, 0.5, 1, 1.5, 2, 3, 4, 6 and their
negatives), two to a byte with the lower column in the low half, and one 8-bit
scale for each block of a row:

  mxfp4   blocks of 32, the scale a power of two (E8M0: 2^(byte - 127))
  nvfp4   blocks of 16, the scale an E4M3 number, and one FP32 scale g for the matrix

Four uses of them are measured:

  quantise   a BF16 or FP32 matrix to 4 bits, along its rows, of its transpose, or
             both in one reading, and back to the values the codes stand for
  product    C = A B^T of two 4-bit matrices (+ bias), FP32 or BF16 result
  weights    C = X W^T, X BF16 rows (activations), W a 4-bit matrix
  step       the three products of a linear layer's training step: Y = X W^T,
             dX = dY W and dW = dY^T X, each operand in 4 bits along the axis its
             product sums over

Quantising a block with largest magnitude m:
  mxfp4: s = 2^clamp(floor(log2 m) - 2, -127, 127)
  nvfp4: s = E4M3(m / (6 g)), g the smallest power of two with 2688 g >= max |X|
then each value over its scale (s, or s g) goes to the nearest E2M1 value (ties
to the even code, magnitudes above 6 to 6). 2688 = 6 x 448, the largest values
of the two formats; a matrix that comes quantised may have any g.
"""
import torch

own = False

BLOCK = {"mxfp4": 32, "nvfp4": 16}
DTYPE = {"f32": torch.float32, "bf16": torch.bfloat16}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)
# Codes of a quantised normal block (64 equally likely draws).
NORMAL_CODES = ([0] * 3 + [8] * 3 + [1] * 6 + [9] * 6 + [2] * 6 + [10] * 6 + [3] * 5 + [11] * 5 +
                [4] * 5 + [12] * 5 + [5] * 4 + [13] * 4 + [6] * 2 + [14] * 2 + [7] + [15])


def listed():
    return [
        # One token's hidden state on its way into a 4-bit layer: launch latency.
        {"name": "quantise_token", "op": "quantise", "rows": 1, "cols": 4096, "fmt": "nvfp4", "type": "bf16",
         "way": "rows"},
        # An FP32 matrix of odd sizes quantised along its columns (a weight stored K x N).
        {"name": "quantise_ragged", "op": "quantise", "rows": 3000, "cols": 1537, "fmt": "mxfp4", "type": "f32",
         "way": "trans"},
        # The gradient of the FFN's wide side, both ways at once, as its two products need it.
        {"name": "quantise_ffn_both", "op": "quantise", "rows": 8192, "cols": 14336, "fmt": "nvfp4", "type": "bf16",
         "way": "both"},
        # A small square product: few tiles, short sums.
        {"name": "product_1024", "op": "product", "M": 1024, "N": 1024, "K": 1024, "fmt": "mxfp4", "type": "f32",
         "bias": False},
        # Sizes that are whole tiles in no direction, K odd.
        {"name": "product_ragged", "op": "product", "M": 3000, "N": 5001, "K": 1537, "fmt": "nvfp4", "type": "f32",
         "bias": True},
        # The FFN's up projection of 8192 tokens.
        {"name": "product_ffn", "op": "product", "M": 8192, "N": 14336, "K": 4096, "fmt": "nvfp4", "type": "bf16",
         "bias": False},
        # The same layer for 16 tokens: bound by reading the weights once.
        {"name": "product_skinny", "op": "product", "M": 16, "N": 14336, "K": 4096, "fmt": "mxfp4", "type": "bf16",
         "bias": False},
        # Decoding one token with BF16 activations: the layer's up projection.
        {"name": "weights_token", "op": "weights", "M": 1, "N": 14336, "K": 4096, "fmt": "mxfp4", "type": "bf16",
         "bias": False},
        # 16 sequences decoding: the down projection, a long sum.
        {"name": "weights_skinny", "op": "weights", "M": 16, "N": 4096, "K": 14336, "fmt": "nvfp4", "type": "f32",
         "bias": True},
        # A prompt of 8192 tokens through the same kept weights.
        {"name": "weights_ffn", "op": "weights", "M": 8192, "N": 14336, "K": 4096, "fmt": "mxfp4", "type": "bf16",
         "bias": False},
        # A small layer's training step.
        {"name": "step_small", "op": "step", "M": 256, "N": 1024, "K": 1024, "fmt": "mxfp4"},
        # The FFN layer's training step on 8192 tokens.
        {"name": "step_ffn", "op": "step", "M": 8192, "N": 14336, "K": 4096, "fmt": "nvfp4"},
    ]


def draw(rng):
    def size(lo, hi):
        n = int(round(lo * (hi / lo) ** rng.random()))
        return 3071 if n == 3072 else n

    op = rng.choice(["quantise", "product", "weights", "step"])
    fmt = rng.choice(["mxfp4", "nvfp4"])
    kind = rng.choice(["f32", "bf16"])
    if op == "quantise":
        return {"op": op, "rows": size(1, 8192), "cols": size(32, 14336), "fmt": fmt, "type": kind,
                "way": rng.choice(["rows", "trans", "both"])}
    if op == "step":
        return {"op": op, "M": size(64, 8192), "N": size(64, 14336), "K": size(64, 4096), "fmt": fmt}
    N, K = size(64, 14336), size(64, 4096)
    if rng.random() < 0.3:
        N, K = K, N
    return {"op": op, "M": size(1, 8192), "N": N, "K": K, "fmt": fmt, "type": kind, "bias": rng.random() < 0.3}


# ------------------------------------------------------------------ inputs

def _blocks(K, fmt):
    return -(-K // BLOCK[fmt])


def _values(rows, cols, std, dtype, g):
    """Normal values with a few columns ten times as large, as activations have them."""
    x = torch.randn((rows, cols), generator=g, device="cuda")
    big = torch.rand((1, cols), generator=g, device="cuda") < 0.005
    return torch.where(big, x * (10 * std), x * std).to(dtype)


def _codes(rows, K, fmt, g):
    """A matrix that is in 4 bits already, as a checkpoint holds it: codes, scales, g."""
    table = torch.tensor(NORMAL_CODES, device="cuda", dtype=torch.uint8)
    pick = torch.randint(0, 64, (rows, 2 * (-(-K // 2))), generator=g, device="cuda")
    c = table[pick]
    c[:, K:] = 0
    codes = c[:, 0::2] | (c[:, 1::2] << 4)
    shape = (rows, _blocks(K, fmt))
    if fmt == "mxfp4":
        scales = torch.randint(117, 121, shape, generator=g, device="cuda").to(torch.uint8)
        return codes, scales, None
    scales = torch.randint(0x58, 0x7F, shape, generator=g, device="cuda").to(torch.uint8)
    return codes, scales, torch.rand(1, generator=g, device="cuda") * 2e-5 + 1e-5


def _inputs(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    fmt, op = case["fmt"], case["op"]
    if op == "quantise":
        return {"X": _values(case["rows"], case["cols"], 1.0, DTYPE[case["type"]], g)}
    M, N, K = case["M"], case["N"], case["K"]
    if op == "step":
        return {"X": _values(M, K, 1.0, torch.bfloat16, g), "W": _values(N, K, 0.02, torch.bfloat16, g),
                "dY": _values(M, N, 1e-4, torch.bfloat16, g)}
    s = {"A": _codes(M, K, fmt, g) if op == "product" else _values(M, K, 1.0, torch.bfloat16, g),
         "B": _codes(N, K, fmt, g)}
    s["bias"] = torch.randn(N, generator=g, device="cuda") * 0.1 if case["bias"] else None
    return s


def prepare(case, seed):
    """The inputs; and where the framework runs, its handles of the matrices that are in 4 bits
    already (weights laid out once when they are loaded)."""
    s = dict(_inputs(case, seed), case=dict(case))
    if own:
        import tiled_matrix_multiplication_sm_gb300 as tg
        for name in ("A", "B"):
            if isinstance(s.get(name), tuple):
                codes, scales, scale = s[name]
                s[name] = tg.mx4_pack(codes, scales, case["fmt"], cols=case["K"], tensor_scale=scale)
    return s


# ------------------------------------------------------------- plain forms

def _round_e2m1(v):
    a = v.abs().clamp(max=6.0)
    step = torch.where(a < 2.0, 0.5, torch.where(a < 4.0, 1.0, 2.0))
    return torch.copysign(torch.round(a / step) * step, v)


def _power(e):
    """2^e for whole e in -126 .. 127, FP32."""
    return ((e + 127) << 23).to(torch.int32).view(torch.float32)


def _tensor_scale(X):
    m, e = torch.frexp(X.abs().max().float() / 2688.0)
    return _power((e - (m == 0.5).int()).clamp(min=-100, max=117))


def _read_back(X, fmt, g):
    """The values X's rows stand for after quantising, FP32."""
    R, K = X.shape
    B, nb = BLOCK[fmt], _blocks(K, fmt)
    x = torch.nn.functional.pad(X.float(), (0, nb * B - K)).reshape(R, nb, B)
    m = x.abs().amax(dim=2, keepdim=True)
    if fmt == "mxfp4":
        e = (torch.frexp(m).exponent - 3).clamp(-127, 127)
        e = torch.where(m == 0, torch.full_like(e, -127), e)
        inverse = _power((-e).clamp(min=-126))
        scale = torch.where(e == -127, torch.full_like(m, 2.0 ** -127), _power(e.clamp(min=-126)))
        v = _round_e2m1(x * inverse) * scale
    else:
        s = (m / (6.0 * g)).clamp(max=448.0).to(torch.float8_e4m3fn).float()
        v = _round_e2m1(torch.where(s > 0, x / (s * g), torch.zeros_like(x))) * s * g
    return v.reshape(R, nb * B)[:, :K]


def _decode(matrix, K, fmt):
    codes, scales, g = matrix
    table = torch.tensor(E2M1, device=codes.device)
    v = torch.stack((table[(codes & 15).int()], table[(codes >> 4).int()]), dim=2)
    v = v.reshape(codes.shape[0], -1)[:, :K]
    s = _power(scales.int() - 127) if fmt == "mxfp4" else scales.view(torch.float8_e4m3fn).float()
    v = v * s.repeat_interleave(BLOCK[fmt], dim=1)[:, :K]
    return v if g is None else v * g


def _plain(s):
    case = s["case"]
    fmt, op = case["fmt"], case["op"]
    if op == "quantise":
        X, kind = s["X"], DTYPE[case["type"]]
        g = _tensor_scale(X) if fmt == "nvfp4" else None
        out = {}
        if case["way"] != "trans":
            out["rows"] = _read_back(X, fmt, g).to(kind)
        if case["way"] != "rows":
            out["trans"] = _read_back(X.t(), fmt, g).to(kind)
        return out
    if op == "step":
        X, W, dY = s["X"], s["W"], s["dY"]
        gx, gw, gy = (_tensor_scale(t) if fmt == "nvfp4" else None for t in (X, W, dY))
        y = _read_back(X, fmt, gx) @ _read_back(W, fmt, gw).t()
        dx = _read_back(dY, fmt, gy) @ _read_back(W.t(), fmt, gw).t()
        dw = _read_back(dY.t(), fmt, gy) @ _read_back(X.t(), fmt, gx).t()
        return {"y": y.bfloat16(), "dx": dx.bfloat16(), "dw": dw}
    K = case["K"]
    a = _decode(s["A"], K, fmt) if op == "product" else s["A"].float()
    c = a @ _decode(s["B"], K, fmt).t()
    if s["bias"] is not None:
        c = c + s["bias"]
    return c.to(DTYPE[case["type"]])


# ------------------------------------------------------- the framework's calls

def _framework(s):
    import tiled_matrix_multiplication_sm_gb300 as tg
    case = s["case"]
    fmt, op = case["fmt"], case["op"]
    if op == "quantise":
        kind, way = DTYPE[case["type"]], case["way"]
        if way == "both":
            q, t = tg.mx4_quantize_both(s["X"], fmt)
            return {"rows": tg.mx4_dequantize(q, kind), "trans": tg.mx4_dequantize(t, kind)}
        return {way: tg.mx4_dequantize(tg.mx4_quantize(s["X"], fmt, trans=way == "trans"), kind)}
    if op == "step":
        x, x_t = tg.mx4_quantize_both(s["X"], fmt)
        w, w_t = tg.mx4_quantize_both(s["W"], fmt)
        y = tg.gemm_mx4(x, w, out_dtype=torch.bfloat16)
        dy, dy_t = tg.mx4_quantize_both(s["dY"], fmt)
        return {"y": y, "dx": tg.gemm_mx4(dy, w_t, out_dtype=torch.bfloat16), "dw": tg.gemm_mx4(dy_t, x_t)}
    call = tg.gemm_mx4 if op == "product" else tg.gemm_w4
    return call(s["A"], s["B"], out_dtype=DTYPE[case["type"]], bias=s["bias"])


def run(state):
    return _framework(state) if own else _plain(state)


# ------------------------------------------------------------------- work

def _held(rows, K, fmt):
    """Bytes of a matrix in 4 bits: codes and scales."""
    return rows * (-(-K // 2) + _blocks(K, fmt))


def work(case):
    fmt, op = case["fmt"], case["op"]
    size = {"f32": 4, "bf16": 2}
    if op == "quantise":
        R, C, e = case["rows"], case["cols"], size[case["type"]]
        held = (_held(R, C, fmt) if case["way"] != "trans" else 0) + (_held(C, R, fmt) if case["way"] != "rows" else 0)
        back = R * C * e * (2 if case["way"] == "both" else 1)
        return {"bytes": R * C * e + held + back, "flops": 0}
    M, N, K = case["M"], case["N"], case["K"]
    if op == "step":
        return {"bytes": 2 * (M * K + N * K + M * N) + 2 * (M * N + M * K) + 4 * N * K, "flops": 6 * M * N * K}
    a = _held(M, K, fmt) if op == "product" else 2 * M * K
    return {"bytes": a + _held(N, K, fmt) + M * N * size[case["type"]] + (4 * N if case["bias"] else 0),
            "flops": 2 * M * N * K}


# ------------------------------------------------------ 64-bit definitions

def _exact_e2m1(v):
    a = v.abs()
    code = ((a > 0.25).int() + (a >= 0.75).int() + (a > 1.25).int() + (a >= 1.75).int() + (a > 2.5).int() +
            (a >= 3.5).int() + (a > 5.0).int())
    value = torch.tensor(E2M1[:8], device=v.device, dtype=torch.float64)[code]
    return torch.where(v < 0, -value, value)


def _exact_exponent(v):
    """floor(log2 v) of positive numbers, from their bits."""
    return ((v.contiguous().view(torch.int64) >> 52) - 1023).double()


def _exact_e4m3(v):
    unit = torch.exp2(_exact_exponent(v.clamp(min=2.0 ** -6)) - 3)
    return (torch.round(v / unit) * unit).clamp(max=448.0)


def _exact_back(X, fmt, g):
    K, B = X.shape[1], BLOCK[fmt]
    whole = torch.zeros((X.shape[0], _blocks(K, fmt) * B), device=X.device, dtype=torch.float64)
    whole[:, :K] = X
    x = whole.unflatten(1, (-1, B))
    m = x.abs().max(dim=2, keepdim=True).values
    if fmt == "mxfp4":
        s = torch.exp2(_exact_exponent(m.clamp(min=2.0 ** -125)) - 2)
    else:
        s = _exact_e4m3(m / (6 * g)) * g
    return torch.where(s > 0, _exact_e2m1(x / s) * s, torch.zeros_like(x)).flatten(1)[:, :K]


def _exact_scale(X):
    most, g = float(X.abs().max()), 2.0 ** -100
    while 2688 * g < most:
        g *= 2
    return g


def _exact_decode(matrix, K, fmt):
    codes, scales, g = matrix
    low, high = (codes % 16).long(), torch.div(codes, 16, rounding_mode="floor").long()
    table = torch.tensor(E2M1, device=codes.device, dtype=torch.float64)
    v = table[torch.stack((low, high), dim=2).flatten(1)[:, :K]]
    b = scales.long()
    if fmt == "mxfp4":
        s = torch.exp2(b.double() - 127)
    else:
        e, f = (b // 8).double(), (b % 8).double()
        s = torch.where(e > 0, torch.exp2(e - 7) * (1 + f / 8), f * 2.0 ** -9) * float(g)
    return v * s[:, torch.arange(K, device=codes.device) // BLOCK[fmt]]


def exact(case, seed):
    s = _inputs(case, seed)
    fmt, op = case["fmt"], case["op"]
    if op == "quantise":
        X = s["X"].double()
        g = _exact_scale(s["X"]) if fmt == "nvfp4" else None
        out = {}
        if case["way"] != "trans":
            out["rows"] = _exact_back(X, fmt, g)
        if case["way"] != "rows":
            out["trans"] = _exact_back(X.t(), fmt, g)
        return out
    if op == "step":
        X, W, dY = s["X"].double(), s["W"].double(), s["dY"].double()
        gx, gw, gy = (_exact_scale(t) for t in (X, W, dY))
        return {"y": _exact_back(X, fmt, gx) @ _exact_back(W, fmt, gw).t(),
                "dx": _exact_back(dY, fmt, gy) @ _exact_back(W.t(), fmt, gw).t(),
                "dw": _exact_back(dY.t(), fmt, gy) @ _exact_back(X.t(), fmt, gx).t()}
    a = _exact_decode(s["A"], case["K"], fmt) if op == "product" else s["A"].double()
    c = a @ _exact_decode(s["B"], case["K"], fmt).t()
    return c if s["bias"] is None else c + s["bias"].double()
