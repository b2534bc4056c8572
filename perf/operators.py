"""Cases, inputs and plain forms of the block-scaled 8-bit linear layer and its 8-bit checkpoints.

A linear layer y = x W^T is computed in 8-bit floating point with one scale for each block of 128:
activations [T][K] in groups of 128 along a row, weights [N][K] in blocks of 128 x 128.  The codes of
x that the product read are kept as the activation checkpoint, and the backward pass works from
them.  Operators:

  linear      quantise x, then y = x^ W^T (with "keep", the codes and scales of x come back too)
  dgrad       quantise dy, then dx = dy^ W
  wgrad       dw = dy^T x^, x^ the checkpoint
  act         y = f(h) with h kept in 8 bits ("next": y in bf16, or quantised for the next product)
  act_back    dh = dy f'(h^) from the checkpoint of h

The quantiser of a block: with m its largest magnitude, the scale is the smallest power of two s with
m <= top * s (top = 448 for e4m3, 57344 for e5m2; s = 1 for a block of zeros) and each code is x / s
rounded to nearest, ties to even.  Products take any positive scales.  Row groups keep their scales
group-major, [groups][T]; weights row-major, [N blocks][K blocks].
"""
import math

import torch

own = False

E4M3, E5M2 = torch.float8_e4m3fn, torch.float8_e5m2
TOP = {E4M3: 448.0, E5M2: 57344.0}
BLOCK = 128


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one new token through the MLP-up layer of the 4096-wide block: weights stream once
        {"name": "linear token", "op": "linear", "T": 1, "K": 4096, "N": 16384, "scale": "f32", "keep": False},
        # a handful of tokens through MLP-down: a long reduction, few outputs
        {"name": "linear few", "op": "linear", "T": 13, "K": 16384, "N": 4096, "scale": "e8m0", "keep": False},
        # a ragged batch between the two: odd token count, channels that fill no tile
        {"name": "linear ragged", "op": "linear", "T": 391, "K": 1936, "N": 1001, "scale": "f32", "keep": False},
        # the MLP-up layer on 4096 latent patches and 512 text tokens, weights with power-of-two scales
        {"name": "linear dit", "op": "linear", "T": 4608, "K": 4096, "N": 16384, "scale": "e8m0", "keep": False},
        # the same layer in training: general fp32 weight scales, the codes kept as the checkpoint
        {"name": "linear dit train", "op": "linear", "T": 4608, "K": 4096, "N": 16384, "scale": "f32", "keep": True},
        # input gradient of a small ragged micro-batch, gradients in e5m2
        {"name": "dgrad ragged", "op": "dgrad", "T": 517, "K": 1040, "N": 2064, "scale": "f32", "grad": "e5m2"},
        # input gradient of the attention-out layer, gradients in e4m3
        {"name": "dgrad dit", "op": "dgrad", "T": 4608, "K": 4096, "N": 4096, "scale": "e8m0", "grad": "e4m3"},
        # weight gradient of a small ragged micro-batch
        {"name": "wgrad ragged", "op": "wgrad", "T": 517, "K": 1040, "N": 2064, "scale": "f32", "out": "f32"},
        # weight gradient of the QKV projection
        {"name": "wgrad dit", "op": "wgrad", "T": 4608, "K": 4096, "N": 12288, "scale": "f32", "out": "bf16"},
        # MLP activation of a modest batch, quantised on its way into MLP-down
        {"name": "act to fp8", "op": "act", "T": 517, "K": 4096, "act": "gelu_tanh", "next": "fp8"},
        # MLP activation of the whole DiT batch
        {"name": "act dit", "op": "act", "T": 4608, "K": 16384, "act": "gelu_tanh", "next": "bf16"},
        # its backward pass from the 8-bit checkpoint
        {"name": "act back dit", "op": "act_back", "T": 4608, "K": 16384, "act": "silu"},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["linear", "linear", "linear", "dgrad", "wgrad", "act", "act_back"])
    scale = rng.choice(["f32", "e8m0"])
    if op in ("act", "act_back"):
        case = {"op": op, "T": _log_int(rng, 1, 4608), "K": 16 * _log_int(rng, 1, 1024),
                "act": rng.choice(["gelu_tanh", "gelu", "silu"])}
        if op == "act":
            case["next"] = rng.choice(["fp8", "bf16"]) if case["T"] * case["K"] <= 1 << 22 else "bf16"
        return case
    case = {"op": op, "T": _log_int(rng, 1, 4608), "K": 16 * _log_int(rng, 8, 1024), "scale": scale}
    if op == "linear":
        case["N"] = _log_int(rng, 100, 16384)
        case["keep"] = rng.random() < 0.5
    else:
        case["N"] = 16 * _log_int(rng, 8, 1024)
        if op == "dgrad":
            case["grad"] = rng.choice(["e4m3", "e5m2"])
        else:
            case["out"] = rng.choice(["f32", "bf16"])
    most = 4608 * 4096 * 16384          # the largest listed product
    while case["T"] * case["K"] * case["N"] > most:
        case["T"] = max(1, case["T"] // 2)
    return case


# ------------------------------------------------------------------ plain forms

def _groups(d):
    return -(-d // BLOCK)


def _pow2_scale(amax, top):
    """Smallest power of two s with amax <= top * s (top = 1.75 * 2^k), 1 where amax is 0."""
    mant, expo = torch.frexp(amax)                       # amax = mant * 2^expo, mant in [1/2, 1)
    e = expo - 1 - int(math.log2(top / 1.75)) + (mant > 0.875).to(expo.dtype)
    one = torch.ones_like(amax)
    return torch.where(amax > 0, torch.ldexp(one, e.clamp(min=-120)), one)


def _quantise_rows(x, fmt):
    """[T][K] -> codes [T][K] and fp32 scales [groups][T]."""
    T, K = x.shape
    g = _groups(K)
    f = torch.nn.functional.pad(x.float(), (0, g * BLOCK - K)).view(T, g, BLOCK)
    s = _pow2_scale(f.abs().amax(2), TOP[fmt])
    return (f / s[:, :, None]).view(T, g * BLOCK)[:, :K].to(fmt), s.t().contiguous()


def _quantise_blocks(w):
    """[N][K] -> e4m3 codes [N][K] and fp32 scales [N blocks][K blocks]."""
    N, K = w.shape
    n, g = _groups(N), _groups(K)
    f = torch.nn.functional.pad(w.float(), (0, g * BLOCK - K, 0, n * BLOCK - N)).view(n, BLOCK, g, BLOCK)
    s = _pow2_scale(f.abs().amax((1, 3)), TOP[E4M3])
    return (f / s[:, None, :, None]).view(n * BLOCK, g * BLOCK)[:N, :K].to(E4M3), s


def _rows(codes, scale):
    """The values that row-grouped codes stand for, fp32."""
    K = codes.shape[1]
    return codes.float() * scale.float().t().repeat_interleave(BLOCK, 1)[:, :K]


def _blocks(codes, scale):
    """The values that block-scaled codes stand for, fp32."""
    N, K = codes.shape
    return codes.float() * scale.float().repeat_interleave(BLOCK, 0)[:N].repeat_interleave(BLOCK, 1)[:, :K]


_GELU_C = math.sqrt(2.0 / math.pi)


def _act(h, act):
    if act == "gelu_tanh":
        return 0.5 * h * (1 + torch.tanh(_GELU_C * (h + 0.044715 * h * h * h)))
    if act == "gelu":
        return 0.5 * h * (1 + torch.erf(h * math.sqrt(0.5)))
    return h / (1 + torch.exp(-h))


def _act_slope(h, act):
    if act == "gelu_tanh":
        t = torch.tanh(_GELU_C * (h + 0.044715 * h * h * h))
        return 0.5 * (1 + t) + 0.5 * h * (1 - t * t) * _GELU_C * (1 + 3 * 0.044715 * h * h)
    if act == "gelu":
        return 0.5 * (1 + torch.erf(h * math.sqrt(0.5))) + h * torch.exp(-0.5 * h * h) / math.sqrt(2 * math.pi)
    p = 1 / (1 + torch.exp(-h))
    return p * (1 + h * (1 - p))


# ------------------------------------------------------------------ inputs

def _activations(g, T, K):
    """Heavy-tailed rows with a few outlier channels, as a linear layer of a transformer meets."""
    x = torch.randn(T, K, generator=g, device="cuda")
    x *= torch.exp(0.5 * torch.randn(T, K, generator=g, device="cuda"))
    cols = torch.randint(0, K, (max(1, K // 256),), generator=g, device="cuda")
    x[:, cols] *= 20.0
    return x.bfloat16()


def _gradients(g, T, N):
    """Output gradients: small, their size differing from token to token."""
    dy = torch.randn(T, N, generator=g, device="cuda")
    return (dy * (1e-3 * torch.exp(torch.randn(T, 1, generator=g, device="cuda")))).bfloat16()


def _stored(s, scale, g):
    """Scales as the case stores them: powers of two in one byte, or general fp32 ones."""
    if scale == "e8m0":
        return s.to(torch.float8_e8m0fnu)
    return s * (0.75 + 0.5 * torch.rand(s.shape, generator=g, device="cuda"))


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op, T, K = case["op"], case["T"], case["K"]
    s = {"case": case}
    scale_t = torch.float8_e8m0fnu if case.get("scale") == "e8m0" else torch.float32

    def empty(*shape, dtype):
        return torch.empty(*shape, dtype=dtype, device="cuda")

    if op in ("linear", "dgrad"):
        N = case["N"]
        w = torch.randn(N, K, generator=g, device="cuda") * (1.0 / math.sqrt(K))
        w *= torch.exp(0.5 * torch.randn(N, 1, generator=g, device="cuda"))
        s["w"], ws = _quantise_blocks(w)
        s["w_scale"] = _stored(ws, case["scale"], g)
    if op == "linear":
        s["x"] = _activations(g, T, K)
        s["y"] = empty(T, N, dtype=torch.bfloat16)
        if case["keep"]:
            s["codes"], s["scale"] = empty(T, K, dtype=E4M3), empty(_groups(K), T, dtype=scale_t)
    elif op == "dgrad":
        s["dy"] = _gradients(g, T, N)
        s["dx"] = empty(T, K, dtype=torch.bfloat16)
        s["fmt"] = E5M2 if case["grad"] == "e5m2" else E4M3
    elif op == "wgrad":
        s["dy"] = _gradients(g, T, case["N"])
        s["codes"], xs = _quantise_rows(_activations(g, T, K), E4M3)
        s["scale"] = xs.to(scale_t)
        s["dw"] = empty(case["N"], K, dtype=torch.float32 if case["out"] == "f32" else torch.bfloat16)
    else:
        h = (1.5 * torch.randn(T, K, generator=g, device="cuda")).bfloat16()
        if op == "act":
            s["h"] = h
            s["codes"], s["scale"] = empty(T, K, dtype=E4M3), empty(_groups(K), T, dtype=torch.float32)
            if case["next"] == "fp8":
                s["y_codes"], s["y_scale"] = empty(T, K, dtype=E4M3), empty(_groups(K), T, dtype=torch.float32)
            else:
                s["y"] = empty(T, K, dtype=torch.bfloat16)
        else:
            s["codes"], s["scale"] = _quantise_rows(h, E4M3)
            s["dy"] = _gradients(g, T, K)
            s["dh"] = empty(T, K, dtype=torch.bfloat16)
    if own:
        import rotation_then_quantize_amd as rtq
        size = {"linear": rtq.fp8_linear_workspace, "dgrad": rtq.fp8_linear_dgrad_workspace,
                "wgrad": rtq.fp8_wgrad_workspace}.get(op)
        if size is not None:
            s["workspace"] = empty(size(T, case["N"], K), dtype=torch.uint8)
    return s


# ------------------------------------------------------------------ one pass

def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_plain(s):
    case = s["case"]
    op = case["op"]
    if op == "linear":
        codes, scale = _quantise_rows(s["x"], E4M3)
        y = (_rows(codes, scale) @ _blocks(s["w"], s["w_scale"]).T).bfloat16()
        return {"y": y, "codes": codes, "scale": scale} if case["keep"] else {"y": y}
    if op == "dgrad":
        codes, scale = _quantise_rows(s["dy"], s["fmt"])
        return {"dx": (_rows(codes, scale) @ _blocks(s["w"], s["w_scale"])).bfloat16()}
    if op == "wgrad":
        return {"dw": (s["dy"].float().T @ _rows(s["codes"], s["scale"])).to(s["dw"].dtype)}
    if op == "act":
        codes, scale = _quantise_rows(s["h"], E4M3)
        y = _act(s["h"].float(), case["act"])
        if case["next"] == "fp8":
            y_codes, y_scale = _quantise_rows(y, E4M3)
            return {"codes": codes, "scale": scale, "y_codes": y_codes, "y_scale": y_scale}
        return {"codes": codes, "scale": scale, "y": y.bfloat16()}
    slope = _act_slope(_rows(s["codes"], s["scale"]), case["act"])
    return {"dh": (s["dy"].float() * slope).bfloat16()}


def _run_own(s):
    import rotation_then_quantize_amd as rtq
    case = s["case"]
    op = case["op"]
    if op == "linear":
        if case["keep"]:
            rtq.fp8_linear(s["x"], s["w"], s["w_scale"], s["y"], x_codes=s["codes"], x_scale=s["scale"],
                           workspace=s["workspace"])
            return {"y": s["y"], "codes": s["codes"], "scale": s["scale"].float()}
        rtq.fp8_linear(s["x"], s["w"], s["w_scale"], s["y"], workspace=s["workspace"])
        return {"y": s["y"]}
    if op == "dgrad":
        rtq.fp8_linear_dgrad(s["dy"], s["w"], s["w_scale"], s["dx"], grad_dtype=s["fmt"], workspace=s["workspace"])
        return {"dx": s["dx"]}
    if op == "wgrad":
        rtq.fp8_wgrad(s["dy"], s["codes"], s["scale"], s["dw"], workspace=s["workspace"])
        return {"dw": s["dw"]}
    act = {"gelu_tanh": rtq.RTQ_ACT_GELU_TANH, "gelu": rtq.RTQ_ACT_GELU, "silu": rtq.RTQ_ACT_SILU}[case["act"]]
    if op == "act":
        if case["next"] == "fp8":
            rtq.act_fp8_forward(s["h"], act, s["codes"], s["scale"], y_codes=s["y_codes"], y_scale=s["y_scale"])
            return {"codes": s["codes"], "scale": s["scale"], "y_codes": s["y_codes"], "y_scale": s["y_scale"]}
        rtq.act_fp8_forward(s["h"], act, s["codes"], s["scale"], y=s["y"])
        return {"codes": s["codes"], "scale": s["scale"], "y": s["y"]}
    rtq.act_fp8_backward(s["dy"], s["codes"], s["scale"], act, s["dh"])
    return {"dh": s["dh"]}


def work(case):
    op, T, K = case["op"], case["T"], case["K"]
    sb = 1 if case.get("scale") == "e8m0" else 4
    g = _groups(K)
    if op == "act":
        out = T * K + 4 * T * g if case["next"] == "fp8" else 2 * T * K
        return {"bytes": 2 * T * K + T * K + 4 * T * g + out, "flops": 10 * T * K}
    if op == "act_back":
        return {"bytes": T * K + 4 * T * g + 2 * T * K + 2 * T * K, "flops": 10 * T * K}
    N = case["N"]
    weights = N * K + sb * _groups(N) * g
    if op == "linear":
        kept = T * K + sb * T * g if case["keep"] else 0
        b = 2 * T * K + weights + 2 * T * N + kept
    elif op == "dgrad":
        b = 2 * T * N + weights + 2 * T * K
    else:
        b = 2 * T * N + T * K + sb * T * g + N * K * (4 if case["out"] == "f32" else 2)
    return {"bytes": b, "flops": 2 * T * N * K}


# ------------------------------------------------------------------ the definition, in 64 bits

def _exact_codes(x, fmt):
    """Codes' values and scales of row groups, from the definition in 64 bits."""
    T, K = x.shape
    bits, low = (3, -6) if fmt == E4M3 else (2, -14)     # mantissa bits, smallest normal exponent
    codes = torch.empty(T, K, dtype=torch.float64, device=x.device)
    scale = torch.ones(_groups(K), T, dtype=torch.float64, device=x.device)
    for j in range(_groups(K)):
        part = x[:, j * BLOCK:(j + 1) * BLOCK]
        m = part.abs().max(1).values
        s = torch.where(m > 0, torch.exp2(torch.ceil(torch.log2(m / TOP[fmt])).clamp(min=-120)), 1.0)
        v = part / s[:, None]
        lead = torch.floor(torch.log2(v.abs().clamp(min=2.0 ** low)))
        step = torch.exp2(lead - bits)
        codes[:, j * BLOCK:(j + 1) * BLOCK] = torch.round(v / step) * step
        scale[j] = s
    return codes, scale


def _exact_matrix(codes, scale, row_block):
    values = codes.to(torch.float64, copy=True)
    s = scale.double()
    if row_block == 1:
        for j in range(s.shape[0]):
            values[:, j * BLOCK:(j + 1) * BLOCK] *= s[j][:, None]
        return values
    for i in range(s.shape[0]):
        for j in range(s.shape[1]):
            values[i * row_block:(i + 1) * row_block, j * BLOCK:(j + 1) * BLOCK] *= s[i, j]
    return values


def _exact_act(h, act):
    if act == "silu":
        return h * torch.sigmoid(h)
    if act == "gelu":
        return h * 0.5 * torch.erfc(-h / math.sqrt(2.0))
    u = math.sqrt(2.0 / math.pi) * (h + 0.044715 * h ** 3)
    return h * torch.sigmoid(2.0 * u)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "linear":
        codes, scale = _exact_codes(s["x"].double(), E4M3)
        y = torch.matmul(_exact_matrix(codes, scale, 1), _exact_matrix(s["w"], s["w_scale"], BLOCK).t().contiguous())
        return {"y": y, "codes": codes, "scale": scale} if case["keep"] else {"y": y}
    if op == "dgrad":
        codes, scale = _exact_codes(s["dy"].double(), s["fmt"])
        return {"dx": torch.matmul(_exact_matrix(codes, scale, 1), _exact_matrix(s["w"], s["w_scale"], BLOCK))}
    if op == "wgrad":
        return {"dw": torch.matmul(s["dy"].double().t().contiguous(), _exact_matrix(s["codes"], s["scale"], 1))}
    if op == "act":
        h = s["h"].double()
        codes, scale = _exact_codes(h, E4M3)
        y = _exact_act(h, case["act"])
        if case["next"] == "fp8":
            y_codes, y_scale = _exact_codes(y, E4M3)
            return {"codes": codes, "scale": scale, "y_codes": y_codes, "y_scale": y_scale}
        return {"codes": codes, "scale": scale, "y": y}
    h = _exact_matrix(s["codes"], s["scale"], 1)
    with torch.enable_grad():
        h.requires_grad_(True)
        (slope,) = torch.autograd.grad(_exact_act(h, case["act"]).sum(), h)
    return {"dh": s["dy"].double() * slope}
