"""Cases, inputs and plain forms of what stands around the 8-bit linear layers of a gated MLP block.

Operators:

  norm        h = x + r (the residual stream, rounded to its type), n = h / sqrt(mean h^2 + eps) * gamma, out
              as e4m3 codes with a scale for each 128 of a row, or as values
  norm_back   the gradients of h (the residual stream's own added) and of gamma
  glu         g = x Wg^T, u = x Wu^T from 8-bit codes with scales for blocks of 128, y = f(g) u, out as values or
              as codes; with "keep" the codes of [g u], the checkpoint, come back too
  glu_back    the gradient of [g u] from the checkpoint, as values (for the weight gradient) and as codes (for
              the input gradient)
  clip        the 2-norm of all gradients together, and the gradients scaled to at most a given norm

The two projections' weights are stacked, [2 N][K], the gate's first.  The quantiser of a group of 128: with m its
largest magnitude, the scale is the smallest power of two s with m <= top * s (top = 448 for e4m3, 57344 for e5m2;
s = 1 for a group of zeros) and each code is x / s rounded to nearest, ties to even.  Row groups keep their scales
group-major, [groups][T]; weights row-major, [N blocks][K blocks].  Codes and their scales come back as the 8-bit
numbers they are.
"""
import math

import torch

own = False

E4M3, E5M2, E8M0 = torch.float8_e4m3fn, torch.float8_e5m2, torch.float8_e8m0fnu
TOP = {E4M3: 448.0, E5M2: 57344.0}
TYPE = {"bf16": torch.bfloat16, "f32": torch.float32}
BLOCK = 128
EPS = 1e-6


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one new token entering an MLP: latency
        {"name": "norm token", "op": "norm", "T": 1, "d": 4096, "x": "bf16", "r": "bf16", "gamma": "bf16", "out": "codes"},
        # the whole batch of 4096 patches and 512 text tokens, quantised on its way into the projections
        {"name": "norm dit", "op": "norm", "T": 4608, "d": 4096, "x": "bf16", "r": "bf16", "gamma": "bf16", "out": "codes"},
        # a small ragged micro-batch with an fp32 residual stream
        {"name": "norm back ragged", "op": "norm_back", "T": 391, "d": 1936, "x": "bf16", "r": "f32", "gamma": "f32"},
        # the whole batch in training
        {"name": "norm back dit", "op": "norm_back", "T": 4608, "d": 4096, "x": "bf16", "r": "bf16", "gamma": "bf16"},
        # one new token through both projections: the weights stream once
        {"name": "glu token", "op": "glu", "T": 1, "K": 4096, "N": 16384, "scale": "f32", "act": "silu", "out": "bf16", "keep": False},
        # a few tokens, quantised on their way into the next product
        {"name": "glu few", "op": "glu", "T": 13, "K": 4096, "N": 10880, "scale": "e8m0", "act": "silu", "out": "codes", "keep": False},
        # a small ragged micro-batch in training
        {"name": "glu ragged train", "op": "glu", "T": 391, "K": 1936, "N": 1152, "scale": "e8m0", "act": "gelu_tanh", "out": "codes", "keep": True},
        # the whole batch in training: general fp32 weight scales
        {"name": "glu dit train", "op": "glu", "T": 4608, "K": 4096, "N": 16384, "scale": "f32", "act": "silu", "out": "codes", "keep": True},
        # gradient of a modest batch
        {"name": "glu back small", "op": "glu_back", "T": 517, "N": 1152, "act": "gelu_tanh", "grad": "e4m3"},
        # gradient of the whole batch
        {"name": "glu back dit", "op": "glu_back", "T": 4608, "N": 16384, "act": "silu", "grad": "e5m2"},
        # the gradients of a small model of many blocks: many tensors, some of a few hundred elements
        {"name": "clip many", "op": "clip", "blocks": 16, "d": 272, "N": 640, "type": "f32", "most": 0.5},
        # those of two blocks of the 4096-wide MLP
        {"name": "clip dit", "op": "clip", "blocks": 2, "d": 4096, "N": 16384, "type": "bf16", "most": 1.0},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm_back", "glu", "glu", "glu", "glu_back", "clip"])
    act = rng.choice(["gelu_tanh", "gelu", "silu"])
    if op in ("norm", "norm_back"):
        case = {"op": op, "T": _log_int(rng, 1, 4608), "d": 16 * _log_int(rng, 1, 1024), "x": rng.choice(["bf16", "f32"]),
                "r": rng.choice(["bf16", "f32", "none"]), "gamma": rng.choice(["bf16", "f32"])}
        if op == "norm":
            case["out"] = rng.choice(["codes", "values"])
        while case["T"] * case["d"] > 4608 * 4096:
            case["T"] = max(1, case["T"] // 2)
        return case
    if op == "glu":
        case = {"op": op, "T": _log_int(rng, 1, 4608), "K": 16 * _log_int(rng, 8, 512), "N": 128 * _log_int(rng, 1, 128),
                "scale": rng.choice(["f32", "e8m0"]), "act": act, "out": rng.choice(["bf16", "codes"]), "keep": rng.random() < 0.5}
        while case["T"] * case["K"] * case["N"] > 4608 * 4096 * 16384 or case["K"] * case["N"] > 4096 * 16384:
            case["T"], case["K"] = max(1, case["T"] // 2), max(128, case["K"] // 32 * 16)
        return case
    if op == "glu_back":
        return {"op": op, "T": _log_int(rng, 1, 4608), "N": 128 * _log_int(rng, 1, 128), "act": act, "grad": rng.choice(["e4m3", "e5m2"])}
    case = {"op": op, "blocks": _log_int(rng, 1, 20), "d": _log_int(rng, 16, 4096), "N": _log_int(rng, 16, 16384),
            "type": rng.choice(["bf16", "f32"]), "most": rng.choice([0.1, 1.0, 1e6])}
    while case["blocks"] * case["d"] * case["N"] > 2 * 4096 * 16384 // (2 if case["type"] == "f32" else 1):
        case["N"] = max(16, case["N"] // 2)
        case["blocks"] = max(1, case["blocks"] // 2)
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
        return h / (1 + torch.exp(-2 * _GELU_C * (h + 0.044715 * h * h * h)))
    if act == "gelu":
        return 0.5 * h * torch.erfc(-h * math.sqrt(0.5))
    return h / (1 + torch.exp(-h))


def _act_slope(h, act):
    if act == "gelu_tanh":
        p = 1 / (1 + torch.exp(-2 * _GELU_C * (h + 0.044715 * h * h * h)))
        return p + h * p * (1 - p) * 2 * _GELU_C * (1 + 3 * 0.044715 * h * h)
    if act == "gelu":
        return 0.5 * torch.erfc(-h * math.sqrt(0.5)) + h * torch.exp(-0.5 * h * h) / math.sqrt(2 * math.pi)
    p = 1 / (1 + torch.exp(-h))
    return p * (1 + h * (1 - p))


def _out(values, fmt):
    """Values as codes and scales, each the 8-bit numbers they are."""
    codes, scale = _quantise_rows(values, fmt)
    return {"codes": codes, "scale": scale.to(E8M0)}


# ------------------------------------------------------------------ inputs

def _activations(g, T, K):
    """Heavy-tailed rows with a few outlier channels, as a layer of a transformer meets."""
    x = torch.randn(T, K, generator=g, device="cuda")
    x *= torch.exp(0.5 * torch.randn(T, K, generator=g, device="cuda"))
    cols = torch.randint(0, K, (max(1, K // 256),), generator=g, device="cuda")
    x[:, cols] *= 20.0
    return x


def _gradients(g, T, N):
    """Output gradients: small, their size differing from token to token."""
    dy = torch.randn(T, N, generator=g, device="cuda")
    return dy * (1e-3 * torch.exp(torch.randn(T, 1, generator=g, device="cuda")))


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op = case["op"]
    s = {"case": case}

    def empty(*shape, dtype):
        return torch.empty(*shape, dtype=dtype, device="cuda")

    if op in ("norm", "norm_back"):
        T, d = case["T"], case["d"]
        xt = TYPE[case["x"]]
        rt = TYPE.get(case["r"], xt)
        s["gamma"] = (1 + 0.2 * torch.randn(d, generator=g, device="cuda")).to(TYPE[case["gamma"]])
        if op == "norm":
            s["x"] = _activations(g, T, d).to(xt)
            if case["r"] != "none":
                s["r"], s["h"] = (3 * _activations(g, T, d)).to(rt), empty(T, d, dtype=rt)
            if case["out"] == "codes":
                s["codes"], s["scale"] = empty(T, d, dtype=E4M3), empty(_groups(d), T, dtype=E8M0)
            else:
                s["y"] = empty(T, d, dtype=xt)
        else:
            s["h"] = (3 * _activations(g, T, d)).to(rt)
            s["dn"] = _gradients(g, T, d).to(xt)
            if case["r"] != "none":
                s["dr"] = _gradients(g, T, d).to(rt)
            s["dh"], s["dgamma"] = empty(T, d, dtype=rt), empty(d, dtype=torch.float32)
    elif op == "glu":
        T, K, N = case["T"], case["K"], case["N"]
        w = torch.randn(2 * N, K, generator=g, device="cuda") * (1.0 / math.sqrt(K))
        w *= torch.exp(0.5 * torch.randn(2 * N, 1, generator=g, device="cuda"))
        s["w"], ws = _quantise_blocks(w)
        st = E8M0 if case["scale"] == "e8m0" else torch.float32
        s["w_scale"] = ws.to(st) if st == E8M0 else ws * (0.75 + 0.5 * torch.rand(ws.shape, generator=g, device="cuda"))
        s["x"], xs = _quantise_rows(_activations(g, T, K), E4M3)
        s["x_scale"] = xs.to(st)
        if case["out"] == "codes":
            s["codes"], s["scale"] = empty(T, N, dtype=E4M3), empty(_groups(N), T, dtype=st)
        else:
            s["y"] = empty(T, N, dtype=torch.bfloat16)
        if case["keep"]:
            s["h_codes"], s["h_scale"] = empty(T, 2 * N, dtype=E4M3), empty(_groups(2 * N), T, dtype=st)
    elif op == "glu_back":
        T, N = case["T"], case["N"]
        s["fmt"] = E5M2 if case["grad"] == "e5m2" else E4M3
        s["h"], s["h_scale"] = _quantise_rows(1.5 * torch.randn(T, 2 * N, generator=g, device="cuda"), E4M3)
        s["h_scale"] = s["h_scale"].to(E8M0)
        s["dy"] = _gradients(g, T, N).bfloat16()
        s["dh"] = empty(T, 2 * N, dtype=torch.bfloat16)
        s["codes"], s["scale"] = empty(T, 2 * N, dtype=s["fmt"]), empty(_groups(2 * N), T, dtype=E8M0)
    else:
        d, N, t = case["d"], case["N"], TYPE[case["type"]]
        shapes = [shape for _ in range(case["blocks"]) for shape in ((d,), (2 * N, d), (d, N))]
        s["grads"] = [(1e-2 * torch.randn(shape, generator=g, device="cuda")).to(t) for shape in shapes]
        s["outs"] = [torch.empty_like(x) for x in s["grads"]]
        s["norm"] = empty(1, dtype=torch.float32)
    if own:
        import rotation_then_quantize_amd as rtq
        need = {"glu": lambda: rtq.fp8_glu_workspace(case["T"], case["N"], case["K"]),
                "norm_back": lambda: rtq.rmsnorm_backward_workspace(case["T"], case["d"])}.get(op)
        if need is not None:
            s["workspace"] = empty(need(), dtype=torch.uint8)
        if op == "clip":
            s["list"] = rtq.TensorList(s["grads"], s["outs"])
            s["workspace"] = empty(rtq.grad_norm_workspace(s["list"]), dtype=torch.uint8)
    return s


# ------------------------------------------------------------------ one pass

def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_plain(s):
    case = s["case"]
    op = case["op"]
    if op == "norm":
        h = (s["x"].float() + s["r"].float()).to(s["r"].dtype) if "r" in s else s["x"]
        f = h.float()
        n = f * torch.rsqrt((f * f).mean(1, keepdim=True) + EPS) * s["gamma"].float()
        out = _out(n, E4M3) if case["out"] == "codes" else {"y": n.to(s["x"].dtype)}
        return {"h": h, **out} if "r" in s else out
    if op == "norm_back":
        f, a = s["h"].float(), s["dn"].float() * s["gamma"].float()
        rho = torch.rsqrt((f * f).mean(1, keepdim=True) + EPS)
        dh = rho * a - f * (rho * rho * rho * (a * f).mean(1, keepdim=True))
        if "dr" in s:
            dh = dh + s["dr"].float()
        return {"dh": dh.to(s["h"].dtype), "dgamma": (s["dn"].float() * f * rho).sum(0)}
    if op == "glu":
        h = _rows(s["x"], s["x_scale"]) @ _blocks(s["w"], s["w_scale"]).T
        N = case["N"]
        y = _act(h[:, :N], case["act"]) * h[:, N:]
        out = _out(y, E4M3) if case["out"] == "codes" else {"y": y.bfloat16()}
        return {**out, "kept": _out(h, E4M3)} if case["keep"] else out
    if op == "glu_back":
        h = _rows(s["h"], s["h_scale"])
        N, dy = case["N"], s["dy"].float()
        dh = torch.cat([dy * h[:, N:] * _act_slope(h[:, :N], case["act"]), dy * _act(h[:, :N], case["act"])], 1)
        return {"dh": dh.bfloat16(), **_out(dh, s["fmt"])}
    norm = torch.stack([x.float().square().sum(dtype=torch.float64) for x in s["grads"]]).sum().sqrt().float()
    c = torch.clamp(case["most"] / (norm + 1e-6), max=1.0)
    return {"norm": norm.view(1), "grads": [(x.float() * c).to(x.dtype) for x in s["grads"]]}


def _run_own(s):
    import rotation_then_quantize_amd as rtq
    case = s["case"]
    op = case["op"]
    if op == "norm":
        rtq.rmsnorm_forward(s["x"], s["gamma"], EPS, residual=s.get("r"), h=s.get("h"), codes=s.get("codes"),
                            scale=s.get("scale"), y=s.get("y"))
        return {k: s[k] for k in ("h", "codes", "scale", "y") if k in s}
    if op == "norm_back":
        rtq.rmsnorm_backward(s["dn"], s["h"], s["gamma"], EPS, s["dh"], dgamma=s["dgamma"], dresidual=s.get("dr"),
                             workspace=s["workspace"])
        return {"dh": s["dh"], "dgamma": s["dgamma"]}
    act = {"gelu_tanh": rtq.RTQ_ACT_GELU_TANH, "gelu": rtq.RTQ_ACT_GELU, "silu": rtq.RTQ_ACT_SILU}.get(case.get("act"))
    if op == "glu":
        rtq.fp8_glu(s["x"], s["x_scale"], s["w"], s["w_scale"], act, y=s.get("y"), y_codes=s.get("codes"),
                    y_scale=s.get("scale"), h_codes=s.get("h_codes"), h_scale=s.get("h_scale"), workspace=s["workspace"])
        out = {"codes": s["codes"], "scale": s["scale"].to(E8M0)} if case["out"] == "codes" else {"y": s["y"]}
        return {**out, "kept": {"codes": s["h_codes"], "scale": s["h_scale"].to(E8M0)}} if case["keep"] else out
    if op == "glu_back":
        rtq.glu_fp8_backward(s["dy"], s["h"], s["h_scale"], act, dh=s["dh"], dh_codes=s["codes"], dh_scale=s["scale"])
        return {"dh": s["dh"], "codes": s["codes"], "scale": s["scale"]}
    rtq.grad_norm(s["list"], s["norm"], workspace=s["workspace"])
    rtq.grad_clip(s["list"], s["norm"], case["most"])
    return {"norm": s["norm"], "grads": s["outs"]}


def work(case):
    op = case["op"]
    if op in ("norm", "norm_back"):
        T, d, size = case["T"], case["d"], {"bf16": 2, "f32": 4}
        xb, rb, gb = size[case["x"]], size.get(case["r"], 0), size[case["gamma"]]
        if op == "norm":
            out = T * d + T * _groups(d) if case["out"] == "codes" else xb * T * d
            return {"bytes": (xb + 2 * rb) * T * d + gb * d + out, "flops": 8 * T * d}
        hb = rb or xb
        return {"bytes": (xb + 2 * hb + rb) * T * d + gb * d + 4 * d, "flops": 14 * T * d}
    if op == "glu":
        T, K, N = case["T"], case["K"], case["N"]
        sb = 1 if case["scale"] == "e8m0" else 4
        b = T * K + sb * T * _groups(K) + 2 * N * K + sb * _groups(2 * N) * _groups(K)
        b += T * N + sb * T * _groups(N) if case["out"] == "codes" else 2 * T * N
        if case["keep"]:
            b += 2 * T * N + sb * T * _groups(2 * N)
        return {"bytes": b, "flops": 4 * T * N * K}
    if op == "glu_back":
        T, N = case["T"], case["N"]
        return {"bytes": T * N * (2 + 2 + 4 + 2) + 2 * T * _groups(2 * N), "flops": 15 * T * N}
    n = case["blocks"] * (case["d"] + 3 * case["d"] * case["N"])
    return {"bytes": 2 * n * (4 if case["type"] == "f32" else 2), "flops": 3 * n}


# ------------------------------------------------------------------ the definition, in 64 bits

def _exact_codes(x, fmt):
    """Codes' values and scales of row groups, from the definition."""
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
    return {"codes": codes, "scale": scale}


def _exact_matrix(codes, scale, row_block):
    values = codes.to(torch.float64, copy=True)
    s = scale.double()
    if row_block == 1:
        for j in range(s.shape[0]):
            values[:, j * BLOCK:(j + 1) * BLOCK] *= s[j][:, None]
        return values
    for j in range(s.shape[1]):
        values[:, j * BLOCK:(j + 1) * BLOCK] *= s[:, j].repeat_interleave(row_block)[:values.shape[0], None]
    return values


def _exact_act(h, act):
    if act == "silu":
        return h * torch.sigmoid(h)
    if act == "gelu":
        return h * 0.5 * torch.special.erfc(-h / math.sqrt(2.0))
    return h * torch.sigmoid(math.sqrt(8.0 / math.pi) * (h + 0.044715 * h ** 3))


def _exact_norm(h, gamma):
    return h / torch.sqrt(h.square().mean(1, keepdim=True) + EPS) * gamma


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        # the residual stream is the rounded sum, and the norm is taken of what it holds
        h = s["x"].double()
        if "r" in s:
            h = (h + s["r"].double()).to(s["r"].dtype).double()
        n = _exact_norm(h, s["gamma"].double())
        out = _exact_codes(n, E4M3) if case["out"] == "codes" else {"y": n}
        return {"h": h, **out} if "r" in s else out
    if op == "norm_back":
        with torch.enable_grad():
            h, gamma = s["h"].double().requires_grad_(True), s["gamma"].double().requires_grad_(True)
            dh, dgamma = torch.autograd.grad(_exact_norm(h, gamma), (h, gamma), s["dn"].double())
        return {"dh": dh + s["dr"].double() if "dr" in s else dh, "dgamma": dgamma}
    if op == "glu":
        N = case["N"]
        h = torch.matmul(_exact_matrix(s["x"], s["x_scale"], 1), _exact_matrix(s["w"], s["w_scale"], BLOCK).t().contiguous())
        y = _exact_act(h[:, :N], case["act"]) * h[:, N:]
        out = _exact_codes(y, E4M3) if case["out"] == "codes" else {"y": y}
        return {**out, "kept": _exact_codes(h, E4M3)} if case["keep"] else out
    if op == "glu_back":
        N = case["N"]
        with torch.enable_grad():
            h = _exact_matrix(s["h"], s["h_scale"], 1).requires_grad_(True)
            (dh,) = torch.autograd.grad(_exact_act(h[:, :N], case["act"]) * h[:, N:], h, s["dy"].double())
        return {"dh": dh, **_exact_codes(dh, s["fmt"])}
    norm = torch.sqrt(sum(x.double().square().sum() for x in s["grads"]))
    c = min(1.0, case["most"] / (float(norm) + 1e-6))
    return {"norm": norm.view(1), "grads": [x.double() * c for x in s["grads"]]}
