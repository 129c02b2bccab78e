"""Cases that measure products with an epilogue, their backward pass, and dropout.

A case is one pass through one operator; `op` names it:

  fp8-forward   a per-tensor FP8 linear with h = x W^T + bias, y = residual +
                drop(act(h)); h is kept for the backward pass where act needs it
  fp8-backward  its gradients from gy: gh = gy drop' act'(h), then x's, W's and
                the bias's gradient
  mx-forward    the same linear with MXFP4 operands, in training
  mx-backward   its gradients
  apply         the same linear in serving: a few new tokens, the weight held
                as MXFP4
  dropout       y = residual + drop(x), and x's gradient

drop keeps element (m, n) of an M x N matrix where 16 bits of a counter-based
generator (Philox 4x32 with 10 rounds: Salmon, Moraes, Dror, Shaw, "Parallel
random numbers: as easy as 1, 2, 3", 2011) are at least t = round(65536 p), and
scales it by 65536 / (65536 - t).  Key: rng[0].  Counter: the group of eight
columns m ceil(N / 8) + n / 8 in its low 64 bits, rng[1] in its high ones;
element n takes half n % 2 (low first) of output word n % 8 / 2.

With `own` false run() computes the operator with elementary torch operations
in 32 bits; with `own` true it calls fp8_scaled_gemm_amd.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BYTES = {"bf16": 2, "f16": 2, "f32": 4}
ACTS = ("none", "relu", "silu", "gelu", "gelu_tanh")


def listed():
    return [
        # the small layer with a biased activation: launches count
        {"name": "forward-small", "op": "fp8-forward", "M": 64, "N": 256, "K": 128, "type": "bf16", "bias": "bf16",
         "act": "gelu_tanh", "residual": False, "p": 0.0},
        # the MLP block's first layer, h kept for its backward pass
        {"name": "forward-mlp-up", "op": "fp8-forward", "M": 8192, "N": 14336, "K": 4096, "type": "bf16",
         "bias": "bf16", "act": "gelu", "residual": False, "p": 0.0},
        # the MLP block's last layer: dropout, then onto the residual stream
        {"name": "forward-mlp-down", "op": "fp8-forward", "M": 8192, "N": 4096, "K": 14336, "type": "bf16",
         "bias": "f32", "act": "none", "residual": True, "p": 0.1},
        {"name": "backward-small", "op": "fp8-backward", "M": 64, "N": 256, "K": 128, "type": "f16", "bias": "f32",
         "act": "gelu_tanh", "p": 0.0},
        {"name": "backward-mlp-up", "op": "fp8-backward", "M": 8192, "N": 14336, "K": 4096, "type": "bf16",
         "bias": "bf16", "act": "gelu", "p": 0.0},
        # a ragged batch in full precision
        {"name": "mx-forward-ragged", "op": "mx-forward", "M": 1000, "N": 1031, "K": 2085, "type": "f32",
         "bias": "f32", "act": "silu", "residual": True, "p": 0.1, "rule": "fit"},
        {"name": "mx-backward-square", "op": "mx-backward", "M": 4096, "N": 4096, "K": 4096, "type": "bf16",
         "bias": "bf16", "act": "relu", "p": 0.1, "rule": "floor"},
        # one token through the MLP block's first layer: latency and the weight's bytes
        {"name": "apply-1-token", "op": "apply", "M": 1, "N": 14336, "K": 4096, "type": "bf16", "bias": "bf16",
         "act": "gelu", "residual": False, "p": 0.0, "rule": "floor"},
        # a small serving batch through its last layer
        {"name": "apply-24-tokens", "op": "apply", "M": 24, "N": 4096, "K": 14336, "type": "f16", "bias": "f16",
         "act": "none", "residual": True, "p": 0.0, "rule": "fit"},
        # a few rows of an odd width
        {"name": "dropout-small", "op": "dropout", "M": 5, "N": 1027, "type": "f32", "residual": True, "p": 0.5},
        # the MLP block's residual stream
        {"name": "dropout-mlp", "op": "dropout", "M": 8192, "N": 4096, "type": "bf16", "residual": True, "p": 0.1},
        # a ragged batch of the block's inner width
        {"name": "dropout-wide", "op": "dropout", "M": 1000, "N": 14333, "type": "f16", "residual": False, "p": 0.25},
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["fp8-forward", "fp8-backward", "mx-forward", "mx-backward", "apply", "dropout"])
    case = {"op": op, "p": rng.choice([0.0, 0.1, 0.5])}
    if op.startswith("fp8"):  # sizes in multiples of 16
        case |= {"type": rng.choice(["bf16", "f16"]), "M": 16 * _spread(rng, 1, 512), "N": 16 * _spread(rng, 1, 896),
                 "K": 16 * _spread(rng, 1, 256)}
    else:
        case["type"] = rng.choice(["bf16", "f16", "f32"])
    if op.startswith("mx"):
        case |= {"M": _spread(rng, 1, 4096), "N": _spread(rng, 1, 8192), "K": _spread(rng, 1, 4096)}
    elif op == "apply":
        case |= {"M": _spread(rng, 1, 64), "N": _spread(rng, 32, 14336), "K": _spread(rng, 32, 14336), "p": 0.0}
    elif op == "dropout":
        case |= {"M": _spread(rng, 1, 8192), "N": _spread(rng, 1, 14336), "p": rng.choice([0.1, 0.25, 0.5])}
    if op != "dropout":
        case |= {"act": rng.choice(ACTS), "bias": rng.choice([case["type"], "f32", "none"])}
        if case["bias"] == "none" and op.endswith("backward"):
            case["bias"] = "f32"
    if op not in ("fp8-backward", "mx-backward"):
        case["residual"] = rng.random() < 0.5
    if op in ("mx-forward", "mx-backward", "apply"):
        case["rule"] = rng.choice(["floor", "fit"])
    return case


# ------------------------------------------------------------------- inputs

def _normal(gen, shape, sigma, dtype, outliers=0.0):
    x = torch.randn(shape, generator=gen, device="cuda") * sigma
    if outliers:
        x = torch.where(torch.rand(shape, generator=gen, device="cuda") < outliers, 50 * x, x)
    return x.to(dtype)


def _inputs(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op, t, M, N, K = case["op"], DTYPES[case["type"]], case["M"], case["N"], case.get("K")
    s = {}
    if op != "dropout":
        s |= {"x": _normal(gen, (M, K), 1.0, t, 1e-3), "w": _normal(gen, (N, K), 0.02, t)}
        if case["bias"] != "none":
            s["bias"] = _normal(gen, (N,), 0.5, DTYPES[case["bias"]])
    else:
        s["x"] = _normal(gen, (M, N), 1.0, t)
    if case.get("residual"):
        s["residual"] = _normal(gen, (M, N), 1.0, t)
    if op.endswith("backward"):
        s["h"] = _normal(gen, (M, N), 1.5, t)
    if op.endswith("backward") or op == "dropout":
        # fp16 gradients come with a loss scale
        s["gy"] = _normal(gen, (M, N), 1e-4 * (1024 if case["type"] == "f16" else 1), t)
    if case["p"] > 0:
        s["rng"] = torch.randint(-2 ** 63, 2 ** 63 - 1, (2,), generator=gen, device="cuda", dtype=torch.int64)
    return s


def prepare(case, seed):
    state = {"case": case, **_inputs(case, seed)}
    op = case["op"]
    if own:
        state["own"] = _buffers(state)
    elif op == "apply":  # the weight is held as MXFP4: the values it stands for
        state["w_val"] = _fp4_values(state["w"].float(), case["rule"])
    elif op == "mx-backward":  # and so is what a forward pass left
        state["x_val"] = _fp4_values(state["x"].float().t().contiguous(), case["rule"])
        state["w_val"] = _fp4_values(state["w"].float().t().contiguous(), case["rule"])
    elif op == "fp8-backward":
        state["x_val"], state["x_inv"] = _fp8_values(state["x"].float(), 448.0, 3, -6)
        state["w_val"], state["w_inv"] = _fp8_values(state["w"].float(), 448.0, 3, -6)
    return state


# --------------------------------------------------------------- plain forms

def _fp8_values(x, top, mantissa, emin):
    """The values of x's FP8 codes before their scale (x in fp32), and the
    inverse scale in 64 bits: e4m3 (448, 3 bits, 2^-6) or e5m2 (57344, 2, 2^-14)."""
    amax = x.abs().amax().double().clamp(min=1e-12)
    scale = top / amax
    v = (x * scale.float()).clamp(-top, top)
    a = v.abs()
    _, ex = torch.frexp(a)
    step = torch.ldexp(torch.ones_like(a), (ex - 1).clamp(min=emin) - mantissa)
    return torch.copysign((torch.round(a / step) * step).clamp(max=top), v), 1 / scale


def _fp4_values(x, rule):
    """The values of x's MXFP4 codes along its rows (x in fp32): blocks of 32
    with one power of two each."""
    rows, cols = x.shape
    v = torch.nn.functional.pad(x, (0, -cols % 32)).reshape(rows, -1, 32)
    amax = v.abs().amax(dim=-1, keepdim=True)
    mant, ex = torch.frexp(amax)  # amax = mant 2^ex, mant in [1/2, 1)
    e = ex - 3
    if rule == "fit":
        e = e + (mant > 0.75).to(e.dtype)
    e = torch.where(amax > 0, e, torch.full_like(e, -127)).clamp(-127, 127)
    # two factors: the whole power may lie outside fp32's normal range
    v = torch.ldexp(torch.ldexp(v, -(e // 2)), -(e - e // 2))
    a = v.abs().clamp(max=6.0)
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    q = torch.copysign((torch.round(a / step) * step).clamp(max=6.0), v)  # torch.round: ties to even
    return torch.ldexp(torch.ldexp(q, e // 2), e - e // 2).reshape(rows, -1)[:, :cols]


def _mul32(a, m):
    """High and low word of a 32-bit value times a 32-bit constant (int64)."""
    prod = a * m  # wraps; its 64 bits are the product's
    return (prod >> 32) & 0xFFFFFFFF, prod & 0xFFFFFFFF


def _dropped(a, s):
    """drop(a), a in fp32."""
    p = s["case"]["p"]
    if p == 0:
        return a
    rows, cols = a.shape
    t = round(65536 * p)
    mask = 0xFFFFFFFF
    g = torch.arange(rows * -(-cols // 8), device=a.device)
    k0, k1 = s["rng"][0] & mask, (s["rng"][0] >> 32) & mask
    c = [g & mask, g >> 32, (s["rng"][1] & mask).expand_as(g), ((s["rng"][1] >> 32) & mask).expand_as(g)]
    for _ in range(10):
        hi0, lo0 = _mul32(c[0], 0xD2511F53)
        hi1, lo1 = _mul32(c[2], 0xCD9E8D57)
        c = [hi1 ^ c[1] ^ k0, lo1, hi0 ^ c[3] ^ k1, lo0]
        k0, k1 = (k0 + 0x9E3779B9) & mask, (k1 + 0xBB67AE85) & mask
    u = torch.stack([h for w in c for h in (w & 0xFFFF, w >> 16)], dim=1)
    u = u.reshape(rows, -1)[:, :cols]
    return torch.where(u >= t, a * (65536 / (65536 - t)), torch.zeros_like(a))


def _act(h, act):
    if act == "relu":
        return h.clamp(min=0)
    if act == "silu":
        return h / (1 + torch.exp(-h))
    if act == "gelu":
        return 0.5 * h * torch.erfc(-h * math.sqrt(0.5))
    if act == "gelu_tanh":
        return h / (1 + torch.exp(-2 * math.sqrt(2 / math.pi) * (h + 0.044715 * h * h * h)))
    return h


def _slope(h, act):
    """act'(h)"""
    if act == "relu":
        return (h > 0).to(h.dtype)
    if act == "silu":
        s = 1 / (1 + torch.exp(-h))
        return s * (1 + h * (1 - s))
    if act == "gelu":
        return 0.5 * torch.erfc(-h * math.sqrt(0.5)) + h * torch.exp(-0.5 * h * h) / math.sqrt(2 * math.pi)
    if act == "gelu_tanh":
        c = 2 * math.sqrt(2 / math.pi)
        s = 1 / (1 + torch.exp(-c * (h + 0.044715 * h * h * h)))
        return s + h * s * (1 - s) * c * (1 + 3 * 0.044715 * h * h)
    return torch.ones_like(h)


def _epilogue(prod, s):
    c = s["case"]
    t = DTYPES[c["type"]]
    h = prod + s["bias"].float() if "bias" in s else prod
    y = _dropped(_act(h, c["act"]), s)
    if "residual" in s:
        y = y + s["residual"].float()
    out = {"y": y.to(t)}
    if c["act"] != "none" and c["op"] != "apply":
        out["h"] = h.to(t)
    return out


def _plain(s):
    c = s["case"]
    op, t = c["op"], DTYPES[c["type"]]
    if op == "dropout":
        y = _dropped(s["x"].float(), s)
        if "residual" in s:
            y = y + s["residual"].float()
        return {"y": y.to(t), "gx": _dropped(s["gy"].float(), s).to(t)}
    if op == "fp8-forward":
        x, xi = _fp8_values(s["x"].float(), 448.0, 3, -6)
        w, wi = _fp8_values(s["w"].float(), 448.0, 3, -6)
        return _epilogue((x @ w.t()) * (xi * wi).float(), s)
    if op == "mx-forward":
        return _epilogue(_fp4_values(s["x"].float(), c["rule"]) @ _fp4_values(s["w"].float(), c["rule"]).t(), s)
    if op == "apply":
        return _epilogue(_fp4_values(s["x"].float(), c["rule"]) @ s["w_val"].t(), s)
    gh = _dropped(s["gy"].float(), s) * _slope(s["h"].float(), c["act"])
    gb = gh.sum(dim=0).to(DTYPES[c["bias"]])
    gh = gh.to(t).float()  # the products' operand is cast from the layer's type
    if op == "fp8-backward":
        g, gi = _fp8_values(gh, 57344.0, 2, -14)
        return {"gx": ((g @ s["w_val"]) * (gi * s["w_inv"]).float()).to(t),
                "gw": ((g.t() @ s["x_val"]) * (gi * s["x_inv"]).float()).to(t), "gb": gb}
    return {"gx": (_fp4_values(gh, c["rule"]) @ s["w_val"].t()).to(t),
            "gw": (_fp4_values(gh.t().contiguous(), c["rule"]) @ s["x_val"].t()).to(t), "gb": gb}


# ------------------------------------------------- the framework's operators

def _buffers(s):
    """What a program that uses the operators keeps between calls: packed
    weights, what a forward pass left, workspaces, the tensors that results go to."""
    import fp8_scaled_gemm_amd as F
    c = s["case"]
    op, M, N, K, t = c["op"], c["M"], c["N"], c.get("K"), DTYPES[c["type"]]
    rule = F.MX_FIT if c.get("rule") == "fit" else F.MX_FLOOR

    def empty(*shape, dtype=t):
        return torch.empty(shape, dtype=dtype, device="cuda")
    h = {"F": F, "rule": rule, "rng": s.get("rng")}
    if op == "dropout":
        return h | {"y": empty(M, N), "gx": empty(M, N)}
    h["act"] = getattr(F, "ACT_" + c["act"].upper())
    if op.endswith("forward") or op == "apply":
        h["y"] = empty(M, N)
        if c["act"] != "none" and op != "apply":
            h["h"] = empty(M, N)
    else:
        h |= {"gx": empty(M, K), "gw": empty(N, K), "gb": empty(N, dtype=DTYPES[c["bias"]]), "gh": empty(M, N),
              "part": empty(F.epilogue_workspace_len(M, N), dtype=torch.float32)}
    if op.startswith("fp8"):
        xt, wt, gt = F.fp8_linear_copies(M, N, K)
        h["saved"] = F.LinearSaved(M, N, K, x_transposed=xt, w_transposed=wt)
        if op == "fp8-backward":
            h["ws"] = F.LinearBwdWs(M, N, transposed=gt)
            F.fp8_scaled_linear_fwd_epilogue(s["x"], s["w"], h["saved"], empty(M, N))
    elif op == "apply":
        h |= {"w": F.Mxfp4(N, K), "ws": F.Mxfp4(M, K)}
        F.mxfp4_quantize(s["w"], h["w"], rule=rule)
    else:
        h |= {"ws": F.Mxfp4LinearWs(M, N, K), "saved": F.Mxfp4LinearSaved(M, N, K)}
        if op == "mx-backward":
            F.mxfp4_linear_fwd(s["x"], s["w"], h["ws"], h["saved"], empty(M, N), rule=rule)
    return h


def run(s):
    if not own:
        return _plain(s)
    h, c = s["own"], s["case"]
    F, op, p, rng, rule = h["F"], c["op"], c["p"], h["rng"], h["rule"]
    if op == "dropout":
        F.dropout_fwd(s["x"], p, rng, h["y"], residual=s.get("residual"))
        F.dropout_bwd(s["gy"], p, rng, h["gx"])
        return {"y": h["y"], "gx": h["gx"]}
    if op.endswith("backward"):
        kw = {"gh": h["gh"], "gb": h["gb"], "pre": s["h"], "act": h["act"], "p": p, "rng": rng, "part": h["part"]}
        if op == "fp8-backward":
            F.fp8_scaled_linear_bwd_epilogue(s["gy"], h["saved"], h["ws"], h["gx"], h["gw"], **kw)
        else:
            F.mxfp4_linear_bwd_epilogue(s["gy"], h["ws"], h["saved"], h["gx"], h["gw"], rule=rule, **kw)
        return {"gx": h["gx"], "gw": h["gw"], "gb": h["gb"]}
    kw = {"bias": s.get("bias"), "act": h["act"], "residual": s.get("residual"), "p": p, "rng": rng}
    if op == "apply":
        F.mxfp4_linear_apply_epilogue(s["x"], h["w"], h["y"], h["ws"], rule=rule, **kw)
        return {"y": h["y"]}
    pre = h.get("h")
    if op == "fp8-forward":
        F.fp8_scaled_linear_fwd_epilogue(s["x"], s["w"], h["saved"], h["y"], pre=pre, **kw)
    else:
        F.mxfp4_linear_fwd_epilogue(s["x"], s["w"], h["ws"], h["saved"], h["y"], pre=pre, rule=rule, **kw)
    return {"y": h["y"]} if pre is None else {"y": h["y"], "h": pre}


# ------------------------------------------------------------ what it has to do

def work(case):
    op, M, N, K, e = case["op"], case["M"], case["N"], case.get("K"), BYTES[case["type"]]
    if op == "dropout":  # x, gy and the residual in; y and gx out
        return {"bytes": M * N * e * (4 + case["residual"]), "flops": 4 * M * N}
    b = N * BYTES.get(case["bias"], 0)
    kept = case["act"] != "none"
    if op.endswith("forward"):  # x, W, the residual in; y and h out
        return {"bytes": (M * K + N * K + M * N * (1 + kept + case["residual"])) * e + b, "flops": 2 * M * N * K}
    if op == "apply":
        return {"bytes": (M * K + M * N * (1 + case["residual"])) * e + N * K * 17 / 32 + b, "flops": 2 * M * N * K}
    # gy and h in, what the forward left of x and W in, the gradients out
    code = 1 if op == "fp8-backward" else 17 / 32
    return {"bytes": (M * N * (1 + kept) + M * K + N * K) * e + (M + N) * K * code + b, "flops": 4 * M * N * K}


# -------------------------------------------------------------- in 64 bits

def _exact_fp8(x, e5m2):
    """x's FP8 values times the inverse scale, in 64 bits: the cast takes
    fl32(x fl32(scale)), rounds it to nearest even and saturates."""
    top, bits, low = (57344.0, 2, 2.0 ** -14) if e5m2 else (448.0, 3, 2.0 ** -6)
    scale = top / max(float(x.abs().max()), 1e-12)
    v = (x.float() * torch.tensor(scale, dtype=torch.float32, device=x.device)).double()
    ulp = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=low))) - bits)
    return (torch.round(v / ulp) * ulp).clamp(-top, top) * (1.0 / scale)


def _exact_fp4(x, rule):
    """MXFP4 along x's rows from the definition, in 64 bits: the nearest of the
    eight magnitudes, a tie going to the even code."""
    rows, cols = x.shape
    n = -(-cols // 32)
    v = torch.zeros(rows, 32 * n, dtype=torch.float64, device=x.device)
    v[:, :cols] = x
    v = v.view(rows * n, 32)
    top = v.abs().max(dim=1, keepdim=True).values
    safe = torch.where(top > 0, top, torch.ones_like(top))
    if rule == "fit":
        p = torch.exp2(torch.ceil(torch.log2(safe / 6)))  # next to the border log2 may be a step off
        p = torch.where(6 * p < safe, 2 * p, torch.where(3 * p >= safe, p / 2, p))
    else:
        p = torch.exp2(torch.floor(torch.log2(safe)))
        p = torch.where(p > safe, p / 2, torch.where(2 * p <= safe, 2 * p, p)) / 4
    p = torch.where(top > 0, p, torch.full_like(p, 2.0 ** -127)).clamp(min=2.0 ** -127)
    mag = torch.tensor((0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0), dtype=torch.float64, device=x.device)
    a = (v / p).abs().clamp(max=6.0)
    hi = torch.searchsorted(mag, a).clamp(max=7)
    lo = (hi - 1).clamp(min=0)
    up, down = mag[hi] - a, a - mag[lo]
    code = torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    return (torch.sign(v) * mag[code] * p).view(rows, 32 * n)[:, :cols]


def _exact_keep(rng, rows, cols, p):
    """1 / (the share kept) where an element is kept, 0 elsewhere, in 64 bits;
    products of 32-bit words from 16-bit pieces."""
    t = int(65536 * p + 0.5)

    def words(v):
        v = int(v) % 2 ** 64
        return v % 2 ** 32, v // 2 ** 32

    def times(c, m):
        low = (c % 65536) * m  # below 2^48
        rest = (c // 65536) * m + low // 65536
        return rest // 65536, (rest % 65536) * 65536 + low % 65536
    (ka, kb), (oa, ob) = words(rng[0]), words(rng[1])
    groups = (cols + 7) // 8
    n = torch.arange(rows, device=rng.device)[:, None] * groups + torch.arange(groups, device=rng.device)
    c0, c1, c2, c3 = n % 2 ** 32, n // 2 ** 32, torch.full_like(n, oa), torch.full_like(n, ob)
    for i in range(10):
        ha, la = times(c0, 0xD2511F53)
        hb, lb = times(c2, 0xCD9E8D57)
        c0, c1, c2, c3 = hb ^ c1 ^ ((ka + i * 0x9E3779B9) % 2 ** 32), lb, ha ^ c3 ^ ((kb + i * 0xBB67AE85) % 2 ** 32), la
    keep = torch.empty(rows, groups, 8, dtype=torch.float64, device=rng.device)
    for j, w in enumerate((c0, c1, c2, c3)):
        keep[:, :, 2 * j] = (w % 65536 >= t).double()
        keep[:, :, 2 * j + 1] = (w // 65536 >= t).double()
    return keep.reshape(rows, 8 * groups)[:, :cols] * (65536 / (65536 - t))


def _exact_act(h, act):
    """act(h) and its derivative"""
    if act == "relu":
        return torch.relu(h), torch.heaviside(h, torch.zeros_like(h))
    if act == "silu":
        s = torch.sigmoid(h)
        return h * s, s + h * s * torch.sigmoid(-h)
    if act == "gelu":
        cdf = torch.special.erfc(-h / 2 ** 0.5) / 2
        return h * cdf, cdf + h * torch.exp(-h ** 2 / 2) / (2 * math.pi) ** 0.5
    if act == "gelu_tanh":
        k = (2 / math.pi) ** 0.5
        s = torch.sigmoid(2 * k * (h + 0.044715 * h ** 3))
        return h * s, s + h * s * (1 - s) * 2 * k * (1 + 0.134145 * h ** 2)
    return h, torch.ones_like(h)


def exact(case, seed):
    s = _inputs(case, seed)
    d = {k: v.double() for k, v in s.items() if k != "rng"}
    op, M, N, rule = case["op"], case["M"], case["N"], case.get("rule")
    keep = _exact_keep(s["rng"], M, N, case["p"]) if case["p"] > 0 else 1.0
    if op == "dropout":
        return {"y": d["x"] * keep + d.get("residual", 0.0), "gx": d["gy"] * keep}
    if op.endswith("backward"):
        gh = d["gy"] * keep * _exact_act(d["h"], case["act"])[1]
        gb = torch.sum(gh, dim=0)
        gh = gh.to(DTYPES[case["type"]]).double()
        if op == "fp8-backward":
            q = _exact_fp8(gh, True)
            return {"gx": torch.mm(q, _exact_fp8(d["w"], False)), "gw": torch.mm(q.t(), _exact_fp8(d["x"], False)),
                    "gb": gb}
        return {"gx": torch.mm(_exact_fp4(gh, rule), _exact_fp4(d["w"].t(), rule).t()),
                "gw": torch.mm(_exact_fp4(gh.t(), rule), _exact_fp4(d["x"].t(), rule).t()), "gb": gb}
    if op == "fp8-forward":
        h = torch.mm(_exact_fp8(d["x"], False), _exact_fp8(d["w"], False).t())
    else:
        h = torch.mm(_exact_fp4(d["x"], rule), _exact_fp4(d["w"], rule).t())
    h = h + d.get("bias", 0.0)
    y = _exact_act(h, case["act"])[0] * keep + d.get("residual", 0.0)
    return {"y": y, "h": h} if case["act"] != "none" and op != "apply" else {"y": y}
