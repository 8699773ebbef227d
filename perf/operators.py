"""The operators around the FP4 products of a transformer's feed-forward block, as cases to
measure: layer norm (forward, backward), the gated GEMM (dense, from BF16 activations, by
experts), the activation's backward pass, and the GEMM epilogue with a residual.

Where ``own`` is false, ``run`` computes them from elementary torch operations in 32 bits;
where it is true, it calls the library."""
import math

import torch

own = False

NVFP4, MXFP4 = 0, 1
ACTS = {"none": 0, "relu": 1, "silu": 2, "gelu": 3, "gelu_tanh": 4}
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-5


# ---------------------------------------------------------------- cases
def listed():
    return [
        # one decode step of 16 sequences: the norm before the feed-forward block (latency)
        dict(name="norm decode", op="norm", M=16, N=8192, dt="bf16"),
        # the same norm over a prompt of 8192 tokens
        dict(name="norm prefill", op="norm", M=8192, N=8192, dt="bf16"),
        # FP32 training on a ragged batch, rows that are no multiple of a warp's chunk count
        dict(name="norm grad fp32", op="norm_grad", M=4095, N=2880, dt="f32", res=False),
        # BF16 training, with the gradient that comes down the residual branch added
        dict(name="norm grad bf16", op="norm_grad", M=16384, N=8192, dt="bf16", res=True),
        # one decode step: BF16 activations quantized in the call, the weights streamed once
        dict(name="gated decode", op="gated_x", M=16, F=28672, K=8192, act="silu", dt="bf16"),
        # a prompt through pre-quantized NVFP4 operands
        dict(name="gated prefill", op="gated", fmt=NVFP4, M=4096, F=28672, K=8192, act="silu", dt="bf16", save=False,
             bias=False),
        # training: both pre-activations are kept for the backward pass
        dict(name="gated train", op="gated", fmt=NVFP4, M=8192, F=4096, K=4096, act="gelu_tanh", dt="bf16", save=True,
             bias=False),
        # mixture of experts in MXFP4: 4096 tokens, 4 of 32 experts each, gate and up biases
        dict(name="gated experts", op="gated_experts", E=32, rows=16384, F=2880, K=2880, act="silu", dt="bf16",
             bias=True),
        # backward pass of the gated activation over a long batch
        dict(name="act grad gated", op="act_grad", M=4096, F=28672, act="silu", dt="bf16", gated=True, bias=False),
        # backward pass of a plain activation with the bias gradient, ragged FP32 batch
        dict(name="act grad bias", op="act_grad", M=1999, F=5760, act="gelu", dt="f32", gated=False, bias=True),
        # one token through the down projection, added to the residual stream
        dict(name="out one token", op="out", fmt=NVFP4, M=1, N=8192, K=28672, act="none", dt="bf16", bias=False,
             save=False),
        # a prompt through a projection with bias, activation and residual, pre-activation kept
        dict(name="out prefill", op="out", fmt=NVFP4, M=8192, N=8192, K=8192, act="gelu", dt="bf16", bias=True,
             save=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "norm_grad", "gated_x", "gated", "gated_experts", "act_grad", "out"])
    dt = rng.choice(["bf16", "bf16", "f32"])
    act = rng.choice(["relu", "silu", "gelu", "gelu_tanh"])
    if op in ("norm", "norm_grad", "act_grad"):
        n = _log(rng, 32, 16384)
        m = min(_log(rng, 1, 16384), (1 << 26) // n)
        if op == "norm":
            return dict(op=op, M=m, N=n, dt=dt)
        if op == "norm_grad":
            return dict(op=op, M=m, N=n, dt=dt, res=rng.random() < 0.5)
        return dict(op=op, M=m, F=n, act=act, dt=dt, gated=rng.random() < 0.5, bias=rng.random() < 0.5)
    k = 32 * _log(rng, 2, 256)
    f = _log(rng, 64, 28672)
    if op == "gated_x":
        return dict(op=op, M=_log(rng, 1, 64), F=f, K=k, act=act, dt=dt)
    if op == "gated_experts":
        e = rng.choice([2, 5, 8, 32])
        return dict(op=op, E=e, rows=_log(rng, 1, 8192), F=_log(rng, 64, 2880), K=32 * rng.randint(2, 90),
                    act=act, dt=dt, bias=rng.random() < 0.5)
    m = min(_log(rng, 1, 8192), max(1, (1 << 38) // (f * k)))
    if op == "gated":
        return dict(op=op, fmt=rng.choice([NVFP4, MXFP4]), M=m, F=f, K=k, act=act, dt=dt, save=rng.random() < 0.5,
                    bias=rng.random() < 0.5)
    return dict(op=op, fmt=rng.choice([NVFP4, MXFP4]), M=m, N=f, K=k, act=rng.choice([act, "none"]), dt=dt,
                bias=rng.random() < 0.5, save=rng.random() < 0.5)


# ---------------------------------------------------------------- FP4 operands
def _codes(t):
    """E2M1 codes of scaled values: nearest grid value, ties to the even code, saturating at 6."""
    a = t.abs()
    c = (a > 0.25).to(torch.uint8)
    c += a >= 0.75
    c += a > 1.25
    c += a >= 1.75
    c += a > 2.5
    c += a >= 3.5
    c += a > 5.0
    return c + torch.signbit(t).to(torch.uint8) * 8


def _pack(c):
    return c[..., 0::2] | (c[..., 1::2] << 4)


def _blocks(x, fmt, g):
    """Scale bytes [rows, cols / block] and packed codes [rows, cols / 2] of FP32 values."""
    rows, cols = x.shape
    b = x.view(rows, -1, 16 if fmt == NVFP4 else 32)
    am = b.abs().amax(2)
    six = torch.full_like(g, 6.0)  # a device divisor: torch divides by it, as the definition does
    if fmt == NVFP4:
        sb = (am / six / g).clamp(max=448.0).to(torch.float8_e4m3fn)
        den = sb.float() * g
        mul = torch.where(den == 0, torch.zeros_like(den), torch.ones_like(den) / den)
        sb = sb.view(torch.uint8)
    else:
        m, e = torch.frexp(am / six)
        e = (e - 1 + (m >= 0.75).to(torch.int32) + 127).clamp(0, 254)
        e = torch.where(am == 0, torch.zeros_like(e), e)
        mul = torch.exp2((127 - e).double()).float()
        sb = e.to(torch.uint8)
    return sb, _pack(_codes((b * mul[..., None]).view(rows, cols)))


def _swizzle(sb):
    """Row-major scale bytes -> 128 x 4 atoms of 512 bytes (rows and columns padded with 0)."""
    r, c = sb.shape
    rp, cp = -(-r // 128) * 128, -(-c // 4) * 4
    p = torch.zeros(rp, cp, dtype=torch.uint8, device=sb.device)
    p[:r, :c] = sb
    return p.view(rp // 128, 4, 32, cp // 4, 4).permute(0, 3, 2, 1, 4).contiguous().view(-1)


def _unswizzle(buf, rows, cols):
    cp = -(-cols // 4) * 4
    return buf.view(-1, cp // 4, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(-1, cp)[:rows, :cols]


def _quantized(x, fmt):
    """What a program keeps of a quantized weight or activation: codes, scale atoms, scale."""
    g = torch.ones(1, device=x.device)
    if fmt == NVFP4:
        am = x.abs().amax().reshape(1)
        g = torch.where(am > 0, am / torch.full_like(am, 2688.0), torch.ones_like(am))
    sb, codes = _blocks(x, fmt, g)
    return dict(codes=codes, scales=_swizzle(sb), g=g)


GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)


def _scale_values(sb, fmt):
    return sb.view(torch.float8_e4m3fn).float() if fmt == NVFP4 else torch.exp2(sb.float() - 127.0)


def _values(codes, sb, fmt):
    """FP32 values of packed codes and row-major scale bytes (the tensor scale left out)."""
    grid = torch.tensor(GRID, device=codes.device)
    pairs = torch.stack((grid.repeat(16), grid.repeat_interleave(16)), 1)  # [byte, (low, high nibble)]
    v = pairs[codes.int()].view(*codes.shape[:-1], -1, 16 if fmt == NVFP4 else 32)
    return (v * _scale_values(sb.contiguous(), fmt)[..., None]).flatten(-2)


def _operand(q, rows, cols, fmt):
    return _values(q["codes"], _unswizzle(q["scales"], rows, cols // (16 if fmt == NVFP4 else 32)), fmt)


# ---------------------------------------------------------------- inputs
def _normal(gen, shape, std=1.0, dtype=torch.float32):
    return (torch.randn(*shape, generator=gen, device="cuda") * std).to(dtype)


def _activations(gen, shape, dtype=torch.float32):
    """N(0, 1) with a few outlier channels, as hidden states have them."""
    x = torch.randn(*shape, generator=gen, device="cuda")
    hot = torch.randint(0, shape[-1], (max(1, shape[-1] // 1000),), generator=gen, device="cuda")
    x[..., hot] *= 20.0
    return x.to(dtype)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case)
    op, dt = case["op"], DT[case["dt"]]

    def empty(*shape, dtype=dt):
        return torch.empty(*shape, dtype=dtype, device="cuda")

    if op in ("norm", "norm_grad"):
        m, n = case["M"], case["N"]
        s["x"] = (_activations(gen, (m, n)) + 0.25).to(dt)
        s["w"] = 1.0 + _normal(gen, (n,), 0.1)
        s["b"] = _normal(gen, (n,), 0.1)
        s["mean"], s["rstd"] = empty(m, dtype=torch.float32), empty(m, dtype=torch.float32)
        if op == "norm":
            s["y"] = empty(m, n)
        else:
            xd = s["x"].double()
            mean = xd.mean(1)
            s["mean"] = mean.float()
            s["rstd"] = ((xd - mean[:, None]).square().mean(1) + EPS).rsqrt().float()
            s["dy"] = _normal(gen, (m, n), 1.0, dt)
            s["dres"] = _normal(gen, (m, n), 1.0, dt) if case["res"] else None
            s["dx"], s["dw"], s["db"] = empty(m, n), empty(n, dtype=torch.float32), empty(n, dtype=torch.float32)
        return s
    if op == "act_grad":
        m, f = case["M"], case["F"]
        s["G"], s["dH"] = _normal(gen, (m, f), 1.5, dt), _normal(gen, (m, f), 1.0, dt)
        s["U"] = _normal(gen, (m, f), 1.5, dt) if case["gated"] else None
        w = 2 * f if case["gated"] else f
        s["dZ"] = empty(m, w)
        s["db"] = empty(w, dtype=torch.float32) if case["bias"] else None
        return s
    k = case["K"]
    if op == "gated_experts":
        e, rows, f = case["E"], case["rows"], case["F"]
        # rows routed to experts uniformly at random, sorted by expert
        cnt = torch.bincount(torch.randint(0, e, (rows,), generator=gen, device="cuda"), minlength=e)
        off = torch.zeros(e + 1, dtype=torch.int32, device="cuda")
        off[1:] = cnt.cumsum(0)
        s["offsets"], s["most"] = off, int(cnt.max())
        sb, s["codes"] = _blocks(_activations(gen, (rows, k)), MXFP4, torch.ones(1, device="cuda"))
        # each expert's scale rows start at a fresh 128-row block
        nb = (cnt + 127) // 128
        start = (nb.cumsum(0) - nb) * 128
        expert = torch.repeat_interleave(torch.arange(e, device="cuda"), cnt)
        at = start[expert] + torch.arange(rows, device="cuda") - off[expert]
        padded = torch.zeros((-(-rows // 128) + e) * 128, k // 32, dtype=torch.uint8, device="cuda")
        padded[at] = sb
        s["scales"], s["expert"], s["at"] = _swizzle(padded), expert, at
        for name in ("wg", "wu"):
            qs = [_quantized(_normal(gen, (f, k), 0.02), MXFP4) for _ in range(e)]
            s[name] = dict(codes=torch.stack([q["codes"] for q in qs]), scales=torch.cat([q["scales"] for q in qs]))
        s["bg"] = _normal(gen, (e, f), 0.5) if case["bias"] else None
        s["bu"] = _normal(gen, (e, f), 0.5) if case["bias"] else None
        s["H"] = empty(rows, f)
        return s
    fmt = case.get("fmt", NVFP4)
    m = case["M"]
    if op == "out":
        n = case["N"]
        s["a"] = _quantized(_activations(gen, (m, k)), fmt)
        s["w"] = _quantized(_normal(gen, (n, k), 0.02), fmt)
        s["res"] = _normal(gen, (m, n), 1.0, dt)
        s["bias_v"] = _normal(gen, (n,), 0.5) if case["bias"] else None
        s["D"], s["pre"] = empty(m, n), empty(m, n) if case["save"] else None
        return s
    f = case["F"]
    s["wg"], s["wu"] = (_quantized(_normal(gen, (f, k), 0.02), fmt) for _ in range(2))
    s["H"] = empty(m, f)
    if op == "gated_x":
        s["x"] = _activations(gen, (m, k), torch.bfloat16)
        nb = -(-(k // 16) // 4) * 4
        s["xc"] = empty(m, k // 2, dtype=torch.uint8)
        s["xs"] = empty(-(-m // 128) * 128 * nb, dtype=torch.uint8)
        s["xg"] = empty(1, dtype=torch.float32)
        return s
    s["a"] = _quantized(_activations(gen, (m, k)), fmt)
    s["bg"] = _normal(gen, (f,), 0.5) if case["bias"] else None
    s["bu"] = _normal(gen, (f,), 0.5) if case["bias"] else None
    s["G"], s["U"] = (empty(m, f), empty(m, f)) if case["save"] else (None, None)
    return s


# ---------------------------------------------------------------- the plain forms
def _sigmoid(x):
    return 1.0 / (1.0 + torch.exp(-x))


TANH_C, TANH_A = math.sqrt(2.0 / math.pi), 0.044715


def _act(x, act):
    if act == "none":
        return x
    if act == "relu":
        return torch.where(x > 0, x, torch.zeros_like(x))
    if act == "silu":
        return x * _sigmoid(x)
    if act == "gelu":
        return 0.5 * x * (1.0 + torch.erf(x * math.sqrt(0.5)))
    return x * _sigmoid(2.0 * TANH_C * (x + TANH_A * x * x * x))


def _act_slope(x, act):
    if act == "none":
        return torch.ones_like(x)
    if act == "relu":
        return (x > 0).to(x.dtype)
    if act == "silu":
        p = _sigmoid(x)
        return p * (1.0 + x * (1.0 - p))
    if act == "gelu":
        return 0.5 * (1.0 + torch.erf(x * math.sqrt(0.5))) + x * torch.exp(-0.5 * x * x) / math.sqrt(2.0 * math.pi)
    p = _sigmoid(2.0 * TANH_C * (x + TANH_A * x * x * x))
    return p * (1.0 + x * (1.0 - p) * 2.0 * TANH_C * (1.0 + 3.0 * TANH_A * x * x))


def _plus(x, b):
    return x if b is None else x + b


def _plain(s):
    op, dt = s["op"], DT[s["dt"]]
    if op == "norm":
        x = s["x"].float()
        mean = x.mean(1)
        c = x - mean[:, None]
        rstd = (c.square().mean(1) + EPS).rsqrt()
        return {"y": (c * rstd[:, None] * s["w"] + s["b"]).to(dt), "mean": mean, "rstd": rstd}
    if op == "norm_grad":
        xh = (s["x"].float() - s["mean"][:, None]) * s["rstd"][:, None]
        dy = s["dy"].float()
        a = dy * s["w"]
        dx = s["rstd"][:, None] * (a - a.mean(1, keepdim=True) - xh * (a * xh).mean(1, keepdim=True))
        if s["dres"] is not None:
            dx = dx + s["dres"].float()
        return {"dx": dx.to(dt), "dw": (dy * xh).sum(0), "db": dy.sum(0)}
    if op == "act_grad":
        g, dh = s["G"].float(), s["dH"].float()
        if s["gated"]:
            z = torch.cat((dh * s["U"].float() * _act_slope(g, s["act"]), dh * _act(g, s["act"])), 1)
        else:
            z = dh * _act_slope(g, s["act"])
        return {"dZ": z.to(dt), "db": z.sum(0) if s["bias"] else None}
    if op == "gated_experts":
        e, f, k = s["E"], s["F"], s["K"]
        sb = _unswizzle(s["scales"], s["scales"].numel(), k // 32)[s["at"]]
        rows = torch.zeros(e, s["most"], k, device="cuda")
        at = torch.arange(s["rows"], device="cuda") - s["offsets"][s["expert"]]
        rows[s["expert"], at] = _values(s["codes"], sb, MXFP4)
        pad = -(-f // 128) * 128

        def product(w, b):
            wsb = _unswizzle(w["scales"], e * pad, k // 32).reshape(e, pad, k // 32)[:, :f]
            y = torch.bmm(rows, _values(w["codes"], wsb, MXFP4).transpose(1, 2))
            return y if b is None else y + b[:, None]

        h = _act(product(s["wg"], s["bg"]), s["act"]) * product(s["wu"], s["bu"])
        return {"H": h[s["expert"], at].to(dt)}
    k = s["K"]
    if op == "out":
        a, w = _operand(s["a"], s["M"], k, s["fmt"]), _operand(s["w"], s["N"], k, s["fmt"])
        z = _plus((a @ w.t()) * (s["a"]["g"] * s["w"]["g"]), s["bias_v"])
        return {"D": (_act(z, s["act"]) + s["res"].float()).to(dt), "pre": z.to(dt) if s["save"] else None}
    if op == "gated_x":
        fmt, q = NVFP4, _quantized(s["x"].float(), NVFP4)
    else:
        fmt, q = s["fmt"], s["a"]
    a = _operand(q, s["M"], k, fmt)
    g = _plus((a @ _operand(s["wg"], s["F"], k, fmt).t()) * (q["g"] * s["wg"]["g"]), s.get("bg"))
    u = _plus((a @ _operand(s["wu"], s["F"], k, fmt).t()) * (q["g"] * s["wu"]["g"]), s.get("bu"))
    out = {"H": (_act(g, s["act"]) * u).to(dt)}
    if s.get("save"):
        out["G"], out["U"] = g.to(dt), u.to(dt)
    return out


# ---------------------------------------------------------------- the library's calls
_kept = {}


def _workspace(s, nbytes):
    """One zero-filled workspace for each problem, as a program keeps them."""
    if not nbytes:
        return None, 0
    import block_scaled_fp4_04_b200 as fp4
    key = tuple((k, v) for k, v in sorted(s.items()) if isinstance(v, (str, int, bool)))
    if key not in _kept:
        _kept[key] = fp4.Workspace().get(nbytes)
    return _kept[key], _kept[key].numel()


def _own(s):
    import block_scaled_fp4_04_b200 as fp4
    op = s["op"]
    oc = fp4.BF16 if s["dt"] == "bf16" else fp4.F32
    if op == "norm":
        fp4.fp4_layernorm(s["x"], s["M"], s["N"], oc, s["w"], s["b"], EPS, s["y"], oc, s["mean"], s["rstd"])
        return {"y": s["y"], "mean": s["mean"], "rstd": s["rstd"]}
    if op == "norm_grad":
        ws, n = _workspace(s, fp4.fp4_layernorm_backward_workspace_size(s["M"], s["N"]))
        fp4.fp4_layernorm_backward(s["dy"], s["x"], s["M"], s["N"], oc, s["w"], s["mean"], s["rstd"], s["dres"],
                                   s["dx"], oc, s["dw"], s["db"], ws, n)
        return {"dx": s["dx"], "dw": s["dw"], "db": s["db"]}
    act = ACTS[s["act"]]
    if op == "act_grad":
        ws, n = _workspace(s, fp4.fp4_act_backward_workspace_size(s["M"], s["F"], s["gated"])) if s["bias"] else (None, 0)
        fp4.fp4_act_backward(s["dH"], s["G"], s["U"], s["M"], s["F"], oc, act, s["dZ"], oc, s["db"], workspace=ws,
                             workspace_bytes=n)
        return {"dZ": s["dZ"], "db": s["db"]}
    if op == "gated_experts":
        wg, wu = s["wg"], s["wu"]
        fp4.fp4_gemm_gated_grouped(MXFP4, s["E"], s["offsets"], s["codes"], s["scales"], None, wg["codes"],
                                   wg["scales"], None, wu["codes"], wu["scales"], None, s["rows"], s["F"], s["K"],
                                   s["bg"], s["bu"], act, s["H"], oc)
        return {"H": s["H"]}
    if op == "out":
        a, w = s["a"], s["w"]
        ws, n = _workspace(s, fp4.fp4_gemm_epilogue_workspace_size(s["M"], s["N"], s["K"], s["fmt"], False))
        fp4.fp4_gemm_epilogue_ex(s["fmt"], a["codes"], a["scales"], a["g"], w["codes"], w["scales"], w["g"], s["M"],
                                 s["N"], s["K"], s["bias_v"], act, s["res"], oc, s["D"], oc, s["pre"], workspace=ws,
                                 workspace_bytes=n)
        return {"D": s["D"], "pre": s["pre"]}
    wg, wu = s["wg"], s["wu"]
    if op == "gated_x":
        ws, n = _workspace(s, fp4.fp4_gemm_gated_bf16a_workspace_size(s["M"], s["F"], s["K"]))
        fp4.fp4_gemm_gated_bf16a(s["x"], wg["codes"], wg["scales"], wg["g"], wu["codes"], wu["scales"], wu["g"],
                                 s["M"], s["F"], s["K"], None, None, act, s["H"], oc, None, None, s["xc"], s["xs"],
                                 s["xg"], ws, n, fp4.GEMM_WEIGHTS_READY)
        return {"H": s["H"]}
    a = s["a"]
    ws, n = _workspace(s, fp4.fp4_gemm_gated_workspace_size(s["M"], s["F"], s["K"], s["fmt"], False))
    fp4.fp4_gemm_gated(s["fmt"], a["codes"], a["scales"], a["g"], wg["codes"], wg["scales"], wg["g"], wu["codes"],
                       wu["scales"], wu["g"], s["M"], s["F"], s["K"], s["bg"], s["bu"], act, s["H"], oc, s["G"],
                       s["U"], workspace=ws, workspace_bytes=n)
    out = {"H": s["H"]}
    if s["save"]:
        out["G"], out["U"] = s["G"], s["U"]
    return out


def run(state):
    if own:
        return _own(state)
    return _plain(state)


# ---------------------------------------------------------------- the definition in 64 bits
def _exact_act(x, act):
    """(value, slope) in 64 bits."""
    if act == "none":
        return x, torch.ones_like(x)
    if act == "relu":
        return x.clamp(min=0), (x > 0).double()
    if act == "gelu":
        phi = torch.special.ndtr(x)
        return x * phi, phi + x * torch.exp(-x * x / 2) / math.sqrt(2 * math.pi)
    y, dy = x, torch.ones_like(x)
    if act == "gelu_tanh":
        t = torch.tanh(math.sqrt(2 / math.pi) * (x + 0.044715 * x ** 3))
        return (x / 2 * (1 + t),
                (1 + t) / 2 + x / 2 * (1 - t * t) * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * x * x))
    p = torch.sigmoid(y)
    return x * p, p + x * p * (1 - p) * dy


def _exact_operand(codes, scales, rows, cols, fmt):
    """64-bit values of an operand: every byte's address from the layout's formula."""
    dev = codes.device
    blk = 16 if fmt == NVFP4 else 32
    n = cols // blk
    r = torch.arange(rows, device=dev)[:, None]
    c = torch.arange(n, device=dev)[None]
    at = ((r // 128) * (-(-n // 4)) + c // 4) * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + c % 4
    sb = scales[at].long()
    if fmt == NVFP4:
        e, m = (sb >> 3) & 15, sb & 7
        sv = torch.where(e == 0, m.double() * 2.0 ** -9, (1 + m.double() / 8) * torch.exp2(e.double() - 7))
    else:
        sv = torch.exp2(sb.double() - 127)
    mag = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=dev)
    v = torch.empty(rows, cols, dtype=torch.float64, device=dev)
    for half in (0, 1):
        nib = (codes >> (4 * half)) & 15
        v[:, half::2] = mag[(nib & 7).int()] * (1 - 2 * (nib >> 3).double())
    v.view(rows, n, blk).mul_(sv[:, :, None])
    return v


def _exact_nvfp4(x):
    """The NVFP4 values of BF16 activations: each step a 64-bit operation rounded to 32 bits as defined."""
    rows, cols = x.shape
    x = x.double()
    am = x.abs().max()
    g = (am / 2688).float().double() if am > 0 else torch.ones((), dtype=torch.float64, device=x.device)
    b = x.view(rows, cols // 16, 16)
    t = ((b.abs().amax(2) / 6).float().double() / g).float().double()
    i = torch.arange(127, device=x.device)
    e4m3 = torch.where(i < 8, i.double() * 2.0 ** -9, (1 + (i % 8).double() / 8) * torch.exp2((i // 8).double() - 7))
    mid = (e4m3[1:] + e4m3[:-1]) / 2
    lo, hi = torch.searchsorted(mid, t.contiguous()), torch.searchsorted(mid, t.contiguous(), right=True)
    k = torch.where(lo % 2 == 0, lo, hi)  # a midpoint goes to the even code
    den = (e4m3[k] * g).float().double()
    mul = torch.where(den == 0, 0.0, 1 / den).float().double()
    a = (b * mul[:, :, None]).float().double()
    mag = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=x.device)
    mid = (mag[1:] + mag[:-1]) / 2
    lo = torch.searchsorted(mid, a.abs().contiguous())
    hi = torch.searchsorted(mid, a.abs().contiguous(), right=True)
    v = mag[torch.where(lo % 2 == 0, lo, hi)] * torch.where(a < 0, -1.0, 1.0)
    return (v * e4m3[k][:, :, None]).view(rows, cols) * g


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        x = s["x"].double()
        var, mean = torch.var_mean(x, 1, correction=0)
        rstd = 1 / torch.sqrt(var + EPS)
        return {"y": (x - mean[:, None]) * rstd[:, None] * s["w"].double() + s["b"].double(), "mean": mean,
                "rstd": rstd}
    if op == "norm_grad":
        n = case["N"]
        xh = (s["x"].double() - s["mean"].double()[:, None]) * s["rstd"].double()[:, None]
        dy = s["dy"].double()
        a = dy * s["w"].double()
        dx = (a - a.sum(1, keepdim=True) / n - xh * ((a * xh).sum(1, keepdim=True) / n)) * s["rstd"].double()[:, None]
        if case["res"]:
            dx += s["dres"].double()
        return {"dx": dx, "dw": (dy * xh).sum(0), "db": dy.sum(0)}
    if op == "act_grad":
        dh = s["dH"].double()
        v, slope = _exact_act(s["G"].double(), case["act"])
        z = torch.cat((dh * s["U"].double() * slope, dh * v), 1) if case["gated"] else dh * slope
        return {"dZ": z, "db": z.sum(0) if case["bias"] else None}
    k = case["K"]
    if op == "gated_experts":
        f, off = case["F"], s["offsets"].tolist()
        h = torch.empty(case["rows"], f, dtype=torch.float64, device="cuda")
        pad = -(-f // 128) * 128 * (-(-(k // 32) // 4) * 4)
        first = 0
        for e in range(case["E"]):
            lo, hi = off[e], off[e + 1]
            if lo == hi:
                continue
            a = _exact_operand(s["codes"][lo:hi], s["scales"][first:], hi - lo, k, MXFP4)
            first += -(-(hi - lo) // 128) * 512 * (-(-(k // 32) // 4))
            z = [a @ _exact_operand(s[w]["codes"][e], s[w]["scales"][e * pad:], f, k, MXFP4).t() for w in ("wg", "wu")]
            if case["bias"]:
                z = [z[0] + s["bg"][e].double(), z[1] + s["bu"][e].double()]
            h[lo:hi] = _exact_act(z[0], case["act"])[0] * z[1]
        return {"H": h}
    fmt = case.get("fmt", NVFP4)

    def whole(q, rows):
        return _exact_operand(q["codes"], q["scales"], rows, k, fmt) * q["g"].double()

    a = _exact_nvfp4(s["x"]) if op == "gated_x" else whole(s["a"], case["M"])
    if op == "out":
        z = a @ whole(s["w"], case["N"]).t()
        if case["bias"]:
            z += s["bias_v"].double()
        return {"D": _exact_act(z, case["act"])[0] + s["res"].double(), "pre": z if case["save"] else None}
    g, u = a @ whole(s["wg"], case["F"]).t(), a @ whole(s["wu"], case["F"]).t()
    if case.get("bias"):
        g, u = g + s["bg"].double(), u + s["bu"].double()
    out = {"H": _exact_act(g, case["act"])[0] * u}
    if case.get("save"):
        out["G"], out["U"] = g, u
    return out


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    op = case["op"]
    e = 2 if case["dt"] == "bf16" else 4
    if op == "norm":
        m, n = case["M"], case["N"]
        return {"bytes": 2 * e * m * n + 8 * n + 8 * m, "flops": 8 * m * n}
    if op == "norm_grad":
        m, n = case["M"], case["N"]
        return {"bytes": (4 if case["res"] else 3) * e * m * n + 12 * n + 8 * m, "flops": 16 * m * n}
    if op == "act_grad":
        m, f = case["M"], case["F"]
        w = 2 if case["gated"] else 1
        return {"bytes": (2 * w + 1 if case["gated"] else 3) * e * m * f + (4 * w * f if case["bias"] else 0),
                "flops": 12 * m * f}
    k = case["K"]
    per = 0.5 + 1 / (16 if case.get("fmt", NVFP4) == NVFP4 else 32)  # bytes an FP4 element takes with its scale
    if op == "gated_experts":
        rows, f, n = case["rows"], case["F"], min(case["E"], case["rows"])
        per = 0.5 + 1 / 32
        return {"bytes": rows * k * per + n * 2 * f * k * per + rows * f * e + (8 * n * f if case["bias"] else 0),
                "flops": 4 * rows * f * k}
    m = case["M"]
    if op == "out":
        n = case["N"]
        return {"bytes": (m + n) * k * per + (3 if case["save"] else 2) * m * n * e + (4 * n if case["bias"] else 0),
                "flops": 2 * m * n * k}
    f = case["F"]
    x = m * k * (2 if op == "gated_x" else per)
    return {"bytes": x + 2 * f * k * per + (3 if case.get("save") else 1) * m * f * e
            + (8 * f if case.get("bias") else 0), "flops": 4 * m * f * k}
