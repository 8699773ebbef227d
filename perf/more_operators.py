"""Tokens sorted by expert and back, with weights applied, their gradients, and the product in
8-bit integers with a scale for each token and channel (dense, by experts), as cases to measure.

Where ``own`` is false, ``run`` computes them from elementary torch operations; where it is true,
it calls the library."""
import math

import torch

own = False

ACTS = {"none": 0, "relu": 1, "silu": 2, "gelu": 3}
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
TINY = 2.0 ** -126  # the smallest scale of an 8-bit row


# ---------------------------------------------------------------- cases
def listed():
    return [
        # one decode step of 16 sequences, 4 of 32 experts each: sorted, and written as the 8-bit
        # operand of the experts' products (latency)
        dict(name="dispatch step", op="dispatch", T=16, k=4, E=32, H=2880, dt="bf16", to="i8", drop=0.0),
        # a prompt of 4096 tokens, sorted and copied to the experts' order
        dict(name="dispatch prompt", op="dispatch", T=4096, k=4, E=32, H=2880, dt="bf16", to="rows", drop=0.0),
        # a long batch over many experts as 8-bit rows, a tenth of the slots without an expert
        # here (padding, or experts that live elsewhere)
        dict(name="dispatch long", op="dispatch", T=16384, k=8, E=128, H=4096, dt="bf16", to="i8", drop=0.1),
        # gradient of the dispatch in FP32 training: ragged batch, odd width
        dict(name="dispatch grad", op="dispatch_grad", T=4095, k=2, E=8, H=8191, dt="f32", drop=0.0),
        # the decode step's way back, added to the residual stream
        dict(name="combine step", op="combine", T=16, k=4, E=32, H=2880, dt="bf16", res=True, drop=0.0),
        # the prompt's way back
        dict(name="combine prompt", op="combine", T=4096, k=4, E=32, H=2880, dt="bf16", res=False, drop=0.0),
        # BF16 training: gradients of the experts' rows and of the weights
        dict(name="combine grad bf16", op="combine_grad", T=8192, k=4, E=32, H=2880, dt="bf16", drop=0.0),
        # FP32 training, ragged batch with slots that have no expert
        dict(name="combine grad fp32", op="combine_grad", T=1999, k=3, E=5, H=5760, dt="f32", drop=0.2),
        # one decode step through a wide projection: BF16 activations quantized, weights streamed
        dict(name="i8 step", op="i8", M=16, N=28672, K=8192, dt="bf16", x=True, act="none", bias=False),
        # a prompt through a projection, from operands already in 8 bits
        dict(name="i8 prompt", op="i8", M=8192, N=8192, K=8192, dt="bf16", x=False, act="gelu", bias=True),
        # a decode step's sorted rows: few per expert, some experts without any
        dict(name="i8 experts step", op="i8_experts", E=32, rows=64, N=5760, K=2880, dt="bf16", act="none", bias=True),
        # a prompt's sorted rows
        dict(name="i8 experts prompt", op="i8_experts", E=32, rows=16384, N=5760, K=2880, dt="bf16", act="silu",
             bias=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["dispatch", "dispatch", "dispatch_grad", "combine", "combine_grad", "i8", "i8", "i8_experts"])
    dt = rng.choice(["bf16", "bf16", "f32"])
    if op in ("i8", "i8_experts"):
        act, bias = rng.choice(["none", "relu", "silu", "gelu"]), rng.random() < 0.5
        k = 16 * _log(rng, 2, 512)
        if op == "i8":
            n = _log(rng, 16, 28672)
            m = min(_log(rng, 1, 8192), max(1, (1 << 37) // (n * k)))
            return dict(op=op, M=m, N=n, K=k, dt=dt, x=rng.random() < 0.5, act=act, bias=bias)
        e = rng.choice([1, 2, 5, 8, 32])
        n = _log(rng, 16, 5760)
        return dict(op=op, E=e, rows=min(_log(rng, 1, 8192), max(1, (1 << 35) // (n * k))), N=n, K=min(k, 2880), dt=dt,
                    act=act, bias=bias)
    e = _log(rng, 1, 256)
    k = rng.randint(1, min(8, e))
    drop = rng.choice([0.0, 0.0, 0.1, 0.5])
    h = _log(rng, 16, 8192)
    to = rng.choice(["rows", "i8"])
    if op == "dispatch" and to == "i8":
        h = -(-h // 16) * 16
    t = min(_log(rng, 1, 16384), max(1, (1 << 27) // (h * k)))
    c = dict(op=op, T=t, k=k, E=e, H=h, dt=dt, drop=drop)
    if op == "dispatch":
        c["to"] = to
    if op == "combine":
        c["res"] = rng.random() < 0.5
    return c


# ---------------------------------------------------------------- inputs
def _normal(gen, shape, std=1.0, dtype=torch.float32):
    return (torch.randn(*shape, generator=gen, device="cuda") * std).to(dtype)


def _activations(gen, shape, dtype):
    """N(0, 1) with a few outlier channels, as hidden states have them."""
    x = torch.randn(*shape, generator=gen, device="cuda")
    hot = torch.randint(0, shape[-1], (max(1, shape[-1] // 1000),), generator=gen, device="cuda")
    x[..., hot] *= 20.0
    return x.to(dtype)


def _ids(gen, case):
    """The experts that a router picks: the k largest of uneven random gates; dropped slots are -1."""
    t, k, e = case["T"], case["k"], case["E"]
    gates = torch.rand(t, e, generator=gen, device="cuda") + 0.3 * torch.rand(e, generator=gen, device="cuda")
    ids = torch.topk(gates, k, dim=1).indices
    if case["drop"]:
        ids = torch.where(torch.rand(t, k, generator=gen, device="cuda") < case["drop"], -1, ids)
    return ids


def _int8_rows(gen, shape, std):
    x = torch.randn(*shape, generator=gen, device="cuda") * std
    s = x.abs().amax(-1) / 127.0
    return torch.round(x / s[..., None]).clamp_(-127, 127).to(torch.int8), s


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case)
    op, dt = case["op"], DT[case["dt"]]

    def zeros(*shape, dtype=dt):
        return torch.zeros(*shape, dtype=dtype, device="cuda")

    if op in ("i8", "i8_experts"):
        n, k = case["N"], case["K"]
        if op == "i8":
            m = case["M"]
            s["w"], s["sw"] = _int8_rows(gen, (n, k), 0.02)
            s["b"] = _normal(gen, (n,), 0.5) if case["bias"] else None
            if case["x"]:
                s["xs"] = _activations(gen, (m, k), torch.bfloat16)
                s["a"], s["sa"] = zeros(m, k, dtype=torch.int8), zeros(m, dtype=torch.float32)
            else:
                s["a"], s["sa"] = _int8_rows(gen, (m, k), 1.0)
            s["D"] = zeros(m, n)
            return s
        e, rows = case["E"], case["rows"]
        # rows routed to experts at random, sorted by expert
        cnt = torch.bincount(torch.randint(0, e, (rows,), generator=gen, device="cuda"), minlength=e)
        off = zeros(e + 1, dtype=torch.int32)
        off[1:] = cnt.cumsum(0)
        s["offsets"], s["most"] = off, int(cnt.max())
        s["expert"] = torch.repeat_interleave(torch.arange(e, device="cuda"), cnt)
        s["a"], s["sa"] = _int8_rows(gen, (rows, k), 1.0)
        w = [_int8_rows(gen, (n, k), 0.02) for _ in range(e)]
        s["w"], s["sw"] = torch.stack([x[0] for x in w]), torch.stack([x[1] for x in w])
        s["b"] = _normal(gen, (e, n), 0.5) if case["bias"] else None
        s["D"] = zeros(rows, n)
        return s
    t, k, h = case["T"], case["k"], case["H"]
    ids = _ids(gen, case)
    rows = t * k
    if op == "dispatch":
        s["ids"], s["x"] = ids, _activations(gen, (t, h), dt)
        s["offsets"], s["row_of"] = zeros(case["E"] + 1, dtype=torch.int32), zeros(t, k, dtype=torch.int32)
        if case["to"] == "i8":
            s["y"], s["sy"] = zeros(rows, h, dtype=torch.int8), zeros(rows, dtype=torch.float32)
        else:
            s["y"] = zeros(rows, h)
        return s
    # the later operators start from rows that were sorted before
    flat = torch.where(ids < 0, case["E"], ids).reshape(-1)
    order = torch.sort(flat, stable=True).indices
    row_of = torch.empty(rows, dtype=torch.int32, device="cuda")
    row_of[order] = torch.arange(rows, dtype=torch.int32, device="cuda")
    s["row_of"] = torch.where(ids.reshape(-1) < 0, -1, row_of).view(t, k)
    s["wt"] = torch.softmax(_normal(gen, (t, k)), 1)
    if op == "dispatch_grad":
        s["y"] = _normal(gen, (rows, h), 1.0, dt)
        s["out"] = zeros(t, h)
        return s
    s["y"] = _activations(gen, (rows, h), dt)
    if op == "combine":
        s["res"] = _normal(gen, (t, h), 1.0, dt) if case["res"] else None
        s["out"] = zeros(t, h)
        return s
    s["dout"] = _normal(gen, (t, h), 1.0, dt)
    s["dy"], s["dw"] = zeros(rows, h), zeros(t, k, dtype=torch.float32)
    return s


# ---------------------------------------------------------------- the plain forms
def _act(x, act):
    if act == "relu":
        return torch.where(x > 0, x, torch.zeros_like(x))
    if act == "silu":
        return x / (1.0 + torch.exp(-x))
    if act == "gelu":
        return 0.5 * x * (1.0 + torch.erf(x * math.sqrt(0.5)))
    return x


def _quantized_rows(x):
    """8-bit values of FP32 rows and their scales (a tensor as the divisor: torch divides by it)."""
    am = x.abs().amax(1)
    sc = torch.where(am > 0, (am / torch.full_like(am, 127.0)).clamp(min=TINY), torch.ones_like(am))
    return torch.round(x * (torch.ones_like(sc) / sc)[:, None]).to(torch.int8), sc


def _scaled(acc, sa, sw, b, act, dt):
    """The sums of integer products are whole numbers, exact in 64 bits; from there in 32."""
    z = acc.float() * sa * sw
    return _act(z if b is None else z + b, act).to(dt)


def _plain(s):
    op, dt = s["op"], DT[s["dt"]]
    if op == "i8":
        a, sa = _quantized_rows(s["xs"].float()) if s["x"] else (s["a"], s["sa"])
        acc = a.double() @ s["w"].double().t()
        return {"D": _scaled(acc, sa[:, None], s["sw"][None], s["b"], s["act"], dt)}
    if op == "i8_experts":
        e, k = s["E"], s["K"]
        at = torch.arange(s["rows"], device="cuda") - s["offsets"][s["expert"]]
        rows = torch.zeros(e, s["most"], k, dtype=torch.float64, device="cuda")
        rows[s["expert"], at] = s["a"].double()
        acc = torch.bmm(rows, s["w"].double().transpose(1, 2))[s["expert"], at]
        b = None if s["b"] is None else s["b"][s["expert"]]
        return {"D": _scaled(acc, s["sa"][:, None], s["sw"][s["expert"]], b, s["act"], dt)}
    t, k, h = s["T"], s["k"], s["H"]
    rows = t * k
    if op == "dispatch":
        e, flat = s["E"], s["ids"].reshape(-1)
        none = (flat < 0) | (flat >= e)
        key, order = torch.sort(torch.where(none, e, flat), stable=True)
        offsets = torch.searchsorted(key, torch.arange(e + 1, device="cuda")).int()
        row_of = torch.empty(rows, dtype=torch.int32, device="cuda")
        row_of[order] = torch.arange(rows, dtype=torch.int32, device="cuda")
        row_of = torch.where(none, -1, row_of).view(t, k)
        here = torch.arange(rows, device="cuda") < offsets[e]
        out = {"offsets": offsets, "row_of": row_of}
        if s["to"] == "i8":
            q, sc = _quantized_rows(s["x"].float())
            out["y"] = torch.where(here[:, None], q[order // k], 0)
            out["sy"] = torch.where(here, sc[order // k], 0.0)
        else:
            out["y"] = torch.where(here[:, None], s["x"][order // k], 0.0)
        return out
    here = s["row_of"] >= 0
    at = torch.where(here, s["row_of"], 0).long()
    if op == "dispatch_grad":
        return {"dx": torch.where(here[..., None], s["y"][at].float(), 0.0).sum(1).to(dt)}
    if op == "combine":
        y = torch.where(here[..., None], s["y"][at].float() * s["wt"][..., None], 0.0).sum(1)
        return {"out": (y if s["res"] is None else y + s["res"].float()).to(dt)}
    dout = s["dout"].float()[:, None]
    dw = torch.where(here, (dout * s["y"][at].float()).sum(2), 0.0)
    dy = torch.zeros(rows + 1, h, dtype=dt, device="cuda")  # slots without an expert go to the last row
    dy[torch.where(here, s["row_of"], rows).long()] = (dout * s["wt"][..., None]).to(dt)
    return {"dy": dy[:rows], "dw": dw}


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
    if op == "i8":
        m, n, k = s["M"], s["N"], s["K"]
        if s["x"]:
            fp4.fp4_quantize_i8(s["xs"], m, k, fp4.BF16, s["a"], s["sa"])
        ws, size = _workspace(s, fp4.fp4_gemm_i8_workspace_size(m, n, k))
        fp4.fp4_gemm_i8(s["a"], s["sa"], s["w"], s["sw"], m, n, k, s["b"], ACTS[s["act"]], s["D"], oc, ws, size,
                        fp4.GEMM_WEIGHTS_READY if s["x"] else 0)
        return {"D": s["D"]}
    if op == "i8_experts":
        ws, size = _workspace(s, fp4.fp4_gemm_i8_grouped_workspace_size(s["E"], s["rows"], s["N"], s["K"]))
        fp4.fp4_gemm_i8_grouped(s["E"], s["offsets"], s["a"], s["sa"], s["w"], s["sw"], s["rows"], s["N"], s["K"],
                                s["b"], ACTS[s["act"]], s["D"], oc, ws, size)
        return {"D": s["D"]}
    t, k, h = s["T"], s["k"], s["H"]
    if op == "dispatch":
        ws, size = _workspace(s, fp4.fp4_moe_sort_workspace_size(t, k, s["E"]))
        fp4.fp4_moe_sort(s["ids"], 8, t, k, s["E"], s["offsets"], s["row_of"], None, ws, size)
        out = {"offsets": s["offsets"], "row_of": s["row_of"], "y": s["y"]}
        if s["to"] == "i8":
            fp4.fp4_moe_dispatch_i8(s["x"], t, h, oc, k, s["row_of"], s["y"], s["sy"])
            out["sy"] = s["sy"]
        else:
            fp4.fp4_moe_dispatch(s["x"], t, h, oc, k, s["row_of"], s["y"], oc)
        return out
    if op == "dispatch_grad":
        fp4.fp4_moe_combine(s["y"], oc, s["row_of"], None, t, k, h, None, oc, s["out"], oc)
        return {"dx": s["out"]}
    if op == "combine":
        fp4.fp4_moe_combine(s["y"], oc, s["row_of"], s["wt"], t, k, h, s["res"], oc, s["out"], oc)
        return {"out": s["out"]}
    fp4.fp4_moe_combine_backward(s["dout"], s["y"], oc, s["row_of"], s["wt"], t, k, h, s["dy"], oc, s["dw"])
    return {"dy": s["dy"], "dw": s["dw"]}


def run(state):
    if own:
        return _own(state)
    return _plain(state)


# ---------------------------------------------------------------- the definition in 64 bits
def _exact_act(x, act):
    if act == "relu":
        return x.clamp(min=0)
    if act == "silu":
        return x * torch.sigmoid(x)
    if act == "gelu":
        return x * torch.special.ndtr(x)
    return x


def _exact_i8(x):
    """The 8-bit values: each step a 64-bit operation rounded to 32 bits as defined."""
    x = x.double()
    top = x.abs().max(1).values
    sc = (top / 127).float().double()
    sc = torch.where(sc < TINY, torch.full_like(sc, TINY), sc)
    sc[top == 0] = 1.0
    return (x * (1 / sc).float().double()[:, None]).float().round(), sc.float()


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "i8":
        a, sa = _exact_i8(s["xs"]) if case["x"] else (s["a"], s["sa"])
        d = torch.empty(case["M"], case["N"], dtype=torch.float64, device="cuda")
        w = s["w"].double().t().contiguous()
        for lo in range(0, case["M"], 1024):
            z = (a[lo:lo + 1024].double() @ w) * sa[lo:lo + 1024, None].double() * s["sw"].double()
            d[lo:lo + 1024] = _exact_act(z if s["b"] is None else z + s["b"].double(), case["act"])
        return {"D": d}
    if op == "i8_experts":
        d, off = torch.empty(case["rows"], case["N"], dtype=torch.float64, device="cuda"), s["offsets"].tolist()
        for e in range(case["E"]):
            lo, hi = off[e], off[e + 1]
            z = (s["a"][lo:hi].double() @ s["w"][e].double().t()) * s["sa"][lo:hi, None].double() * s["sw"][e].double()
            d[lo:hi] = _exact_act(z if s["b"] is None else z + s["b"][e].double(), case["act"])
        return {"D": d}
    t, k, h = case["T"], case["k"], case["H"]
    if op == "dispatch":
        # counted expert by expert: a slot's row is its expert's start plus the slots before it
        flat = s["ids"].reshape(-1)
        row_of, start = torch.full_like(flat, -1), 0
        offsets = [0]
        for e in range(case["E"]):
            mine = torch.nonzero(flat == e).view(-1)
            row_of[mine] = start + torch.arange(mine.numel(), device="cuda")
            start += mine.numel()
            offsets.append(start)
        out = {"offsets": torch.tensor(offsets, dtype=torch.int32), "row_of": row_of.int().view(t, k)}
        slots = torch.nonzero(row_of >= 0).view(-1)
        if case["to"] == "i8":
            q, sc = _exact_i8(s["x"])
            y, sy = s["y"], torch.zeros(t * k, dtype=torch.float64, device="cuda")
            y[row_of[slots]] = q[slots // k].to(torch.int8)
            sy[row_of[slots]] = sc[slots // k].double()
            out["y"], out["sy"] = y, sy
        else:
            y = torch.zeros(t * k, h, dtype=torch.float64, device="cuda")
            y[row_of[slots]] = s["x"][slots // k].double()
            out["y"] = y
        return out
    row = s["row_of"].long()
    if op in ("dispatch_grad", "combine"):
        y = torch.zeros(t, h, dtype=torch.float64, device="cuda")
        for j in range(k):
            on = torch.nonzero(row[:, j] >= 0).view(-1)
            part = s["y"][row[on, j]].double()
            y[on] += part * s["wt"][on, j, None].double() if op == "combine" else part
        if op == "dispatch_grad":
            return {"dx": y}
        return {"out": y if s["res"] is None else y + s["res"].double()}
    dy = torch.zeros(t * k, h, dtype=torch.float64, device="cuda")
    dw = torch.zeros(t, k, dtype=torch.float64, device="cuda")
    for j in range(k):
        on = torch.nonzero(row[:, j] >= 0).view(-1)
        g = s["dout"][on].double()
        dy[row[on, j]] = g * s["wt"][on, j, None].double()
        dw[on, j] = (g * s["y"][row[on, j]].double()).sum(1)
    return {"dy": dy, "dw": dw}


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    op = case["op"]
    e = 2 if case["dt"] == "bf16" else 4
    if op == "i8":
        m, n, k = case["M"], case["N"], case["K"]
        return {"bytes": m * k * (2 if case["x"] else 1) + n * k + 4 * (m + n) + e * m * n + (4 * n if case["bias"] else 0),
                "flops": 2 * m * n * k}
    if op == "i8_experts":
        rows, n, k, used = case["rows"], case["N"], case["K"], min(case["E"], case["rows"])
        return {"bytes": rows * k + used * n * k + 4 * (rows + used * n) + e * rows * n
                + (4 * used * n if case["bias"] else 0), "flops": 2 * rows * n * k}
    t, k, h = case["T"], case["k"], case["H"]
    rows = round(t * k * (1 - case["drop"]))  # that have an expert
    if op == "dispatch":
        out = rows * (h + 4) if case["to"] == "i8" else rows * h * e
        return {"bytes": t * h * e + out + 12 * t * k + 4 * case["E"], "flops": 3 * t * h if case["to"] == "i8" else 0}
    if op == "dispatch_grad":
        return {"bytes": (rows + t) * h * e + 4 * t * k, "flops": rows * h}
    if op == "combine":
        return {"bytes": (rows + t * (2 if case["res"] else 1)) * h * e + 8 * t * k, "flops": 2 * rows * h}
    return {"bytes": (2 * rows + t) * h * e + 12 * t * k, "flops": 3 * rows * h}
