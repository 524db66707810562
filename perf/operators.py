"""The operators of the wide appearance network and its training step, as measured cases.

Six kinds of case: the root-mean-square norm with the residual's addition and an 8-bit output (`norm`) and its
backward (`norm_bwd`), the 8-bit matrix product with a scale for each block of 128 (`matmul`) and a linear layer's
backward made of it (`matmul_bwd`), the global gradient norm with clipping (`clip`) and the Adam step that clips by
it (`adam`).  8-bit values are e4m3; a block's scale is its largest magnitude / 448, scales are laid out one row per
block of 128 along the contracted axis.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "f16": 2, "bf16": 2}
FP8 = torch.float8_e4m3fn
BLOCK = 128
EPS = 1e-6
WORKSPACE = 96 << 20   # bytes of scratch that a training loop keeps for all of its calls
ADAM = dict(beta1=0.9, beta2=0.999, eps=1e-15)
# the scene's parameter groups: rows per Gaussian, learning rate, activation (0 none, 1 exp, 2 sigmoid)
SCENE = (("means", 3, 1.6e-4, 0), ("scales", 3, 1e-3, 1), ("quats", 4, 1e-3, 0), ("opacity", 1, 1e-2, 2),
         ("sh_dc", 3, 2.5e-3, 0), ("sh_rest", 45, 1.25e-4, 0))


def listed():
    return [
        # one Gaussian's (or one pixel's) features through a wide layer's norm: latency alone
        {"name": "norm, 1 row", "op": "norm", "rows": 1, "cols": 4096, "dtype": "bf16", "residual": True},
        # a feature width that is no multiple of a block, first layer (nothing to add yet)
        {"name": "norm, odd width, no residual", "op": "norm", "rows": 4099, "cols": 777, "dtype": "f16",
         "residual": False},
        # every Gaussian of the 250k training scene at width 512, as a training step keeps it (y and rstd too)
        {"name": "norm, 250k rows", "op": "norm", "rows": 250000, "cols": 512, "dtype": "bf16", "residual": True},
        # the backward on the 160k scene in float32, and an odd wide one in 16 bits
        {"name": "norm backward, 160k rows", "op": "norm_bwd", "rows": 160000, "cols": 256, "dtype": "f32"},
        {"name": "norm backward, odd", "op": "norm_bwd", "rows": 10007, "cols": 1000, "dtype": "bf16"},
        # serving: one row against a wide layer's weights
        {"name": "matmul, 1 row", "op": "matmul", "rows": 1, "n": 4096, "k": 4096, "out": "bf16"},
        # a few rows, nothing a multiple of anything, float32 out
        {"name": "matmul, odd", "op": "matmul", "rows": 37, "n": 1001, "k": 777, "out": "f32"},
        # a hidden layer over the 160k scene
        {"name": "matmul, 160k rows", "op": "matmul", "rows": 160000, "n": 512, "k": 512, "out": "bf16"},
        # the largest: a wide layer over many rows, bound by the products
        {"name": "matmul, wide", "op": "matmul", "rows": 65536, "n": 2048, "k": 2048, "out": "f16"},
        # backward of a hidden layer over the 160k scene: both quantisations, dX and dW, through the relu
        {"name": "matmul backward, 160k rows", "op": "matmul_bwd", "rows": 160000, "n": 512, "k": 256,
         "dtype": "bf16"},
        # many odd tensors of mixed types (a network's layers), the norm above the limit
        {"name": "clip, 40 tensors", "op": "clip", "tensors": 40, "mean": 30000, "dtype": "mixed"},
        # the clipped step over all parameters of a 1M-Gaussian scene with degree-3 SH
        {"name": "clipped Adam, 1M Gaussians", "op": "adam", "gaussians": 1000000},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, hi):
    """A width as networks have it (a multiple of 64) or an odd one."""
    w = _log(rng, 64, hi)
    return max(64, w // 64 * 64) if rng.random() < 0.6 else w | 1


def draw(rng):
    op = rng.choice(["norm", "norm_bwd", "matmul", "matmul", "matmul_bwd", "clip", "adam"])
    if op in ("norm", "norm_bwd"):
        cols = _width(rng, 2500)
        rows = _log(rng, 1, min(250000, 120_000_000 // cols))
        c = {"op": op, "rows": rows, "cols": cols, "dtype": rng.choice(["f32", "f16", "bf16"])}
        return c | {"residual": rng.random() < 0.7} if op == "norm" else c
    if op == "matmul":
        n, k = _width(rng, 2500), _width(rng, 2500)
        rows = _log(rng, 1, min(160000, 100_000_000 // max(n, k)))
        return {"op": op, "rows": rows, "n": n, "k": k, "out": rng.choice(["f32", "f16", "bf16"])}
    if op == "matmul_bwd":
        n, k = _width(rng, 1500), _width(rng, 1500)
        rows = _log(rng, 100, min(160000, 50_000_000 // max(n, k)))
        return {"op": op, "rows": rows, "n": n, "k": k, "dtype": rng.choice(["f16", "bf16"])}
    if op == "clip":
        return {"op": op, "tensors": rng.randint(1, 60), "mean": _log(rng, 50, 300000),
                "dtype": rng.choice(["f32", "bf16", "f16", "mixed"])}
    return {"op": op, "gaussians": _log(rng, 1000, 1000000)}


# ------------------------------------------------------------------ inputs

def _quantised(x, axis_rows=False, blocks=False):
    """(q, scales) of x [r][c] in 32 bits: a scale for each row and 128 columns ([c/128][r]); with `blocks` for each
    128 x 128 ([c/128][r/128])."""
    r, c = x.shape
    kb = -(-c // BLOCK)
    xp = torch.nn.functional.pad(x.float(), (0, kb * BLOCK - c))
    a = xp.view(r, kb, BLOCK).abs().amax(2).t().contiguous()                     # [kb][r]
    if blocks:
        rb = -(-r // BLOCK)
        a = torch.nn.functional.pad(a, (0, rb * BLOCK - r)).view(kb, rb, BLOCK).amax(2)
    a = a.clamp_min(2.0 ** -100)
    top = torch.full_like(a, 448.0)   # a tensor: a division by or of a plain number becomes a reciprocal, rounded twice
    inv = top / a
    full = inv.repeat_interleave(BLOCK, 1)[:, :r] if blocks else inv
    q = (xp.view(r, kb, BLOCK) * full.t().unsqueeze(2)).to(FP8).view(r, kb * BLOCK)[:, :c]
    return q, a / top


def _rows16(q):
    """q with rows padded to a multiple of 16 bytes, as the products read them."""
    r, c = q.shape
    out = torch.zeros(r, -(-c // 16) * 16, dtype=torch.uint8, device=q.device)
    out[:, :c] = q.view(torch.uint8)
    return out.view(FP8)[:, :c]


def prepare(case, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    rand = lambda *s: torch.randn(*s, device="cuda", generator=g)
    op = case["op"]
    s = {"case": dict(case), "workspace": torch.empty(WORKSPACE, dtype=torch.uint8, device="cuda")}
    if op in ("norm", "norm_bwd"):
        r, c, dt = case["rows"], case["cols"], DTYPES[case["dtype"]]
        outlier = 1 + 8 * (torch.rand(c, device="cuda", generator=g) < 0.01)      # some features run larger
        s["x"] = (rand(r, c) * outlier).to(dt)
        s["weight"] = 1 + 0.2 * rand(c)
        if op == "norm":
            s["residual"] = (0.5 * rand(r, c)).to(dt) if case["residual"] else None
            s["q"] = torch.empty(r, -(-c // 16) * 16, dtype=torch.uint8, device="cuda").view(FP8)[:, :c]
            s["scales"] = torch.empty(-(-c // BLOCK), r, device="cuda")
            s["sum"] = torch.empty_like(s["x"]) if case["residual"] else None
            s["rstd"] = torch.empty(r, device="cuda")
        else:
            s["rstd"] = (s["x"].float().square().mean(1) + EPS).rsqrt()
            s["dy"] = rand(r, c).to(dt)
            s["dsum"] = rand(r, c).to(dt)
            s["dx"] = torch.empty_like(s["x"])
            s["dweight"] = torch.empty(c, device="cuda")
    elif op in ("matmul", "matmul_bwd"):
        m, n, k = case["rows"], case["n"], case["k"]
        w = rand(n, k) / math.sqrt(k)
        if op == "matmul":
            q, s["a_scales"] = _quantised(rand(m, k) * (1 + torch.rand(m, 1, device="cuda", generator=g)))
            s["a"] = _rows16(q)
            q, s["b_scales"] = _quantised(w, blocks=True)
            s["b"] = _rows16(q)
            s["out"] = torch.empty(m, n, dtype=DTYPES[case["out"]], device="cuda")
        else:
            dt = DTYPES[case["dtype"]]
            s["x"] = rand(m, k).to(dt)
            s["u"] = rand(m, n).relu().to(dt)                                      # the relu's output
            s["du"] = (rand(m, n) * 1e-3).to(dt)
            q, ws = _quantised(w, blocks=True)                                     # kept with the weights
            s["wt"], s["wt_scales"] = _rows16(q.view(torch.uint8).t().contiguous().view(FP8)), ws.t().contiguous()
            s["dx"] = torch.empty(m, k, dtype=dt, device="cuda")
            s["dw"] = torch.empty(n, k, device="cuda")
            b = lambda r, c: torch.empty(r, -(-c // 16) * 16, dtype=torch.uint8, device="cuda").view(FP8)[:, :c]
            sc = lambda r, c: torch.empty(-(-c // BLOCK), r, device="cuda")
            s["dq"], s["dq_scales"], s["dqt"], s["dqt_scales"] = b(m, n), sc(m, n), b(n, m), sc(n, m)
            s["xqt"], s["xqt_scales"] = b(k, m), sc(k, m)
    elif op == "clip":
        sizes = np.random.RandomState(case["tensors"]).uniform(0.05, 2.0, case["tensors"])
        kinds = ["f32", "bf16", "f16"] if case["dtype"] == "mixed" else [case["dtype"]]
        s["grads"] = [(0.01 * rand(max(1, int(case["mean"] * u)))).to(DTYPES[kinds[i % len(kinds)]])
                      for i, u in enumerate(sizes)]
        s["outs"] = [torch.empty_like(x) for x in s["grads"]]
        s["max_norm"] = 0.5 * 0.01 * math.sqrt(sum(x.numel() for x in s["grads"]))
        s["norm"] = torch.empty(1, device="cuda")
        if own:  # the table of tensors that a training loop builds once
            from gaussian_splatting_tile_gb300 import rs
            s["table"] = rs.GradTable([rs.GradTensor(x, out=o) for x, o in zip(s["grads"], s["outs"])])
    else:
        n = case["gaussians"]
        s["groups"] = []
        for name, rows, lr, act in SCENE:
            p = rand(rows, n) * 0.5 - (4.0 if act == 1 else 0.0)
            grad = rand(rows, n) * 1e-3
            s["groups"].append({"p": p, "g": grad, "m": 1e-4 * rand(rows, n), "v": 1e-7 * rand(rows, n).square() + 1e-9,
                                "lr": lr, "act": act,
                                "a": torch.empty_like(p) if act else None})
        s["max_norm"], s["step"] = 0.3 * 1e-3 * math.sqrt(59 * n), 100
        s["norm"] = torch.empty(1, device="cuda")
    return s


# ------------------------------------------------------------------ the framework's operators

def _run_own(s):
    from gaussian_splatting_tile_gb300 import rs
    op = s["case"]["op"]
    if op == "norm":
        rs.rs_rms_norm_fwd(s["x"], s["weight"], s["q"], s["scales"], residual=s["residual"], sum=s["sum"],
                           rstd=s["rstd"], eps=EPS)
        out = {"q": s["q"], "scales": s["scales"], "rstd": s["rstd"]}
        return out | {"sum": s["sum"]} if s["sum"] is not None else out
    if op == "norm_bwd":
        rs.rs_rms_norm_bwd(s["x"], s["weight"], s["rstd"], s["dy"], s["dx"], s["dweight"], s["workspace"],
                           dL_dsum=s["dsum"])
        return {"dx": s["dx"], "dweight": s["dweight"]}
    if op == "matmul":
        rs.rs_matmul_fp8(s["a"], s["a_scales"], s["b"], s["b_scales"], s["out"], s["workspace"])
        return {"out": s["out"]}
    if op == "matmul_bwd":
        rs.rs_quantize_fp8(s["du"], s["dq"], s["dq_scales"], s["dqt"], s["dqt_scales"], relu=s["u"])
        rs.rs_quantize_fp8(s["x"], None, None, s["xqt"], s["xqt_scales"])
        rs.rs_matmul_fp8(s["dq"], s["dq_scales"], s["wt"], s["wt_scales"], s["dx"], s["workspace"])
        rs.rs_matmul_fp8(s["dqt"], s["dqt_scales"], s["xqt"], s["xqt_scales"], s["dw"], s["workspace"])
        return {"dx": s["dx"], "dw": s["dw"]}
    if op == "clip":
        rs.rs_grad_clip(s["table"], s["max_norm"], s["norm"], s["workspace"])
        return {"norm": s["norm"], "outs": s["outs"]}
    groups = [rs.AdamGroup(q["p"], q["g"], q["m"], q["v"], q["lr"], q["act"], q["a"]) for q in s["groups"]]
    rs.rs_adam_step_clipped(groups, s["step"], s["max_norm"], s["norm"], s["workspace"], **ADAM)
    return _adam_outputs(s)


def _adam_outputs(s):
    return {"norm": s["norm"], "groups": [{x: q[x] for x in ("p", "m", "v", "a") if q[x] is not None}
                                          for q in s["groups"]]}


# ------------------------------------------------------------------ the plain forms

def _dequantised(q, scales, blocks=False):
    f = scales.repeat_interleave(BLOCK, 0)[:q.shape[1]].t()
    if blocks:
        f = f.repeat_interleave(BLOCK, 0)[:q.shape[0]]
    return q.float() * f


def _adam_plain(q, coef, b1, b2, eps, step):
    g = q["g"] * coef
    if q["act"] == 1:
        g = g * q["p"].exp()
    elif q["act"] == 2:
        a = q["p"].sigmoid()
        g = g * a * (1 - a)
    q["m"].mul_(b1).add_(g, alpha=1 - b1)
    q["v"].mul_(b2).add_(g * g, alpha=1 - b2)
    q["p"].sub_(q["lr"] * (q["m"] / (1 - b1 ** step)) / ((q["v"] / (1 - b2 ** step)).sqrt() + eps))
    if q["act"]:
        q["a"].copy_(q["p"].exp() if q["act"] == 1 else q["p"].sigmoid())


def _chain(q):
    """The group's gradient with respect to its stored parameter."""
    if q["act"] == 1:
        return q["g"] * q["p"].exp()
    if q["act"] == 2:
        a = q["p"].sigmoid()
        return q["g"] * a * (1 - a)
    return q["g"]


def run(s):
    if own:
        return _run_own(s)
    op = s["case"]["op"]
    if op == "norm":
        x = s["x"].float()
        if s["residual"] is not None:
            x = x + s["residual"].float()
        rstd = (x.square().mean(1) + EPS).rsqrt()
        q, scales = _quantised(x * rstd.unsqueeze(1) * s["weight"])
        out = {"q": q, "scales": scales, "rstd": rstd}
        return out | {"sum": x.to(s["x"].dtype)} if s["residual"] is not None else out
    if op == "norm_bwd":
        x, dy, rstd = s["x"].float(), s["dy"].float(), s["rstd"].unsqueeze(1)
        xh, t = x * rstd, dy * s["weight"]
        dx = rstd * (t - xh * (t * xh).mean(1, keepdim=True)) + s["dsum"].float()
        return {"dx": dx.to(s["x"].dtype), "dweight": (dy * xh).sum(0)}
    if op == "matmul":
        a, b = _dequantised(s["a"], s["a_scales"]), _dequantised(s["b"], s["b_scales"], blocks=True)
        return {"out": (a @ b.t()).to(s["out"].dtype)}
    if op == "matmul_bwd":
        du = s["du"].float() * (s["u"] > 0)
        dq, dqt, xqt = (_dequantised(*_quantised(v)) for v in (du, du.t(), s["x"].float().t()))
        wt = _dequantised(s["wt"], s["wt_scales"], blocks=True)
        return {"dx": (dq @ wt.t()).to(s["dx"].dtype), "dw": dqt @ xqt.t()}
    if op == "clip":
        norm = torch.stack([x.float().square().sum() for x in s["grads"]]).sum().sqrt()
        coef = (s["max_norm"] / (norm + 1e-6)).clamp(max=1.0)
        return {"norm": norm.view(1), "outs": [(x.float() * coef).to(x.dtype) for x in s["grads"]]}
    norm = torch.stack([_chain(q).square().sum() for q in s["groups"]]).sum().sqrt()
    coef = (s["max_norm"] / (norm + 1e-6)).clamp(max=1.0)
    s["norm"].copy_(norm.view(1))
    [_adam_plain(q, coef, ADAM["beta1"], ADAM["beta2"], ADAM["eps"], s["step"]) for q in s["groups"]]
    return _adam_outputs(s)


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    op = case["op"]
    if op in ("norm", "norm_bwd"):
        r, c, b = case["rows"], case["cols"], BYTES[case["dtype"]]
        if op == "norm":
            return {"bytes": r * c * (b * (3 if case["residual"] else 1) + 1) + 4 * r * (-(-c // BLOCK) + 1) + 4 * c,
                    "flops": 7 * r * c}
        return {"bytes": 4 * b * r * c + 4 * r + 8 * c, "flops": 11 * r * c}
    if op in ("matmul", "matmul_bwd"):
        m, n, k = case["rows"], case["n"], case["k"]
        if op == "matmul":
            kb = -(-k // BLOCK)
            return {"bytes": m * k + n * k + m * n * BYTES[case["out"]] + 4 * kb * (m + -(-n // BLOCK)),
                    "flops": 2 * m * n * k}
        return {"bytes": 2 * (2 * m * n + 2 * m * k) + 5 * n * k, "flops": 4 * m * n * k}
    if op == "clip":
        kinds = ["f32", "bf16", "f16"] if case["dtype"] == "mixed" else [case["dtype"]]
        sizes = np.random.RandomState(case["tensors"]).uniform(0.05, 2.0, case["tensors"])
        counts = [(max(1, int(case["mean"] * u)), BYTES[kinds[i % len(kinds)]]) for i, u in enumerate(sizes)]
        return {"bytes": sum(2 * k * b for k, b in counts), "flops": sum(3 * k for k, _ in counts)}
    n = case["gaussians"]
    return {"bytes": 4 * n * (59 * 7 + 4), "flops": 59 * n * 17}


# ------------------------------------------------------------------ the definitions in 64 bits

def _e4m3(x):
    """x (64 bits) rounded to the nearest e4m3 value, ties to even: 4 significant bits, steps of 2^-9 below 2^-6."""
    e = torch.frexp(x)[1].clamp_min(-5)
    step = torch.ldexp(torch.ones_like(x), e - 4)
    return ((x / step).round() * step).clamp(-448.0, 448.0)


def _as_8bit(x):
    """The values that the 8-bit form of x [r][c] with a scale for each row and 128 columns stands for, 64 bits; by
    definition a block's two factors, 448 / A and A / 448, and the scaled value that is rounded are of 32 bits (16-bit
    inputs often fall on a tie exactly, so the definition has to say which number is rounded)."""
    got = []
    for p in x.split(BLOCK, 1):
        top = p.abs().amax(1, keepdim=True).clamp_min(2.0 ** -100)
        inv, scale = (v.float().double() for v in (torch.full_like(top, 448.0) / top, top / 448.0))
        got.append(_e4m3((p * inv).float().double()) * scale)
    return torch.cat(got, 1)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    d = lambda t: t.to(torch.float32).double() if t.dtype != torch.float32 else t.double()
    if op == "norm":
        # the 8-bit output's value before its rounding to 8 bits
        x = d(s["x"]) + (d(s["residual"]) if s["residual"] is not None else 0)
        rstd = 1 / (x.pow(2).sum(1) / x.shape[1] + EPS).sqrt()
        y = x * rstd[:, None] * d(s["weight"])
        tops = [p.abs().amax(1).clamp_min(2.0 ** -100) / 448.0 for p in y.split(BLOCK, 1)]
        out = {"q": torch.cat([p / t[:, None] for p, t in zip(y.split(BLOCK, 1), tops)], 1),
               "scales": torch.stack(tops), "rstd": rstd}
        return out | {"sum": x} if s["residual"] is not None else out
    if op == "norm_bwd":
        x, dy, w, rho = d(s["x"]), d(s["dy"]), d(s["weight"]), d(s["rstd"])[:, None]
        inner = (dy * w * x).sum(1, keepdim=True) / x.shape[1]
        return {"dx": rho * dy * w - rho.pow(3) * x * inner + d(s["dsum"]), "dweight": (rho * x * dy).sum(0)}
    if op == "matmul":
        m, n, k = case["rows"], case["n"], case["k"]
        total = 0
        for kb in range(-(-k // BLOCK)):
            cut = slice(kb * BLOCK, min(k, (kb + 1) * BLOCK))
            sb = d(s["b_scales"])[kb][torch.arange(n, device="cuda") // BLOCK]
            total = total + (d(s["a"][:, cut]) @ d(s["b"][:, cut]).t()) * d(s["a_scales"])[kb][:, None] * sb[None, :]
        return {"out": total}
    if op == "matmul_bwd":
        du = torch.where(s["u"] > 0, d(s["du"]), torch.zeros((), dtype=torch.float64, device="cuda"))
        wt, ws = d(s["wt"]), d(s["wt_scales"])
        wt = wt * ws.repeat_interleave(BLOCK, 0)[:wt.shape[1]].t().repeat_interleave(BLOCK, 0)[:wt.shape[0]]
        dx = _as_8bit(du) @ wt.t()
        return {"dx": dx, "dw": _as_8bit(du.t()) @ _as_8bit(d(s["x"]).t()).t()}
    if op == "clip":
        norm = math.sqrt(sum(float(d(x).pow(2).sum()) for x in s["grads"]))
        c = min(1.0, s["max_norm"] / (norm + 1e-6))
        return {"norm": torch.tensor([norm], dtype=torch.float64), "outs": [d(x) * c for x in s["grads"]]}
    slope = {0: lambda p: torch.ones_like(p), 1: torch.exp, 2: lambda p: torch.sigmoid(p) * torch.sigmoid(-p)}
    grads = [d(q["g"]) * slope[q["act"]](d(q["p"])) for q in s["groups"]]
    norm = math.sqrt(sum(float(g.pow(2).sum()) for g in grads))
    c = min(1.0, s["max_norm"] / (norm + 1e-6))
    b1, b2, t = ADAM["beta1"], ADAM["beta2"], s["step"]
    groups = []
    for q, g in zip(s["groups"], grads):
        m, v = b1 * d(q["m"]) + (1 - b1) * c * g, b2 * d(q["v"]) + (1 - b2) * (c * g) ** 2
        p = d(q["p"]) - q["lr"] * (m / (1 - b1 ** t)) / ((v / (1 - b2 ** t)).sqrt() + ADAM["eps"])
        groups.append({"p": p, "m": m, "v": v} | ({"a": p.exp() if q["act"] == 1 else p.sigmoid()} if q["act"] else {}))
    return {"norm": torch.tensor([norm], dtype=torch.float64), "groups": groups}
