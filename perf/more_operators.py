"""The operators of gated residual blocks between two norms and of activation checkpoints in 8 bits, as measured cases.

Five kinds of case: the norms before and after a block with its gate and residual scale (`sandwich`) and their backward
(`sandwich_bwd`), an 8-bit matrix product whose result leaves in 8 bits (`matmul_q`), a checkpoint turned into the operand
of a weight's gradient (`transpose`) and a gradient through a relu whose output was kept in 8 bits (`relu8`).

8-bit values are e4m3; a block's scale is its largest magnitude / 448, scales are laid out one row per block of 128 along
the row.  Kept operands are such matrices.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "f16": 2, "bf16": 2}
FP8 = torch.float8_e4m3fn
BLOCK = 128
EPS = 1e-6
WORKSPACE = 96 << 20   # bytes of scratch that a training loop keeps for all of its calls


def listed():
    return [
        # one Gaussian's features through a block's end while serving: latency alone, nothing kept
        {"name": "sandwich, 1 row", "op": "sandwich", "rows": 1, "cols": 4096, "dtype": "bf16", "gate": "element",
         "scale": False, "kept": False},
        # a width that is no multiple of a block, one gate for each Gaussian, a learned residual scale
        {"name": "sandwich, odd width, a gate a row", "op": "sandwich", "rows": 4099, "cols": 777, "dtype": "f16",
         "gate": "row", "scale": True, "kept": True},
        # every Gaussian of the 250k training scene, gated by element, operands kept for the backward
        {"name": "sandwich, 250k rows", "op": "sandwich", "rows": 250000, "cols": 512, "dtype": "bf16",
         "gate": "element", "scale": True, "kept": True},
        # a handful of rows, no gate, float32 operands
        {"name": "sandwich backward, 37 rows", "op": "sandwich_bwd", "rows": 37, "cols": 1001, "dtype": "f32",
         "gate": "none", "scale": False, "kept": False},
        # a gate a row, operands as they were
        {"name": "sandwich backward, 10k rows", "op": "sandwich_bwd", "rows": 10007, "cols": 1000, "dtype": "f16",
         "gate": "row", "scale": True, "kept": False},
        # the 160k scene from its checkpoints
        {"name": "sandwich backward, 160k rows", "op": "sandwich_bwd", "rows": 160000, "cols": 512, "dtype": "bf16",
         "gate": "element", "scale": True, "kept": True},
        # a hidden layer's result kept in 8 bits: few rows of odd sizes, and the 160k scene
        {"name": "product kept, odd", "op": "matmul_q", "rows": 37, "n": 1001, "k": 777},
        {"name": "product kept, 160k rows", "op": "matmul_q", "rows": 160000, "n": 512, "k": 512},
        # a checkpoint as the operand of a weight's gradient
        {"name": "checkpoint transposed, odd", "op": "transpose", "rows": 2001, "cols": 777},
        {"name": "checkpoint transposed, 250k rows", "op": "transpose", "rows": 250000, "cols": 512},
        # a hidden layer's gradient through the relu that a checkpoint holds
        {"name": "relu from a checkpoint, odd", "op": "relu8", "rows": 2001, "cols": 200, "dtype": "f32"},
        {"name": "relu from a checkpoint, 160k rows", "op": "relu8", "rows": 160000, "cols": 512, "dtype": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, hi):
    """A width as networks have it (a multiple of 64) or an odd one."""
    w = _log(rng, 64, hi)
    return max(64, w // 64 * 64) if rng.random() < 0.6 else w | 1


def draw(rng):
    op = rng.choice(["sandwich", "sandwich", "sandwich_bwd", "sandwich_bwd", "matmul_q", "transpose", "relu8"])
    if op in ("sandwich", "sandwich_bwd"):
        cols = _width(rng, 2500)
        rows = _log(rng, 1, min(160000, 80_000_000 // cols))
        return {"op": op, "rows": rows, "cols": cols, "dtype": rng.choice(["f32", "f16", "bf16"]),
                "gate": rng.choice(["none", "row", "element"]), "scale": rng.random() < 0.5, "kept": rng.random() < 0.5}
    if op == "matmul_q":
        n, k = _width(rng, 1500), _width(rng, 1500)
        return {"op": op, "rows": _log(rng, 1, min(160000, 50_000_000 // max(n, k))), "n": n, "k": k}
    cols = _width(rng, 2500)
    c = {"op": op, "rows": _log(rng, 1, min(250000, 80_000_000 // cols)), "cols": cols}
    return c | {"dtype": rng.choice(["f32", "f16", "bf16"])} if op == "relu8" else c


# ------------------------------------------------------------------ inputs

def _quantised(x, blocks=False):
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
    """q with rows padded to a multiple of 16 bytes, as the kernels read them."""
    r, c = q.shape
    out = torch.zeros(r, -(-c // 16) * 16, dtype=torch.uint8, device=q.device)
    out[:, :c] = q.view(torch.uint8)
    return out.view(FP8)[:, :c]


def _kept(x):
    q, sc = _quantised(x)
    return _rows16(q), sc.contiguous()


def _empty8(r, c):
    return (torch.empty(r, -(-c // 16) * 16, dtype=torch.uint8, device="cuda").view(FP8)[:, :c],
            torch.empty(-(-c // BLOCK), r, device="cuda"))


def prepare(case, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    rand = lambda *s: torch.randn(*s, device="cuda", generator=g)
    op, r = case["op"], case["rows"]
    s = {"case": dict(case), "workspace": torch.empty(WORKSPACE, dtype=torch.uint8, device="cuda")}
    if op in ("sandwich", "sandwich_bwd"):
        c, dt = case["cols"], DTYPES[case["dtype"]]
        outlier = 1 + 8 * (torch.rand(c, device="cuda", generator=g) < 0.01)      # some features run larger
        s["x"] = (rand(r, c) * outlier).to(dt)
        s["r"] = (0.5 * rand(r, c)).to(dt)
        s["gate"] = (1.5 * rand(r, {"row": 1, "element": c}[case["gate"]])).to(dt) if case["gate"] != "none" else None
        s["residual_scale"] = 1 + 0.1 * rand(c) if case["scale"] else None
        s["post_weight"], s["pre_weight"] = 1 + 0.2 * rand(c), 1 + 0.2 * rand(c)
        if op == "sandwich":
            s["q"], s["scales"] = _empty8(r, c)
            s["sum"] = torch.empty_like(s["x"])
            s["rstd_r"], s["rstd_s"] = torch.empty(r, device="cuda"), torch.empty(r, device="cuda")
            kept = ["x", "r"] + (["gate"] if case["gate"] == "element" else []) if case["kept"] else []
            s["kept"] = {k: _empty8(r, c) for k in kept}
        else:
            # what the forward left: the statistics of its operands, and the operands or their checkpoints
            ssum, s["rstd_r"], s["rstd_s"] = _forward(s)[:3]
            del ssum
            if case["kept"]:
                for k in ("x", "r") + (("gate",) if case["gate"] == "element" else ()):
                    s[k] = _kept(s[k])
            s["dy"], s["dsum"] = rand(r, c).to(dt), rand(r, c).to(dt)
            s["dx"], s["dr"] = torch.empty_like(s["dy"]), torch.empty_like(s["dy"])
            s["dgate"] = (None if s["gate"] is None else torch.empty_like(s["dy"]) if case["gate"] == "element" else
                          torch.empty(r, 1, dtype=dt, device="cuda"))
            s["dpost"], s["dpre"] = torch.empty(c, device="cuda"), torch.empty(c, device="cuda")
            s["dscale"] = torch.empty(c, device="cuda") if case["scale"] else None
    elif op == "matmul_q":
        n, k = case["n"], case["k"]
        s["a"], s["a_scales"] = _kept(rand(r, k) * (1 + torch.rand(r, 1, device="cuda", generator=g)))
        q, s["b_scales"] = _quantised(rand(n, k) / math.sqrt(k), blocks=True)
        s["b"] = _rows16(q)
        s["q"], s["scales"] = _empty8(r, n)
    elif op == "transpose":
        c = case["cols"]
        s["q"], s["scales"] = _kept(rand(r, c) * (1 + torch.rand(r, 1, device="cuda", generator=g)))
        s["qt"], s["scales_t"] = _empty8(c, r)
    else:
        c, dt = case["cols"], DTYPES[case["dtype"]]
        s["du"] = (rand(r, c) * 1e-3).to(dt)
        s["u"], _ = _kept(rand(r, c).relu())
        s["q"], s["scales"] = _empty8(r, c)
        s["qt"], s["scales_t"] = _empty8(c, r)
    return s


# ------------------------------------------------------------------ the framework's operators

def _run_own(s):
    from gaussian_splatting_tile_gb300 import rs
    op = s["case"]["op"]
    if op == "sandwich":
        rs.rs_sandwich_norm_fwd(s["x"], s["r"], s["post_weight"], s["pre_weight"], s["q"], s["scales"], gate=s["gate"],
                                residual_scale=s["residual_scale"], sum=s["sum"], rstd_r=s["rstd_r"],
                                rstd_s=s["rstd_s"], kept_x=s["kept"].get("x"), kept_r=s["kept"].get("r"),
                                kept_gate=s["kept"].get("gate"), eps=EPS)
        return {k: s[k] for k in ("sum", "rstd_r", "rstd_s", "q", "scales", "kept")}
    if op == "sandwich_bwd":
        rs.rs_sandwich_norm_bwd(s["x"], s["r"], s["post_weight"], s["pre_weight"], s["rstd_r"], s["rstd_s"], s["dy"],
                                s["dx"], s["dr"], s["workspace"], gate=s["gate"], dL_dgate=s["dgate"],
                                residual_scale=s["residual_scale"], dL_dsum=s["dsum"], dL_dpost_weight=s["dpost"],
                                dL_dpre_weight=s["dpre"], dL_dresidual_scale=s["dscale"])
        return {k: s[k] for k in ("dx", "dr", "dgate", "dpost", "dpre", "dscale") if s[k] is not None}
    if op == "matmul_q":
        rs.rs_matmul_fp8_q(s["a"], s["a_scales"], s["b"], s["b_scales"], s["q"], s["scales"], s["workspace"], relu=True)
        return {"q": s["q"], "scales": s["scales"]}
    if op == "transpose":
        rs.rs_transpose_fp8(s["q"], s["scales"], s["qt"], s["scales_t"])
        return {"qt": s["qt"], "scales_t": s["scales_t"]}
    rs.rs_quantize_fp8_relu8(s["du"], s["u"], s["q"], s["scales"], s["qt"], s["scales_t"])
    return {k: s[k] for k in ("q", "scales", "qt", "scales_t")}


# ------------------------------------------------------------------ the plain forms

def _dequantised(q, scales, blocks=False):
    f = scales.repeat_interleave(BLOCK, 0)[:q.shape[1]].t()
    if blocks:
        f = f.repeat_interleave(BLOCK, 0)[:q.shape[0]]
    return q.float() * f


def _operand(v):
    """A stored matrix or a checkpoint (q, scales), in 32 bits."""
    return _dequantised(*v) if isinstance(v, tuple) else v.float()


def _forward(s, rstd_r=None):
    """(sum, rstd_r, rstd_s, g, rh) in 32 bits."""
    x, r = _operand(s["x"]), _operand(s["r"])
    if rstd_r is None:
        rstd_r = (r.square().mean(1) + EPS).rsqrt()
    rh = r * rstd_r.unsqueeze(1)
    g = 1.0 / (1.0 + (-_operand(s["gate"])).exp()) if s["gate"] is not None else torch.ones(1, 1, device="cuda")
    total = (x if s["residual_scale"] is None else x * s["residual_scale"]) + g * (rh * s["post_weight"])
    return total, rstd_r, (total.square().mean(1) + EPS).rsqrt(), g, rh


def run(s):
    if own:
        return _run_own(s)
    op = s["case"]["op"]
    if op == "sandwich":
        total, rstd_r, rstd_s, _, _ = _forward(s)
        q, scales = _quantised(total * rstd_s.unsqueeze(1) * s["pre_weight"])
        return {"sum": total.to(s["x"].dtype), "rstd_r": rstd_r, "rstd_s": rstd_s, "q": q, "scales": scales,
                "kept": {k: _quantised(s[k]) for k in s["kept"]}}
    if op == "sandwich_bwd":
        total, _, _, g, rh = _forward(s, s["rstd_r"])
        dt, rho = s["dy"].dtype, s["rstd_s"].unsqueeze(1)
        sh, dy = total * rho, s["dy"].float()
        t = dy * s["pre_weight"]
        ds = rho * (t - sh * (t * sh).mean(1, keepdim=True)) + s["dsum"].float()
        dn = ds * g
        v = dn * s["post_weight"]
        dr = s["rstd_r"].unsqueeze(1) * (v - rh * (v * rh).mean(1, keepdim=True))
        out = {"dx": (ds if s["residual_scale"] is None else ds * s["residual_scale"]).to(dt), "dr": dr.to(dt)}
        if s["gate"] is not None:
            dg = ds * rh * s["post_weight"]
            if s["dgate"].shape[1] == 1:
                dg = dg.sum(1, keepdim=True)
            e = (-_operand(s["gate"])).exp()
            out["dgate"] = (dg * e / (1.0 + e).square()).to(dt)
        out |= {"dpost": (dn * rh).sum(0), "dpre": (dy * sh).sum(0)}
        return out | {"dscale": (ds * _operand(s["x"])).sum(0)} if s["residual_scale"] is not None else out
    if op == "matmul_q":
        a, b = _dequantised(s["a"], s["a_scales"]), _dequantised(s["b"], s["b_scales"], blocks=True)
        q, scales = _quantised((a @ b.t()).clamp_min(0.0))
        return {"q": q, "scales": scales}
    if op == "transpose":
        qt, scales = _quantised(_dequantised(s["q"], s["scales"]).t().contiguous())
        return {"qt": qt, "scales_t": scales}
    du = s["du"].float() * (s["u"].float() > 0)
    (q, sc), (qt, sct) = _quantised(du), _quantised(du.t().contiguous())
    return {"q": q, "scales": sc, "qt": qt, "scales_t": sct}


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    op, r = case["op"], case["rows"]
    if op in ("sandwich", "sandwich_bwd"):
        c, b = case["cols"], BYTES[case["dtype"]]
        kb, gates = -(-c // BLOCK), {"none": 0, "row": r, "element": r * c}[case["gate"]]
        kept = (3 if case["gate"] == "element" else 2) if case["kept"] else 0
        vectors = 4 * c * (2 + case["scale"])
        if op == "sandwich":
            return {"bytes": b * (3 * r * c + gates) + (1 + kept) * (r * c + 4 * r * kb) + 8 * r + vectors,
                    "flops": 30 * r * c}
        operands = kept * (r * c + 4 * r * kb) + (0 if case["gate"] == "element" else b * gates) if kept else \
            b * (2 * r * c + gates)
        return {"bytes": operands + b * (4 * r * c + gates) + 8 * r + 2 * vectors, "flops": 45 * r * c}
    if op == "matmul_q":
        n, k = case["n"], case["k"]
        return {"bytes": r * k + n * k + r * n + 4 * -(-k // BLOCK) * (r + -(-n // BLOCK)) + 4 * -(-n // BLOCK) * r,
                "flops": 2 * r * n * k}
    c = case["cols"]
    forms = r * c + 4 * r * -(-c // BLOCK), r * c + 4 * c * -(-r // BLOCK)      # by rows, by columns
    if op == "transpose":
        return {"bytes": sum(forms), "flops": 4 * r * c}
    return {"bytes": sum(forms) + r * c * (BYTES[case["dtype"]] + 1), "flops": 6 * r * c}


# ------------------------------------------------------------------ the definitions in 64 bits

def _tops(y):
    """[c/128][r]: what a block's scale is times 448."""
    return torch.stack([p.abs().amax(1).clamp_min(2.0 ** -100) for p in y.split(BLOCK, 1)])


def _over_scales(y):
    """(scaled values before their rounding to 8 bits, scales) of y in 64 bits."""
    sc = _tops(y) / 448.0
    return torch.cat([p / f[:, None] for p, f in zip(y.split(BLOCK, 1), sc)], 1), sc


def _e4m3(x):
    """x (64 bits) rounded to the nearest e4m3 value, ties to even: 4 significant bits, steps of 2^-9 below 2^-6."""
    e = torch.frexp(x)[1].clamp_min(-5)
    step = torch.ldexp(torch.ones_like(x), e - 4)
    return ((x / step).round() * step).clamp(-448.0, 448.0)


def _form(v):
    """(e4m3 values, scales) of v, whose elements are numbers of 32 bits: by definition a block's two factors, 448 / A and
    A / 448, and the scaled value that is rounded are of 32 bits, so that what falls on a tie is the same everywhere."""
    top = _tops(v)
    inv = (torch.full_like(top, 448.0) / top).float().double()
    q = torch.cat([_e4m3((p * f[:, None]).float().double()) for p, f in zip(v.split(BLOCK, 1), inv)], 1)
    return q, (top / 448.0).float().double()


def _wide(v):
    """A stored matrix or a checkpoint's values in 64 bits."""
    if not isinstance(v, tuple):
        return v.double()
    q, sc = v
    col = torch.arange(q.shape[1], device=q.device) // BLOCK
    return q.float().double() * sc.double()[col].t()


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("sandwich", "sandwich_bwd"):
        x, r = _wide(s["x"]), _wide(s["r"])
        wpost, wpre = s["post_weight"].double(), s["pre_weight"].double()
        z = None if s["gate"] is None else _wide(s["gate"])
        g = 1.0 if z is None else torch.sigmoid(z)
        alpha = 1.0 if s["residual_scale"] is None else s["residual_scale"].double()
    if op == "sandwich":
        rho_r = 1 / (r.pow(2).sum(1) / r.shape[1] + EPS).sqrt()
        total = alpha * x + g * (r * rho_r[:, None] * wpost)
        rho_s = 1 / (total.pow(2).sum(1) / r.shape[1] + EPS).sqrt()
        q, scales = _over_scales(total * rho_s[:, None] * wpre)
        return {"sum": total, "rstd_r": rho_r, "rstd_s": rho_s, "q": q, "scales": scales,
                "kept": {k: _form(s[k].double()) for k in s["kept"]}}
    if op == "sandwich_bwd":
        c, rho_r, rho_s = r.shape[1], s["rstd_r"].double()[:, None], s["rstd_s"].double()[:, None]
        total = alpha * x + g * (r * rho_r * wpost)
        dy = s["dy"].double()
        inner = (dy * wpre * total).sum(1, keepdim=True) / c
        ds = rho_s * dy * wpre - rho_s.pow(3) * total * inner + s["dsum"].double()
        b = ds * g * wpost                                             # the gradient of r / rms(r)
        dr = rho_r * b - rho_r.pow(3) * r * ((b * r).sum(1, keepdim=True) / c)
        out = {"dx": alpha * ds, "dr": dr}
        if z is not None:
            dz = ds * r * rho_r * wpost
            if case["gate"] == "row":
                dz = dz.sum(1, keepdim=True)
            out["dgate"] = dz * torch.sigmoid(z) * torch.sigmoid(-z)
        out |= {"dpost": (ds * g * r * rho_r).sum(0), "dpre": (dy * total * rho_s).sum(0)}
        return out | {"dscale": (ds * x).sum(0)} if case["scale"] else out
    if op == "matmul_q":
        a, n = _wide((s["a"], s["a_scales"])), case["n"]
        total = 0
        for kb, cut in enumerate(range(0, case["k"], BLOCK)):
            sb = s["b_scales"].double()[kb][torch.arange(n, device="cuda") // BLOCK]
            total = total + a[:, cut:cut + BLOCK] @ (s["b"][:, cut:cut + BLOCK].float().double() * sb[:, None]).t()
        q, scales = _over_scales(torch.relu(total))
        return {"q": q, "scales": scales}
    if op == "transpose":
        v = _wide((s["q"], s["scales"])).float().double()              # by definition the value is the product in 32 bits
        qt, scales = _form(v.t().contiguous())
        return {"qt": qt, "scales_t": scales}
    du = torch.where(s["u"].float() > 0, s["du"].double(), torch.zeros((), dtype=torch.float64, device="cuda"))
    (q, sc), (qt, sct) = _form(du), _form(du.t().contiguous())
    return {"q": q, "scales": sc, "qt": qt, "scales_t": sct}
