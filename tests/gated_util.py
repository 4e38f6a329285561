"""Plain 64-bit forms of the gated linear recurrence and of the token norm (torch on the CPU),
and the error bounds that their kernels are held to.

Bounds.  Every output is a sum of products of inputs and decays.  Running the same form on the
inputs' absolute values gives the sum A of the terms' magnitudes, and an element's error is at
most (number of roundings on a term's way) u A, u = 2^-24.  On the recurrence: a product chain
over d features and 64 tokens, a decay (its argument's rounding, at most 126 ln 2 u for a decay
that is not 0, and 2 u for the function), the rate, and per later chunk the state's own product
and sum: n = 64 + 2 d + 90 + 8 + 4 ceil(T / 64).  Outputs in bfloat16 add the last rounding,
2^-8 of the value, and may come from factors split into two bfloat16 parts, which are off by
2^-8 2^-8 of a term: 2^-16 A twice, on the products inside a chunk and on the state.
"""
import numpy as np
import torch

U = 2.0 ** -24
BF16_HALF = 2.0 ** -8


def gated_inputs(B, H, T, d, io, gate="soft", rates=False, lengths=None, batch_w0=False, seed=0):
    """Seeded CPU inputs, in the I/O dtype where that applies."""
    rng = np.random.default_rng(seed)
    dt = torch.bfloat16 if io == "bf16" else torch.float32
    normal = lambda *s: torch.from_numpy(rng.standard_normal(s).astype(np.float32))
    x = {n: normal(B, H, T, d).to(dt) for n in ("q", "k", "v", "dz")}
    x["k"] = (x["k"].float() / d ** 0.5).to(dt)
    x["w0"] = 0.3 * (normal(B, H, d, d) if batch_w0 else normal(H, d, d))
    x["dw_out"] = normal(B, H, d, d)
    u = torch.from_numpy(rng.uniform(size=(B, H, T)).astype(np.float32))
    g = {"none": None, "soft": -0.1 * u, "strong": -20.0 * u, "grow": 0.05 * (u - 0.5),
         "zero": torch.zeros(B, H, T)}.get(gate, -0.1 * u)
    if gate == "resets":
        g = torch.where(u < 0.05, torch.full_like(g, -float("inf")), g)
    if gate == "lowest":  # the type's lowest value, and the first and last tokens
        g = torch.where(u < 0.05, torch.full_like(g, torch.finfo(torch.float32).min), g)
        g[..., 0] = g[..., -1] = torch.finfo(torch.float32).min
    x["log_gate"] = g
    x["eta_tok"] = torch.from_numpy(rng.uniform(size=(B, H, T)).astype(np.float32)) if rates else None
    x["lengths"] = torch.tensor(lengths, dtype=torch.int32) if lengths is not None else None
    x["eta"] = 0.5
    return x


def gated_reference(x, with_dw_out=True, absolute=False, backward=True):
    """Token by token in float64: a dict of outputs and gradients."""
    f = (lambda t: t.double().abs()) if absolute else (lambda t: t.double())
    q, k, v, dz = (f(x[n]) for n in ("q", "k", "v", "dz"))
    B, H, T, d = q.shape
    w = f(x["w0"]).expand(B, H, d, d)
    a = torch.exp(x["log_gate"].double()) if x["log_gate"] is not None else torch.ones(B, H, T).double()
    a = torch.where(a.float() == 0, torch.zeros_like(a), a)
    e = x["eta"] * (x["eta_tok"].double() if x["eta_tok"] is not None else torch.ones(B, H, T).double())
    live = torch.ones(B, H, T).double()
    if x["lengths"] is not None:
        live = (torch.arange(T)[None] < x["lengths"][:, None]).double()[:, None].expand(B, H, T)
    a, e = a * live + (1 - live), e * live
    q, k, v, dz = (torch.where(live[..., None] > 0, t, torch.zeros_like(t)) for t in (q, k, v, dz))
    keep = lambda at, s: torch.where(at == 0, torch.zeros_like(s), at * s)
    states, z = [w], torch.zeros(B, H, T, d).double()
    for t in range(T):
        w = keep(a[:, :, t, None, None], w) + e[:, :, t, None, None] * v[:, :, t, :, None] * k[:, :, t, None, :]
        z[:, :, t] = (w @ q[:, :, t, :, None])[..., 0]
        states.append(w)
    out = {"z": z, "w_out": w}
    if not backward:
        return out
    gw = f(x["dw_out"]) if with_dw_out else torch.zeros(B, H, d, d).double()
    for n in ("dq", "dk", "dv"):
        out[n] = torch.zeros(B, H, T, d).double()
    out["dlog_gate"], out["deta_tok"] = torch.zeros(B, H, T).double(), torch.zeros(B, H, T).double()
    for t in reversed(range(T)):
        gw = gw + dz[:, :, t, :, None] * q[:, :, t, None, :]
        out["dq"][:, :, t] = (dz[:, :, t, None, :] @ states[t + 1])[:, :, 0]
        gk = (gw @ k[:, :, t, :, None])[..., 0]
        out["dv"][:, :, t] = e[:, :, t, None] * gk
        out["dk"][:, :, t] = e[:, :, t, None] * (v[:, :, t, None, :] @ gw)[:, :, 0]
        out["deta_tok"][:, :, t] = x["eta"] * (v[:, :, t] * gk).sum(-1) * live[:, :, t]
        out["dlog_gate"][:, :, t] = keep(a[:, :, t], (gw * states[t]).sum((-1, -2))) * live[:, :, t]
        gw = keep(a[:, :, t, None, None], gw)
    out["dw0"] = gw
    out["qdq"], out["kdk"] = (q * out["dq"]).sum(-1), (k * out["dk"]).sum(-1)
    return out


def gated_bounds(x, ref, with_dw_out=True, backward=True):
    """Largest allowed |error| per output element (see the module's text)."""
    q = x["q"]
    B, H, T, d = q.shape
    mag = gated_reference(x, with_dw_out, absolute=True, backward=backward)
    n = 64 + 2 * d + 98 + 4 * -(-T // 64)
    half = BF16_HALF if q.dtype == torch.bfloat16 else 0.0
    split = 2 * 2.0 ** -16 if q.dtype == torch.bfloat16 else 0.0
    tol = {}
    for name in ("z", "dq", "dk", "dv") if backward else ("z",):
        tol[name] = half * ref[name].abs() + (1 + half) * (n * U + split) * mag[name] + 1e-30
    for name in ("w_out", "dw0", "deta_tok") if backward else ("w_out",):
        tol[name] = n * U * mag[name] + 1e-30
    if backward:
        # dlog_gate also sums its chunk's row and column sums, which cancel in part
        m = mag["qdq"] + mag["kdk"]
        m = torch.nn.functional.pad(m, (0, -T % 64)).reshape(B, H, -1, 64).sum(-1, keepdim=True).expand(-1, -1, -1, 64)
        tol["dlog_gate"] = n * U * (mag["dlog_gate"] + m.reshape(B, H, -1)[..., :T]) + 1e-30
    return tol


def assert_within(name, got, ref, tol):
    got = got.detach().cpu().double()
    assert got.shape == ref.shape, (name, got.shape, ref.shape)
    assert torch.isfinite(got).all(), f"{name}: not finite"
    over = (got - ref).abs() / tol
    worst = float(over.max()) if over.numel() else 0.0
    print(f"{name}: at most {worst:.3f} of the bound", flush=True)
    assert worst <= 1.0, f"{name}: {worst:.3g} times the bound at {np.unravel_index(int(over.argmax()), over.shape)}"


def norm_reference(p, kind, act, eps, dy=None):
    """Token norm in float64 on dict p (x and any of weight, bias, gate, scale, res): y, or its
    gradients by autograd when dy is given."""
    t = {n: v.double().detach().requires_grad_(dy is not None) for n, v in p.items() if v is not None}
    x = t["x"]
    if kind == "layer":
        x = x - x.mean(-1, keepdim=True)
    s = (x * x).sum(-1, keepdim=True)
    n = x / torch.sqrt((s if kind == "l2" else s / x.shape[-1]) + eps)
    per_head = lambda w: w[None, :, None, :]
    if "weight" in t:
        n = n * per_head(t["weight"])
    if "bias" in t:
        n = n + per_head(t["bias"])
    if "gate" in t:
        g = t["gate"]
        n = n * {"none": g, "silu": g * torch.sigmoid(g), "sigmoid": torch.sigmoid(g),
                 "gelu": 0.5 * g * (1 + torch.erf(g / 2 ** 0.5))}[act]
    if "scale" in t:
        n = n * per_head(t["scale"])
    if "res" in t:
        n = n + t["res"]
    if dy is None:
        return n
    names = list(t)
    return {"d" + k: g for k, g in zip(names, torch.autograd.grad(n, [t[k] for k in names], dy.double()))}


def norm_bounds(p, kind, act, eps, ref_y=None, dy=None, ref=None):
    """Bounds as above.  A centred value is off by u (|x| + |mean|); a row's sum of up to 16384
    terms is taken by at most 64 lanes-or-waves steps of at most 64 terms each (n = 128); the
    activations are off by (8 + |g|) u of themselves, GELU by as much of |g| (it subtracts)."""
    x = p["x"].double()
    m = x.mean(-1, keepdim=True).abs() if kind == "layer" else 0.0
    c = x - x.mean(-1, keepdim=True) if kind == "layer" else x
    s = (c * c).sum(-1, keepdim=True)
    d = x.shape[-1]
    r = 1 / torch.sqrt((s if kind == "l2" else s / d) + eps)
    xh = (x.abs() + m) * r
    # the centred sum of squares is off by 2 u (|x| + |m|) |c| a term
    xh = xh * (1 + (2 * (x.abs() + m) * c.abs()).sum(-1, keepdim=True) / (s + eps) / 128)
    per_head = lambda w: w.double().abs()[None, :, None, :] if w is not None else 1.0
    w, sc = per_head(p.get("weight")), per_head(p.get("scale"))
    b = per_head(p["bias"]) if p.get("bias") is not None else 0.0
    n = xh * w + b
    a, da, lose = 1.0, 0.0, 1.0
    if p.get("gate") is not None:
        g = p["gate"].double()
        s_ = torch.sigmoid(g)
        a = {"none": g.abs(), "silu": (g * s_).abs(), "sigmoid": s_, "gelu": g.abs()}[act]
        da = {"none": 1.0, "silu": s_ * (1 + g.abs()), "sigmoid": s_, "gelu": 1 + g.abs()}[act]
        lose = 1 + g.abs() / 128
    half = BF16_HALF if p["x"].dtype == torch.bfloat16 else 0.0
    N = 160 * U
    if dy is None:
        res = p["res"].double().abs() if p.get("res") is not None else 0.0
        return half * ref_y.abs() + (1 + half) * N * lose * (n * a * sc + res) + 1e-30
    dy = dy.double().abs()
    t = dy * a * sc * lose
    u = t * w
    mean = (lambda v: v.sum(-1, keepdim=True)) if kind == "l2" else (lambda v: v.mean(-1, keepdim=True))
    dx = r * (u + (u.mean(-1, keepdim=True) if kind == "layer" else 0.0) + xh * mean(u * xh))
    tol = {"dx": half * ref["dx"].abs() + (1 + half) * 3 * N * dx + 1e-30}
    if "dgate" in ref:
        tol["dgate"] = half * ref["dgate"].abs() + (1 + half) * N * lose * dy * sc * n * da + 1e-30
    # the parameters' sums: at most 512 more terms one after another
    for name, terms in (("dweight", t * xh), ("dbias", t), ("dscale", dy * a * lose * n)):
        if name in ref:
            tol[name] = (N + 512 * U) * terms.sum((0, 2)) + 1e-30
    return tol
