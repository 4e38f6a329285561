"""The operators around and beside the TTT layers, as measured cases.

Two groups, on token tensors [B, H, T, d]:

  the gated linear recurrence, with e = eta * eta_tok[t] and a decay exp(log_gate[t]):
      W_t = exp(g_t) W_{t-1} + e_t v_t k_t^T,   z_t = W_t q_t
    gated_linear_fwd (z and the final state), gated_linear_bwd (all gradients) and
    gated_linear_step (one token per sequence, the state updated in place);

  the norm before and after such a layer, over the d features of a token,
      y = res + scale * act(gate) * (norm(x) * weight + bias)
    token_norm_fwd and token_norm_bwd.

With own = False the cases run in plain torch operations; with own = True through this package.
"""
import math

import torch
import torch.nn.functional as F

own = False

_DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
_CHUNK = 64  # tokens per chunk of the plain form of the recurrence


def listed():
    def gl(name, op, dtype, B, H, T, d, gate="soft", rates=False, ragged=False):
        return {"name": name, "op": op, "dtype": dtype, "B": B, "H": H, "T": T, "d": d,
                "gate": gate, "rates": rates, "ragged": ragged}

    def norm(name, op, dtype, B, H, T, d, kind, after):
        return {"name": name, "op": op, "dtype": dtype, "B": B, "H": H, "T": T, "d": d,
                "kind": kind, "act": "silu" if after else "none", "after": after}

    return [
        # one request answered token by token: latency of a single call
        gl("step_B1", "gl_step", "bf16", 1, 12, 1, 64),
        # a full serving batch, one token each: the states are read and written once
        gl("step_B512", "gl_step", "bf16", 512, 12, 1, 64, rates=True),
        # the smallest layer call (the tiny float32 workload's shape)
        gl("fwd_tiny_f32", "gl_fwd", "f32", 1, 1, 64, 16),
        # a training batch at the headline shape, with per-token rates
        gl("fwd_2k", "gl_fwd", "bf16", 8, 12, 2048, 64, rates=True),
        # one long packed sequence (documents end in resets), few heads, an odd length
        gl("fwd_long", "gl_fwd", "bf16", 1, 16, 32749, 64, gate="resets"),
        # a padded float32 batch at an odd length
        gl("bwd_ragged_f32", "gl_bwd", "f32", 3, 5, 1021, 32, rates=True, ragged=True),
        # the backward pass of the training batch
        gl("bwd_2k", "gl_bwd", "bf16", 8, 12, 2048, 64, rates=True),
        # the backward pass over long packed sequences, the largest case
        gl("bwd_8k", "gl_bwd", "bf16", 4, 16, 8192, 64, gate="resets"),
        # after the layer: per-head RMS norm, gate, residual scale, residual
        norm("norm_after", "norm_fwd", "bf16", 8, 12, 2048, 64, "rms", True),
        # before the layer: layer norm over the model width of a vision batch, float32
        norm("norm_before_f32", "norm_fwd", "f32", 64, 1, 196, 384, "layer", False),
        # their backward passes
        norm("norm_after_bwd", "norm_bwd", "bf16", 8, 12, 2048, 64, "rms", True),
        norm("norm_before_bwd", "norm_bwd", "bf16", 1, 1, 8191, 768, "layer", False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["gl_step", "gl_fwd", "gl_fwd", "gl_bwd", "gl_bwd", "norm_fwd", "norm_bwd"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op.startswith("norm"):
        after = rng.random() < 0.5
        c = {"op": op, "dtype": dtype, "B": _log(rng, 1, 16), "H": _log(rng, 1, 16),
             "T": _log(rng, 1, 8192), "d": _log(rng, 16, 8192),
             "kind": rng.choice(["rms", "layer", "l2"]),
             "act": rng.choice(["silu", "gelu", "sigmoid"]) if after else "none", "after": after}
        while c["B"] * c["H"] * c["T"] * c["d"] > 16_000_000:
            big = max(("B", "H", "T"), key=lambda n: c[n])
            c[big] = max(1, c[big] // 2)
        return c
    d = rng.choice([16, 32, 64, 64])
    c = {"op": op, "dtype": dtype, "B": _log(rng, 1, 16), "H": _log(rng, 1, 24),
         "T": _log(rng, 1, 16384), "d": d, "gate": rng.choice(["soft", "strong", "resets", "none"]),
         "rates": rng.random() < 0.5, "ragged": rng.random() < 0.3}
    if op == "gl_step":
        c["B"], c["T"], c["ragged"] = _log(rng, 1, 400), 1, False
    while c["B"] * c["H"] * c["T"] * d > 200_000 * 64:
        big = max(("B", "H", "T"), key=lambda n: c[n])
        c[big] = max(1, c[big] // 2)
    return c


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 13)
    dt = _DTYPES[case["dtype"]]
    B, H, T, d = case["B"], case["H"], case["T"], case["d"]

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)

    def uniform(*shape):
        return torch.rand(shape, generator=gen, device="cuda", dtype=torch.float32)

    s = {"case": case}
    if case["op"].startswith("norm"):
        s["x"] = normal(B, H, T, d).to(dt)
        s["weight"] = 1.0 + 0.1 * normal(H, d)
        s["bias"] = 0.1 * normal(H, d) if case["kind"] == "layer" else None
        s["gate"] = normal(B, H, T, d).to(dt) if case["after"] else None
        s["scale"] = 0.2 + 0.1 * normal(H, d) if case["after"] else None
        if case["op"] == "norm_fwd":
            s["res"] = normal(B, H, T, d).to(dt) if case["after"] else None
        else:
            s["dy"] = normal(B, H, T, d).to(dt)
        return s
    tok = (B, H, d) if case["op"] == "gl_step" else (B, H, T, d)
    s["q"], s["v"] = normal(*tok).to(dt), normal(*tok).to(dt)
    k = normal(*tok)
    s["k"] = (k / k.norm(dim=-1, keepdim=True)).to(dt)  # unit keys, as every linear workload here
    g = None
    if case["gate"] != "none":
        # a learned forget gate, sigmoid of a projection: memories of about 50 tokens (soft), of 2 (strong)
        g = F.logsigmoid(normal(*tok[:-1]) + (0.0 if case["gate"] == "strong" else 4.0))
        if case["gate"] == "resets":  # a new document about every 700 tokens
            g = torch.where(uniform(*tok[:-1]) < 1.0 / 700.0, torch.full_like(g, -math.inf), g)
    s["log_gate"] = g
    s["eta_tok"] = uniform(*tok[:-1]) if case["rates"] else None
    s["eta"] = 0.5
    if case["op"] == "gl_step":
        s["w"] = 0.02 * normal(B, H, d, d)
        return s
    s["w0"] = 0.02 * normal(H, d, d)
    s["lengths"] = None
    if case["ragged"]:
        n = torch.randint(0, T + 1, (B,), generator=gen, device="cuda")
        n[0] = T
        s["lengths"] = n.to(torch.int32)
    if case["op"] == "gl_bwd":
        s["dz"] = normal(*tok).to(dt)
        s["dw_out"] = normal(B, H, d, d)
    return s


# ---------------------------------------------------------------- the recurrence in plain torch

class _Chunks:
    """The recurrence taken _CHUNK tokens at a time: decays, and the states at every chunk's start.

    Logarithms of decays are summed in 64 bits; a decay that is 0 in 32 bits counts as a reset
    (`seg` numbers the stretches between resets)."""

    def __init__(self, s):
        q = s["q"]
        self.B, self.H, self.T, self.d = B, H, T, d = q.shape
        self.n = n = -(-T // _CHUNK)
        self.pad = n * _CHUNK - T
        dev = q.device
        t = torch.arange(T, device=dev)
        lengths = s["lengths"]
        self.live = (torch.ones(B, 1, T, dtype=torch.bool, device=dev) if lengths is None
                     else t < lengths.long()[:, None, None])
        g = s["log_gate"] if s["log_gate"] is not None else torch.zeros(B, H, T, device=dev)
        reset = (g < -104.0) & self.live
        self.reset = reset
        g = torch.where(reset | ~self.live, torch.zeros_like(g), g).double()
        e = torch.full((B, H, T), float(s["eta"]), device=dev)
        if s["eta_tok"] is not None:
            e = e * s["eta_tok"]
        e = torch.where(self.live, e, torch.zeros_like(e))
        self.e = self.per_token(e)                                    # [B, H, n, C]
        b = self.per_token(g).cumsum(-1)
        seg = self.per_token(reset.to(torch.int64)).cumsum(-1)
        tri = torch.ones(_CHUNK, _CHUNK, dtype=torch.bool, device=dev).tril()
        same = (seg[..., :, None] == seg[..., None, :]) & tri
        diff = torch.where(same, b[..., :, None] - b[..., None, :], torch.zeros((), dtype=torch.float64, device=dev))
        self.dec = torch.exp(diff.float()) * same                     # decay from token s to token u
        self.from_start = torch.exp(b.float()) * (seg == 0)           # chunk start to token u
        last_b, last_seg = b[..., -1:], seg[..., -1:]
        self.to_end = torch.exp((last_b - b).float()) * (seg == last_seg)
        self.whole = (torch.exp(last_b.float()) * (last_seg == 0))[..., 0]
        # decay from the end of chunk c' to the start of chunk c (c = n: the end of the sequence)
        tb = F.pad(last_b[..., 0].cumsum(-1), (1, 0))                 # [B, H, n + 1], before chunk c
        ts = F.pad(last_seg[..., 0].cumsum(-1), (1, 0))
        before = torch.ones(n + 1, n, dtype=torch.bool, device=dev).tril(-1)
        ok = before & (ts[..., :, None] == ts[..., None, 1:])
        between = torch.where(ok, tb[..., :, None] - tb[..., None, 1:], torch.zeros((), dtype=torch.float64, device=dev))
        self.carry = torch.exp(between.float()) * ok                  # [B, H, n + 1, n]
        self.carry0 = torch.exp(tb.float()) * (ts == 0)               # [B, H, n + 1]
        self.k = self.tokens(s["k"])
        self.v = self.tokens(s["v"])
        self.q = self.tokens(q)
        self.w0 = s["w0"].float()[None].expand(B, H, d, d)
        u = (self.v * (self.e * self.to_end)[..., None]).transpose(-1, -2).contiguous() @ self.k
        w = self.carry @ u.reshape(B, H, n, d * d) + self.carry0[..., None] * self.w0.reshape(B, H, 1, d * d)
        w = w.reshape(B, H, n + 1, d, d)
        self.w, self.w_out = w[:, :, :n], w[:, :, n]                  # states at chunk starts, at the end

    def per_token(self, x):
        return F.pad(x, (0, self.pad)).reshape(self.B, self.H, self.n, _CHUNK)

    def tokens(self, x):
        x = torch.where(self.live[..., None], x.float(), torch.zeros((), device=x.device))
        return F.pad(x, (0, 0, 0, self.pad)).reshape(self.B, self.H, self.n, _CHUNK, self.d)

    def whole_sequence(self, x):
        return x.reshape(self.B, self.H, self.n * _CHUNK, *x.shape[4:])[:, :, :self.T]


def _t(x):
    return x.transpose(-1, -2).contiguous()


def _gl_fwd(s):
    c = _Chunks(s)
    p = (c.q @ _t(c.k)) * c.dec * c.e[..., None, :]
    z = p @ c.v + c.from_start[..., None] * (c.q @ _t(c.w))
    return {"z": c.whole_sequence(z).to(s["q"].dtype), "w_out": c.w_out}


def _gl_bwd(s):
    c = _Chunks(s)
    B, H, n, d = c.B, c.H, c.n, c.d
    dt = s["q"].dtype
    dz = c.tokens(s["dz"])
    # gradients of the states at every chunk's end
    h = _t(dz * c.from_start[..., None]) @ c.q
    dw_out = s["dw_out"].reshape(B, H, 1, d * d)
    h = h.reshape(B, H, n, d * d)
    gw = _t(c.carry[:, :, :n]) @ h + c.carry[:, :, n, :, None] * dw_out
    dw0 = (c.carry0[:, :, :n, None] * h).sum(2) + c.carry0[:, :, n, None] * dw_out[:, :, 0]
    gw = gw.reshape(B, H, n, d, d)
    p = (c.q @ _t(c.k)) * c.dec
    r = dz @ _t(c.v)
    rd = r * c.dec
    zi = c.from_start[..., None] * (c.q @ _t(c.w))
    dq = (rd * c.e[..., None, :]) @ c.k + c.from_start[..., None] * (dz @ c.w)
    dk = _t(rd) @ c.q + c.to_end[..., None] * (c.v @ gw)
    gk = c.to_end[..., None] * (c.k @ _t(gw))
    dv = _t(p) @ dz + gk
    out = {"dq": c.whole_sequence(dq).to(dt),
           "dk": c.whole_sequence(c.e[..., None] * dk).to(dt),
           "dv": c.whole_sequence(c.e[..., None] * dv).to(dt),
           "dw0": dw0.reshape(B, H, d, d)}
    if s["eta_tok"] is not None:
        out["deta_tok"] = c.whole_sequence(float(s["eta"]) * (c.v * dv).sum(-1))
    if s["log_gate"] is not None:
        # pairs (s, u), s < t <= u: within the chunk, from before it, to after it, and past it
        m = (p * r * c.e[..., None, :]).double().tril(-1)
        flip = lambda x: x.flip(-1).cumsum(-1).flip(-1)  # noqa: E731
        inside = flip(m.sum(-1) - m.sum(-2))
        into = flip((dz * zi).sum(-1).double())
        out_of = (c.e * (c.v * gk).sum(-1)).double()
        out_of = out_of.cumsum(-1) - out_of
        past = (c.whole.double() * (gw * c.w).sum((-1, -2)).double())[..., None]
        dg = c.whole_sequence((inside + into + out_of + past).float())
        out["dlog_gate"] = torch.where(c.reset | ~c.live, torch.zeros_like(dg), dg)
    return out


def _gl_step(s):
    q, k, v = s["q"].float(), s["k"].float(), s["v"].float()
    e = float(s["eta"]) * (s["eta_tok"] if s["eta_tok"] is not None else 1.0)
    w = s["w"] if s["log_gate"] is None else torch.exp(s["log_gate"])[..., None, None] * s["w"]
    ev = v * (e[..., None] if torch.is_tensor(e) else e)
    s["w"].copy_(w + ev[..., :, None] * k[..., None, :])
    return {"z": (s["w"] * q[..., None, :]).sum(-1).to(s["q"].dtype), "w": s["w"]}


# ---------------------------------------------------------------- the norm in plain torch

_EPS = 1e-5


def _act(name, g):
    """The gate's activation and its derivative."""
    if name == "none":
        return g, torch.ones_like(g)
    if name == "sigmoid":
        a = torch.sigmoid(g)
        return a, a * (1 - a)
    if name == "silu":
        a = torch.sigmoid(g)
        return g * a, a * (1 + g * (1 - a))
    cdf = 0.5 * (1 + torch.erf(g * 0.5 ** 0.5))
    return g * cdf, cdf + g * torch.exp(-0.5 * g * g) * (2 * math.pi) ** -0.5


def _normalised(x, kind):
    """norm(x) and 1 / its denominator, over the last axis."""
    if kind == "layer":
        x = x - x.mean(-1, keepdim=True)
    ss = (x * x).sum(-1, keepdim=True) if kind == "l2" else (x * x).mean(-1, keepdim=True)
    r = torch.rsqrt(ss + _EPS)
    return x * r, r


def _head(p):
    return p[None, :, None, :]


def _norm_fwd(s):
    c = s["case"]
    y, _ = _normalised(s["x"].float(), c["kind"])
    y = y * _head(s["weight"])
    if s["bias"] is not None:
        y = y + _head(s["bias"])
    if s["gate"] is not None:
        y = y * _act(c["act"], s["gate"].float())[0]
    if s["scale"] is not None:
        y = y * _head(s["scale"])
    if s["res"] is not None:
        y = y + s["res"].float()
    return {"y": y.to(s["x"].dtype)}


def _norm_bwd(s):
    c = s["case"]
    dt, kind = s["x"].dtype, c["kind"]
    xh, r = _normalised(s["x"].float(), kind)
    n = xh * _head(s["weight"])
    if s["bias"] is not None:
        n = n + _head(s["bias"])
    dy, out = s["dy"].float(), {}
    if s["gate"] is not None:
        a, da = _act(c["act"], s["gate"].float())
    else:
        a, da = torch.ones((), device=dy.device), None
    if s["scale"] is not None:
        out["dscale"] = (dy * a * n).sum((0, 2))
        dy = dy * _head(s["scale"])
    if s["gate"] is not None:
        out["dgate"] = (dy * n * da).to(dt)
        dy = dy * a
    out["dweight"] = (dy * xh).sum((0, 2))
    if s["bias"] is not None:
        out["dbias"] = dy.sum((0, 2))
    dxh = dy * _head(s["weight"])
    m2 = (dxh * xh).sum(-1, keepdim=True) / (1 if kind == "l2" else c["d"])
    dx = dxh - xh * m2
    if kind == "layer":
        dx = dx - dxh.mean(-1, keepdim=True)
    out["dx"] = (r * dx).to(dt)
    return out


_PLAIN = {"gl_fwd": _gl_fwd, "gl_bwd": _gl_bwd, "gl_step": _gl_step, "norm_fwd": _norm_fwd, "norm_bwd": _norm_bwd}


def _own_run(s):
    import test_sequence_layers_amd as ttt
    c = s["case"]
    if c["op"] == "gl_step":
        z = ttt.gated_linear_step(s["q"], s["k"], s["v"], s["w"], s["eta"], s["log_gate"], eta_tok=s["eta_tok"])
        return {"z": z, "w": s["w"]}
    if c["op"] == "gl_fwd":
        z, w_out = ttt.gated_linear_fwd(s["q"], s["k"], s["v"], s["w0"], s["eta"], s["log_gate"],
                                        eta_tok=s["eta_tok"], lengths=s["lengths"], return_state=True)
        return {"z": z, "w_out": w_out}
    if c["op"] == "gl_bwd":
        names = ["dq", "dk", "dv", "dw0"]
        names += ["dlog_gate"] if s["log_gate"] is not None else []
        names += ["deta_tok"] if s["eta_tok"] is not None else []
        return dict(zip(names, ttt.gated_linear_bwd(s["q"], s["k"], s["v"], s["w0"], s["eta"], s["log_gate"],
                                                    s["dz"], s["dw_out"], eta_tok=s["eta_tok"],
                                                    lengths=s["lengths"])))
    if c["op"] == "norm_fwd":
        return {"y": ttt.token_norm_fwd(s["x"], c["kind"], _EPS, weight=s["weight"], bias=s["bias"], gate=s["gate"],
                                        act=c["act"], scale=s["scale"], res=s["res"])}
    got = ttt.token_norm_bwd(s["x"], s["dy"], c["kind"], _EPS, weight=s["weight"], bias=s["bias"], gate=s["gate"],
                             act=c["act"], scale=s["scale"])
    names = ("dx", "dweight", "dbias", "dgate", "dscale")
    return {n: x for n, x in zip(names, got) if x is not None}


def run(state):
    if own:
        return _own_run(state)
    return _PLAIN[state["case"]["op"]](state)


def work(case):
    B, H, T, d = case["B"], case["H"], case["T"], case["d"]
    es = 2 if case["dtype"] == "bf16" else 4
    rows, state = B * H * T, B * H * d * d * 4
    tok = rows * d * es
    if case["op"].startswith("norm"):
        extra = case["after"]  # the gate and, forward, the residual or, backward, the gate's gradient
        tensors = (2 if case["op"] == "norm_fwd" else 3) + (2 if extra else 0)
        return {"bytes": tensors * tok + 4 * H * d * 4, "flops": rows * d * (12 if case["op"] == "norm_fwd" else 30)}
    per_token = 4 * rows * ((case["gate"] != "none") + case["rates"])
    if case["op"] == "gl_step":
        return {"bytes": 4 * tok + per_token + 2 * state, "flops": 5 * rows * d * d}
    if case["op"] == "gl_fwd":  # q, k, v, z; the shared initial state; the final states
        return {"bytes": 4 * tok + per_token + H * d * d * 4 + state, "flops": 4 * rows * d * d}
    # q, k, v, dz, dq, dk, dv; the gate and rates with their gradients; initial state, dw_out, dw0
    return {"bytes": 7 * tok + 2 * per_token + H * d * d * 4 + 2 * state, "flops": 10 * rows * d * d}


# ---------------------------------------------------------------- 64 bits, token by token

def _exact_linear(case, s):
    B, H, d = case["B"], case["H"], case["d"]
    step = case["op"] == "gl_step"
    up = lambda x: x.double() if x is not None else None  # noqa: E731
    q, k, v, g, r = (up(s[n]) for n in ("q", "k", "v", "log_gate", "eta_tok"))
    if step:
        q, k, v = (x[:, :, None] for x in (q, k, v))
        g = g[:, :, None] if g is not None else None
        r = r[:, :, None] if r is not None else None
    T = q.shape[2]
    a = torch.exp(g) if g is not None else torch.ones(B, H, T, dtype=torch.float64, device=q.device)
    eta = float(s["eta"])
    e = eta * r if r is not None else torch.full_like(a, eta)
    inside = torch.ones_like(a)
    if not step and s["lengths"] is not None:
        inside = (torch.arange(T, device=q.device)[None] < s["lengths"][:, None]).double()[:, None].expand(B, H, T)
    a, e = torch.where(inside > 0, a, torch.ones_like(a)), e * inside
    q, k, v = (x * inside[..., None] for x in (q, k, v))
    w = s["w"].double() if step else s["w0"].double().expand(B, H, d, d)
    states, z = [w], []
    for t in range(T):
        w = a[:, :, t, None, None] * w + (e[:, :, t, None] * v[:, :, t])[..., None] * k[:, :, t, None, :]
        z.append(torch.matmul(w, q[:, :, t, :, None])[..., 0])
        if case["op"] == "gl_bwd":
            states.append(w)
    if step:
        return {"z": z[0], "w": w}
    if case["op"] == "gl_fwd":
        return {"z": torch.stack(z, 2), "w_out": w}
    dz, gw = s["dz"].double() * inside[..., None], s["dw_out"].double()
    dq, dk, dv, dg, de = [], [], [], [], []
    for t in reversed(range(T)):
        gw = gw + dz[:, :, t, :, None] * q[:, :, t, None, :]
        dq.append(torch.matmul(dz[:, :, t, None, :], states[t + 1])[:, :, 0])
        gk = torch.matmul(gw, k[:, :, t, :, None])[..., 0]
        dv.append(e[:, :, t, None] * gk)
        dk.append(e[:, :, t, None] * torch.matmul(v[:, :, t, None, :], gw)[:, :, 0])
        de.append(eta * (v[:, :, t] * gk).sum(-1))
        dg.append(a[:, :, t] * (gw * states[t]).sum((-1, -2)) * inside[:, :, t])
        gw = a[:, :, t, None, None] * gw
    back = lambda x: torch.stack(x[::-1], 2)  # noqa: E731
    out = {"dq": back(dq), "dk": back(dk), "dv": back(dv), "dw0": gw}
    if r is not None:
        out["deta_tok"] = back(de)
    if g is not None:
        out["dlog_gate"] = back(dg)
    return out


def _exact_norm(case, s):
    names = ["x", "weight", "bias", "gate", "scale"]
    p = {n: s[n].double().requires_grad_(case["op"] == "norm_bwd") for n in names if s[n] is not None}
    x, per_head = p["x"], lambda t: t.reshape(1, case["H"], 1, case["d"])  # noqa: E731
    if case["kind"] == "layer":
        n = (x - x.mean(-1, keepdim=True)) / torch.sqrt(x.var(-1, keepdim=True, unbiased=False) + _EPS)
    elif case["kind"] == "rms":
        n = x / torch.sqrt(x.square().mean(-1, keepdim=True) + _EPS)
    else:
        n = x / torch.sqrt(x.square().sum(-1, keepdim=True) + _EPS)
    n = n * per_head(p["weight"])
    if "bias" in p:
        n = n + per_head(p["bias"])
    if "gate" in p:
        g = p["gate"]
        phi = (1 + torch.erf(g / math.sqrt(2.0))) / 2
        n = n * {"silu": g / (1 + torch.exp(-g)), "sigmoid": 1 / (1 + torch.exp(-g)), "gelu": g * phi, "none": g}[case["act"]]
    if "scale" in p:
        n = n * per_head(p["scale"])
    if case["op"] == "norm_fwd":
        return {"y": n + s["res"].double() if s["res"] is not None else n}
    grads = torch.autograd.grad(n, list(p.values()), s["dy"].double())
    return {"d" + name: grad for name, grad in zip(p, grads)}


def exact(case, seed):
    s = prepare(case, seed)
    return _exact_norm(case, s) if case["op"].startswith("norm") else _exact_linear(case, s)
