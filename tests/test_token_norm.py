"""The token norm with gate, scale and residual (token_norm_fwd, _bwd), alone and around the
gated linear recurrence.  The bounds are derived in gated_util.py."""
import pytest
import torch

import test_sequence_layers_amd as ttt
from tests.gated_util import assert_within, gated_inputs, norm_bounds, norm_reference

FAKE = 0x1000
INVALID, UNSUPPORTED = -1, -2


def _inputs(B, H, T, d, io, parts="wbgsr", seed=0, spread=1.0, shift=0.0):
    gen = torch.Generator().manual_seed(seed)
    dt = torch.bfloat16 if io == "bf16" else torch.float32
    normal = lambda *s: torch.randn(s, generator=gen)
    p = {"x": (spread * normal(B, H, T, d) + shift).to(dt), "weight": 1 + 0.3 * normal(H, d), "bias": 0.3 * normal(H, d),
         "gate": (2 * normal(B, H, T, d)).to(dt), "scale": normal(H, d), "res": normal(B, H, T, d).to(dt)}
    drop = {"weight": "w", "bias": "b", "gate": "g", "scale": "s", "res": "r"}
    return {n: t if n == "x" or drop[n] in parts else None for n, t in p.items()}, normal(B, H, T, d).to(dt)


def _gpu(p):
    return {n: t.cuda() if t is not None else None for n, t in p.items()}


def _fwd(p, kind, act, eps, **kw):
    return ttt.token_norm_fwd(p["x"], kind, eps, weight=p["weight"], bias=p["bias"], gate=p["gate"], act=act,
                              scale=p["scale"], res=p["res"], **kw)


def _bwd(p, dy, kind, act, eps, **kw):
    got = ttt.token_norm_bwd(p["x"], dy, kind, eps, weight=p["weight"], bias=p["bias"], gate=p["gate"], act=act,
                             scale=p["scale"], **kw)
    return {n: t for n, t in zip(("dx", "dweight", "dbias", "dgate", "dscale"), got) if t is not None}


def _check(p, dy, kind, act="silu", eps=1e-5):
    print({n: tuple(t.shape) for n, t in p.items() if t is not None}, p["x"].dtype, kind, act, flush=True)
    g = _gpu(p)
    ref = norm_reference(p, kind, act, eps)
    assert_within("y", _fwd(g, kind, act, eps), ref.detach(), norm_bounds(p, kind, act, eps, ref_y=ref.detach()))
    grads = norm_reference(p, kind, act, eps, dy)
    tol = norm_bounds(p, kind, act, eps, dy=dy, ref=grads)
    got = _bwd(g, dy.cuda(), kind, act, eps)
    assert set(got) == set(tol)
    for n, t in got.items():
        assert_within(n, t, grads[n], tol[n])


def test_reference_gradients_against_differences():
    p, dy = _inputs(1, 2, 3, 5, "f32", seed=1)
    p = {n: t.double() for n, t in p.items()}
    for kind in ("layer", "rms", "l2"):
        for act in ("none", "silu", "gelu", "sigmoid"):
            grads = norm_reference(p, kind, act, 1e-5, dy)
            for n in p:
                step = torch.randn(p[n].shape, dtype=torch.float64, generator=torch.Generator().manual_seed(2))
                f = lambda h: float((norm_reference({**p, n: p[n] + h * step}, kind, act, 1e-5) * dy.double()).sum())
                # central differences at h = 1e-5: 1e-10 of third derivatives below 1e4
                assert abs((f(1e-5) - f(-1e-5)) / 2e-5 - float((grads["d" + n] * step).sum())) < 1e-5, (kind, act, n)


def _call(lib, back, **kw):
    a = dict(x=FAKE, weight=FAKE, bias=FAKE, gate=FAKE, scale=FAKE, res=FAKE, y=FAKE, dy=FAKE, dx=FAKE, dweight=FAKE,
             dbias=FAKE, dgate=FAKE, dscale=FAKE, B=1, H=2, T=3, d=16, kind=1, act=1, eps=1e-5, io=1, ws=FAKE,
             ws_bytes=1 << 30)
    a.update(kw)
    tail = [a[n] for n in ("B", "H", "T", "d", "kind", "act", "eps", "io")]
    head = [a[n] for n in ("x", "weight", "bias", "gate", "scale")]
    if back:
        return lib.token_norm_bwd(*head, *(a[n] for n in ("dy", "dx", "dweight", "dbias", "dgate", "dscale")), *tail,
                                  a["ws"], a["ws_bytes"], None)
    return lib.token_norm_fwd(*head, a["res"], a["y"], *tail, None)


@pytest.mark.parametrize("back", [False, True])
@pytest.mark.parametrize("bad, want", [
    (dict(x=None), INVALID), (dict(y=None, dx=None), INVALID), (dict(B=0), INVALID), (dict(T=-1), INVALID),
    (dict(d=0), INVALID), (dict(kind=3), INVALID), (dict(kind=-1), INVALID), (dict(act=4), INVALID),
    (dict(eps=0.0), INVALID), (dict(eps=float("nan")), INVALID), (dict(eps=float("inf")), INVALID), (dict(io=5), INVALID),
    (dict(x=FAKE + 1), INVALID), (dict(weight=FAKE + 2), INVALID), (dict(d=16385), UNSUPPORTED),
    (dict(H=65536), UNSUPPORTED), (dict(B=1 << 16, T=1 << 15), UNSUPPORTED)])
def test_refusals(back, bad, want):
    assert _call(ttt.load_library(), back, **bad) == want
    assert ("token_norm_bwd" if back else "token_norm_fwd") in ttt.last_error()


@pytest.mark.parametrize("bad", [dict(dy=None), dict(weight=None), dict(bias=None), dict(gate=None), dict(scale=None),
                                 dict(ws=None), dict(ws_bytes=8), dict(ws=FAKE + 8)])
def test_refusals_of_the_backward_pass(bad):
    assert _call(ttt.load_library(), True, **bad) == INVALID
    assert "token_norm_bwd" in ttt.last_error()


@pytest.mark.gpu
@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("kind", ["layer", "rms", "l2"])
@pytest.mark.parametrize("d", [1, 7, 16, 24, 64, 65, 100, 128, 384, 768, 1000, 1030])
def test_widths(io, kind, d):
    _check(*_inputs(2, 3, 11, d, io, seed=d), kind)


@pytest.mark.gpu
@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("d", [2048, 2056, 4096, 4100, 5001, 8192, 8200, 16383, 16384])
def test_wide_rows(io, d):
    _check(*_inputs(1, 2, 5, d, io, seed=d), "layer")


@pytest.mark.gpu
@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("parts", ["wb", "wbg"])
@pytest.mark.parametrize("d", [5, 65, 768, 1032, 2052, 4100, 8200, 12288, 16384])
def test_several_rows_of_every_width(io, parts, d):
    """More rows than a workgroup holds at once, with and without a gate."""
    _check(*_inputs(2, 2, 33, d, io, parts, seed=d), "layer")


@pytest.mark.gpu
@pytest.mark.parametrize("parts", ["", "w", "wb", "g", "ws", "r", "wgsr", "wbgs"])
@pytest.mark.parametrize("act", ["none", "silu", "gelu", "sigmoid"])
def test_parts(parts, act):
    _check(*_inputs(2, 2, 37, 64, "bf16", parts, seed=3), "rms", act)


@pytest.mark.gpu
@pytest.mark.parametrize("BHT", [(1, 1, 1), (1, 12, 1), (300, 5, 1), (1, 1, 700), (3, 2, 2000), (1, 40, 130)])
@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_batches(BHT, io):
    _check(*_inputs(*BHT, 32, io, seed=4), "layer")


@pytest.mark.gpu
@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_more_rows_than_one_pass_of_the_grid(io):
    _check(*_inputs(2, 3, 40000, 16, io, "w", seed=5), "rms")


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["layer", "rms", "l2"])
def test_rows_without_spread(kind):
    """Rows of zeros and of one value, and a mean that is large next to the spread."""
    p, dy = _inputs(1, 2, 6, 64, "f32", "wbs", seed=6, spread=0.01, shift=3.0)
    p["x"][:, :, 0] = 0.0
    p["x"][:, :, 1] = 2.5
    _check(p, dy, kind, eps=1e-3)


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 65, 600])
def test_a_row_that_is_not_finite_stays_by_itself(d):
    p, dy = _inputs(1, 2, 40, d, "bf16", seed=12)
    g = _gpu(p)
    want, grads = _fwd(g, "layer", "silu", 1e-5), _bwd(g, dy.cuda(), "layer", "silu", 1e-5)
    bad = {**g, "x": g["x"].clone()}
    bad["x"][0, 1, 7, 3] = float("inf")
    keep = torch.ones(1, 2, 40, dtype=torch.bool, device="cuda")
    keep[0, 1, 7] = False
    y, got = _fwd(bad, "layer", "silu", 1e-5), _bwd(bad, dy.cuda(), "layer", "silu", 1e-5)
    assert not torch.isfinite(y[0, 1, 7].float()).all()
    for a, b in ((want, y), (grads["dx"], got["dx"]), (grads["dgate"], got["dgate"])):
        assert torch.equal(a[keep], b[keep])
    assert torch.equal(grads["dweight"][0], got["dweight"][0])  # the other head's sums


@pytest.mark.gpu
def test_more_than_2_to_32_elements():
    B, H, T, d = 1, 3, 90_000, 16_000
    gen = torch.Generator("cuda").manual_seed(13)
    x = torch.randn((B, H, T, d), generator=gen, device="cuda", dtype=torch.bfloat16)
    assert x.numel() > 1 << 32
    w = torch.randn((H, d), generator=gen, device="cuda")
    y = ttt.token_norm_fwd(x, "rms", 1e-5, weight=w)
    dx, dw, _, _, _ = ttt.token_norm_bwd(x, x, "rms", 1e-5, weight=w)
    tail = {"x": x[:, 2:, -4:].cpu(), "weight": w[2:].cpu()}
    ref = norm_reference(tail, "rms", "none", 1e-5)
    assert_within("y", y[:, 2:, -4:], ref, norm_bounds(tail, "rms", "none", 1e-5, ref_y=ref))
    grads = norm_reference(tail, "rms", "none", 1e-5, tail["x"])
    tol = norm_bounds(tail, "rms", "none", 1e-5, dy=tail["x"], ref=grads)
    assert_within("dx", dx[:, 2:, -4:], grads["dx"], tol["dx"])
    # sum over rows of x xh, with xh = x r: every term is positive, so 512 roundings bound the sum's error
    part = torch.zeros(H, d, dtype=torch.float64, device="cuda")
    for t in range(0, T, 5000):
        xs = x[0, :, t:t + 5000].double()
        part += (xs * xs * torch.rsqrt(xs.square().mean(-1, keepdim=True) + 1e-5)).sum(1)
    assert float(((dw.double() - part) / part).abs().max()) < 1000 * 2.0 ** -24


@pytest.mark.gpu
def test_no_tokens():
    p, dy = _inputs(2, 3, 0, 64, "bf16", seed=7)
    g = _gpu(p)
    assert _fwd(g, "rms", "silu", 1e-5).shape == (2, 3, 0, 64)
    got = _bwd(g, dy.cuda(), "rms", "silu", 1e-5)
    assert not got["dweight"].any() and not got["dscale"].any() and not got["dbias"].any()


@pytest.mark.gpu
@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_tensors_off_their_alignment(io):
    """Views that start one element into their storage take the element-wise path: same values."""
    p, dy = _inputs(2, 2, 9, 64, io, seed=8)
    g = _gpu(p)
    shift = lambda t: torch.cat([t.new_zeros(1), t.reshape(-1)])[1:].view(t.shape)
    moved = {n: shift(t) for n, t in g.items()}
    assert moved["x"].data_ptr() % 16
    ref = norm_reference(p, "layer", "gelu", 1e-5)
    assert_within("y", _fwd(moved, "layer", "gelu", 1e-5), ref.detach(), norm_bounds(p, "layer", "gelu", 1e-5, ref_y=ref.detach()))
    grads = norm_reference(p, "layer", "gelu", 1e-5, dy)
    tol = norm_bounds(p, "layer", "gelu", 1e-5, dy=dy, ref=grads)
    for n, t in _bwd(moved, shift(dy.cuda()), "layer", "gelu", 1e-5).items():
        assert_within(n, t, grads[n], tol[n])


@pytest.mark.gpu
def test_streams_repeats_and_replays():
    p, dy = _inputs(2, 3, 500, 64, "bf16", seed=9)
    g, dy = _gpu(p), dy.cuda()
    y, grads = _fwd(g, "rms", "silu", 1e-5), _bwd(g, dy, "rms", "silu", 1e-5)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = [(_fwd(g, "rms", "silu", 1e-5, stream=s), _bwd(g, dy, "rms", "silu", 1e-5, stream=s)) for s in (None, side)]
    torch.cuda.synchronize()
    for y2, g2 in got:
        assert torch.equal(y, y2) and all(torch.equal(grads[n], g2[n]) for n in grads)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y3, g3 = _fwd(g, "rms", "silu", 1e-5), _bwd(g, dy, "rms", "silu", 1e-5)
    for i in range(3):
        g["x"].mul_(0.5)
        graph.replay()
        torch.cuda.synchronize()
        y, grads = _fwd(g, "rms", "silu", 1e-5), _bwd(g, dy, "rms", "silu", 1e-5)
        torch.cuda.synchronize()
        assert torch.equal(y, y3) and all(torch.equal(grads[n], g3[n]) for n in grads)


@pytest.mark.gpu
def test_bindings_refuse():
    p, dy = _inputs(2, 2, 4, 32, "bf16", seed=10)
    g = _gpu(p)
    with pytest.raises(ValueError, match="kind"):
        ttt.token_norm_fwd(g["x"], "batch")
    with pytest.raises(ValueError, match="act"):
        ttt.token_norm_fwd(g["x"], "rms", act="relu")
    with pytest.raises(ValueError, match="weight"):
        ttt.token_norm_fwd(g["x"], "rms", weight=g["weight"][:1])
    with pytest.raises(ValueError, match="gate"):
        ttt.token_norm_fwd(g["x"], "rms", gate=g["gate"].float())
    with pytest.raises(ValueError, match="contiguous"):
        ttt.token_norm_fwd(g["x"].transpose(1, 2), "rms")
    with pytest.raises(ttt.TTTError, match="workspace"):
        ttt.token_norm_bwd(g["x"], dy.cuda(), "rms", weight=g["weight"], workspace=torch.empty(16, device="cuda"))


@pytest.mark.gpu
def test_layer_between_its_norms():
    """Unit keys, the gated recurrence, then norm, gate and residual: outputs and every gradient
    of the run against float64 autograd.  Each of the three operators rounds to float32 only, so
    the run is held to the operators' bounds in relative terms: three chains of under 1000
    roundings, on sums whose terms are at most 30 times the result's norm (1000 * 30 * 2^-24 = 2e-3)."""
    B, H, T, d = 2, 2, 90, 32
    x = gated_inputs(B, H, T, d, "f32", "soft", rates=True, seed=22)
    p, dy = _inputs(B, H, T, d, "f32", "wgsr", seed=11)
    raw = x["k"]
    leaves = {"q": x["q"], "k": raw, "v": x["v"], "w0": x["w0"], "log_gate": x["log_gate"], "eta_tok": x["eta_tok"],
              "weight": p["weight"], "gate": p["gate"], "scale": p["scale"]}
    t = {n: v.double().requires_grad_() for n, v in leaves.items()}
    k = t["k"] / torch.sqrt((t["k"] ** 2).sum(-1, keepdim=True) + 1e-6)
    w, z = t["w0"].expand(B, H, d, d), []
    for i in range(T):
        w = torch.exp(t["log_gate"][:, :, i, None, None]) * w + 0.5 * t["eta_tok"][:, :, i, None, None] * (
            t["v"][:, :, i, :, None] * k[:, :, i, None, :])
        z.append((w @ t["q"][:, :, i, :, None])[..., 0])
    z = torch.stack(z, 2)
    n = z / torch.sqrt((z ** 2).mean(-1, keepdim=True) + 1e-5) * t["weight"][None, :, None]
    out = p["res"].double() + t["scale"][None, :, None] * (t["gate"] * torch.sigmoid(t["gate"])) * n
    want = dict(zip(t, torch.autograd.grad(out, list(t.values()), dy.double())))

    g = {n: v.cuda() for n, v in leaves.items()}
    unit = ttt.token_norm_fwd(g["k"], "l2", 1e-6)
    zk = ttt.gated_linear_fwd(g["q"], unit, g["v"], g["w0"], 0.5, g["log_gate"], eta_tok=g["eta_tok"])
    after = dict(weight=g["weight"], gate=g["gate"], act="silu", scale=g["scale"])
    y = ttt.token_norm_fwd(zk, "rms", 1e-5, res=p["res"].cuda(), **after)
    dzk, dweight, _, dgate, dscale = ttt.token_norm_bwd(zk, dy.cuda(), "rms", 1e-5, **after)
    dq, dunit, dv, dw0, dlog_gate, deta = ttt.gated_linear_bwd(g["q"], unit, g["v"], g["w0"], 0.5, g["log_gate"], dzk,
                                                               eta_tok=g["eta_tok"])
    dk = ttt.token_norm_bwd(g["k"], dunit, "l2", 1e-6)[0]
    got = {"q": dq, "k": dk, "v": dv, "w0": dw0.sum(0), "log_gate": dlog_gate, "eta_tok": deta, "weight": dweight,
           "gate": dgate, "scale": dscale}
    rel = lambda a, b: float((a.cpu().double() - b).norm() / b.norm())
    assert rel(y, out.detach()) < 2e-3
    for name in want:
        assert rel(got[name], want[name]) < 2e-3, name
