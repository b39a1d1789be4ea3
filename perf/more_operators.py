"""Cases that time the operators of a dense block, and their plain forms.

  ffn_fwd   the gated feed-forward block: gate and up projections, activation,
            product and down projection
  ffn_bwd   its gradient: of the input and of both weights
  ln_fwd    layer norm
  ln_bwd    its gradient, with the reduction of the weight's and the bias's
  clip      the global norm of many gradients, and the gradients clipped to it

``run`` makes the framework's calls where ``own`` is true; otherwise it computes
the same operators from elementary torch operations in 32 bits, rounded once.
``exact`` is each operator's definition in 64 bits.
"""
import math

import torch

own = False

DEV = "cuda:0"
EPS = 1e-5
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def listed():
    return [
        # the smallest call: one token of the smoke test's layer, latency alone
        dict(name="ffn fwd tiny 1 row", op="ffn_fwd", rows=1, H=256, I=128, act="silu", dtype="bf16", save=False),
        # a decode step through the full-size layer's shared expert
        dict(name="ffn fwd 8 rows", op="ffn_fwd", rows=8, H=7168, I=2048, act="silu", dtype="bf16", save=False),
        # a ragged prefill chunk of a mid-size dense block with odd widths
        dict(name="ffn fwd 1021 rows fp16", op="ffn_fwd", rows=1021, H=2056, I=1032, act="gelu_tanh", dtype="fp16", save=False),
        # a training step of the full-size layer's shared expert, pre-activations kept
        dict(name="ffn fwd 16384 rows", op="ffn_fwd", rows=16384, H=7168, I=2048, act="silu", dtype="bf16", save=True),
        # a short ragged batch of a small block, activations computed again
        dict(name="ffn bwd 333 rows fp16", op="ffn_bwd", rows=333, H=1032, I=520, act="gelu", dtype="fp16", save=False),
        # the gradient of the full-size layer's shared expert over a macrobatch
        dict(name="ffn bwd 8192 rows", op="ffn_bwd", rows=8192, H=7168, I=2048, act="silu", dtype="bf16", save=True),
        # one token of a decode step
        dict(name="ln fwd 1 row", op="ln_fwd", rows=1, H=7168, x="bf16", y="bf16", bias=True),
        # the full-size layer's tokens
        dict(name="ln fwd 57344 rows", op="ln_fwd", rows=57344, H=7168, x="bf16", y="bf16", bias=True),
        # an odd number of rows of an odd width, fp32 residual stream whose own gradient is added
        dict(name="ln bwd 4095 rows fp32", op="ln_bwd", rows=4095, H=2049, x="fp32", y="bf16", bias=True, res=True),
        # a macrobatch of the full-size layer
        dict(name="ln bwd 16384 rows", op="ln_bwd", rows=16384, H=7168, x="bf16", y="bf16", bias=True, res=False),
        # the gradients of one tiny block
        dict(name="clip 5 tensors", op="clip", layers=1, H=256, I=128, E=8, mats="fp32", kind="l2", max_norm=0.5),
        # the fp32 gradients of 96 mid-size blocks, norms and routers among them
        dict(name="clip 480 tensors", op="clip", layers=96, H=2048, I=1024, E=64, mats="fp32", kind="l2", max_norm=1.0),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(("ffn_fwd", "ffn_fwd", "ffn_bwd", "ffn_bwd", "ln_fwd", "ln_bwd", "clip"))
    if op in ("ffn_fwd", "ffn_bwd"):
        H, I = 8 * _log(rng, 8, 1024), 8 * _log(rng, 8, 512)
        top = (16384 if op == "ffn_fwd" else 8192) * 7168 * 2048 // (H * I)
        return dict(op=op, rows=_log(rng, 1, min(16384, top)), H=H, I=I, act=rng.choice(("silu", "silu", "gelu", "gelu_tanh", "relu")),
                    dtype=rng.choice(("bf16", "bf16", "fp16")), save=rng.random() < 0.5)
    if op == "clip":
        H, I, E = 8 * _log(rng, 8, 512) + rng.choice((0, 0, 1)), 8 * _log(rng, 8, 256), rng.choice((8, 64))
        per = 3 * H * I + 2 * H + E * H
        return dict(op=op, layers=_log(rng, 1, min(100, max(1, 600_000_000 // per))), H=H, I=I, E=E, mats=rng.choice(("fp32", "bf16")),
                    kind=rng.choice(("l2", "l2", "max")), max_norm=rng.choice((0.01, 1.0, 1e6)))
    H = _log(rng, 32, 8192)
    if rng.random() < 0.5:
        H = -(-H // 8) * 8
    rows = _log(rng, 1, min(60000, (16384 if op == "ln_bwd" else 57344) * 7168 // (2 * H)))
    x, y = rng.choice((("bf16", "bf16"), ("bf16", "bf16"), ("fp16", "fp16"), ("fp32", "fp32"), ("fp32", "bf16")))
    c = dict(op=op, rows=rows, H=H, x=x, y=y, bias=rng.random() < 0.7)
    return c if op == "ln_fwd" else dict(c, res=rng.random() < 0.5)


# ---------------------------------------------------------------------------
# Inputs.
# ---------------------------------------------------------------------------

def _randn(g, shape, std, dtype=torch.bfloat16):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32).mul_(std).to(dtype)


def _prepare_ffn(c, g):
    n, H, I, t = c["rows"], c["H"], c["I"], TYPES[c["dtype"]]
    s = dict(c=c, X=_randn(g, (n, H), 1.0, t), W13=_randn(g, (2 * I, H), H ** -0.5 * 1.5, t), W2=_randn(g, (H, I), I ** -0.5, t))
    if c["op"] == "ffn_bwd":  # what a training step has kept of the forward, and what arrives
        s["HU"], s["A"] = _hidden(s)
        if not c["save"]:
            s["A"] = None
        s["dOut"] = _randn(g, (n, H), 0.02, t)
    return s


def _prepare_ln(c, g):
    n, H, tx, ty = c["rows"], c["H"], TYPES[c["x"]], TYPES[c["y"]]
    spread = 1.0 + 4.0 * (torch.rand(H, generator=g, device=DEV) < 0.02)  # a few channels are far larger, as in a residual stream
    s = dict(c=c, x=(torch.randn((n, H), generator=g, device=DEV) * spread + 0.3).to(tx), gain=1.0 + 0.2 * _randn(g, (H,), 1.0, torch.float32),
             bias=_randn(g, (H,), 0.1, torch.float32) if c["bias"] else None)
    if c["op"] == "ln_bwd":
        s["stats"] = _ln_fwd_plain(s)[1]  # the forward's, which a training step keeps
        s["dy"] = _randn(g, (n, H), 0.01, ty)
        s["dres"] = _randn(g, (n, H), 0.01, tx) if c["res"] else None
    return s


def _prepare_clip(c, g):
    # one flat buffer for the matrices and one for the fp32 vectors, as gradients lie for their reduction over
    # ranks; the tensors are views of them
    H, I, E, L = c["H"], c["I"], c["E"], c["layers"]
    mats, vecs = L * 3 * H * I, L * (2 * H + E * H)
    s = dict(c=c, flat=[_randn(g, (mats,), 0.002, TYPES[c["mats"]]), _randn(g, (vecs,), 0.01, torch.float32)])
    s["flat"][1][: L * H] *= 10  # the norms' gradients are larger than the others
    s["out"] = [torch.empty_like(t) for t in s["flat"]]
    sizes = ([2 * H * I, H * I] * L, [H, H, E * H] * L)
    s["grads"], s["clipped"] = ([v for t, n in zip(s[k], sizes) for v in t.split(n)] for k in ("flat", "out"))
    return s


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    make = {"ffn_fwd": _prepare_ffn, "ffn_bwd": _prepare_ffn, "ln_fwd": _prepare_ln, "ln_bwd": _prepare_ln, "clip": _prepare_clip}
    return make[case["op"]](dict(case), g)


# ---------------------------------------------------------------------------
# Plain forms.
# ---------------------------------------------------------------------------

def _act(kind, h):
    """The activation and its derivative."""
    if kind == "silu":
        s = 1 / (1 + torch.exp(-h))
        return h * s, s * (1 + h * (1 - s))
    if kind == "relu":
        on = (h > 0).to(h.dtype)
        return h * on, on
    if kind == "gelu":
        cdf = 0.5 * (1 + torch.erf(h * math.sqrt(0.5)))
        return h * cdf, cdf + h * torch.exp(-0.5 * h * h) * (1 / math.sqrt(2 * math.pi))
    k = math.sqrt(2 / math.pi)
    s = 1 / (1 + torch.exp(-2 * k * (h + 0.044715 * h * h * h)))  # 0.5 (1 + tanh(v)) = sigmoid(2 v)
    return h * s, s + h * s * (1 - s) * 2 * k * (1 + 3 * 0.044715 * h * h)


def _hidden(s):
    c, t = s["c"], TYPES[s["c"]["dtype"]]
    hu = torch.matmul(s["X"].float(), s["W13"].float().t())
    a = _act(c["act"], hu[:, : c["I"]])[0] * hu[:, c["I"]:]
    return hu.to(t), a.to(t)


def _ffn_fwd_plain(s):
    c, t = s["c"], TYPES[s["c"]["dtype"]]
    hu = torch.matmul(s["X"].float(), s["W13"].float().t())
    a = _act(c["act"], hu[:, : c["I"]])[0] * hu[:, c["I"]:]
    out = torch.matmul(a, s["W2"].float().t()).to(t)
    return (out, hu.to(t), a.to(t)) if c["save"] else out


def _ffn_bwd_plain(s):
    c, t = s["c"], TYPES[s["c"]["dtype"]]
    h, u, d = s["HU"][:, : c["I"]].float(), s["HU"][:, c["I"]:].float(), s["dOut"].float()
    v, dv = _act(c["act"], h)
    a = v * u if s["A"] is None else s["A"].float()
    dA = torch.matmul(d, s["W2"].float())
    dhu = torch.cat([dA * u * dv, dA * v], 1)
    dX = torch.matmul(dhu, s["W13"].float())
    return dX.to(t), torch.matmul(dhu.t(), s["X"].float()).to(t), torch.matmul(d.t(), a).to(t)


def _ln_fwd_plain(s):
    x = s["x"].float()
    mean = x.mean(1, keepdim=True)
    xc = x - mean
    rstd = torch.rsqrt(xc.square().mean(1, keepdim=True) + EPS)
    y = xc * rstd * s["gain"]
    if s["bias"] is not None:
        y = y + s["bias"]
    return y.to(TYPES[s["c"]["y"]]), torch.cat([mean, rstd], 1)


def _ln_bwd_plain(s):
    mean, rstd, dy = s["stats"][:, :1], s["stats"][:, 1:], s["dy"].float()
    xh = (s["x"].float() - mean) * rstd
    dg, db = (dy * xh).sum(0), dy.sum(0)
    t = dy * s["gain"]
    dx = rstd * (t - t.mean(1, keepdim=True) - xh * (t * xh).mean(1, keepdim=True))
    if s["dres"] is not None:
        dx = dx + s["dres"].float()
    return dx.to(s["x"].dtype), dg, db if s["bias"] is not None else None


def _clip_plain(s):
    c, (m, v) = s["c"], s["flat"]
    if c["kind"] == "l2":
        norm = torch.sqrt(torch.sum(m.float().square(), dtype=torch.float64) + torch.sum(v.square(), dtype=torch.float64))
    else:
        norm = torch.maximum(m.abs().max().double(), v.abs().max().double())
    coef = torch.clamp(c["max_norm"] / (norm + 1e-6), max=1.0).float()
    s["out"][0].copy_((m.float() * coef).to(m.dtype))
    s["out"][1].copy_(v * coef)
    return norm.float().reshape(1), s["out"][0], s["out"][1]


# ---------------------------------------------------------------------------
# The framework's calls.
# ---------------------------------------------------------------------------

def _ffn_own(s):
    from routing_schedule_expert_amd import ops

    c = s["c"]
    if "n" not in s:  # the descriptor, outputs and workspace, which a model keeps
        act = {"silu": ops.MOE_ACT_SILU, "gelu": ops.MOE_ACT_GELU, "gelu_tanh": ops.MOE_ACT_GELU_TANH, "relu": ops.MOE_ACT_RELU}[c["act"]]
        s["n"] = ops.make_ffn_desc(c["rows"], c["H"], c["I"], act=act, dtype=TYPES[c["dtype"]])
        s["bufs"] = (ops.alloc_gated_ffn(s["n"], DEV, save_hu=c["save"]) if c["op"] == "ffn_fwd" else
                     ops.alloc_gated_ffn_bwd(s["n"], DEV, dw_dtype=TYPES[c["dtype"]]))
    b = s["bufs"]
    if c["op"] == "ffn_fwd":
        ops.gated_ffn_fwd(s["n"], s["X"], s["W13"], s["W2"], b)
        return (b.out, b.HU, b.A) if c["save"] else b.out
    ops.gated_ffn_bwd(s["n"], s["dOut"], s["X"], s["HU"], s["A"], s["W13"], s["W2"], b)
    return b.dX, b.dW13, b.dW2


def _ln_own(s):
    from routing_schedule_expert_amd import ops

    c = s["c"]
    if "n" not in s:
        s["n"] = ops.make_layer_norm_desc(c["rows"], c["H"], x_dtype=TYPES[c["x"]], y_dtype=TYPES[c["y"]], eps=EPS)
        s["bufs"] = ops.alloc_layer_norm(s["n"], DEV) if c["op"] == "ln_fwd" else ops.alloc_layer_norm_bwd(s["n"], DEV, bias=c["bias"])
    b = s["bufs"]
    if c["op"] == "ln_fwd":
        ops.layer_norm_fwd(s["n"], s["x"], s["gain"], s["bias"], b)
        return b.y, b.stats
    ops.layer_norm_bwd(s["n"], s["x"], s["gain"], s["stats"], s["dy"], s["dres"], b)
    return b.dx, b.dg, b.db


def _clip_own(s):
    from routing_schedule_expert_amd import ops

    c = s["c"]
    if "list" not in s:  # the list of the gradients' buffers, which a training loop keeps
        s["list"] = ops.make_grad_list(s["grads"], s["clipped"])
    kind = ops.MOE_NORM_L2 if c["kind"] == "l2" else ops.MOE_NORM_MAX
    norm = ops.grad_clip(s["list"], c["max_norm"], kind=kind).norm
    return norm, s["out"][0], s["out"][1]


def run(state):
    op = state["c"]["op"]
    if own:
        return {"ffn_fwd": _ffn_own, "ffn_bwd": _ffn_own, "ln_fwd": _ln_own, "ln_bwd": _ln_own, "clip": _clip_own}[op](state)
    return {"ffn_fwd": _ffn_fwd_plain, "ffn_bwd": _ffn_bwd_plain, "ln_fwd": _ln_fwd_plain, "ln_bwd": _ln_bwd_plain, "clip": _clip_plain}[op](state)


# ---------------------------------------------------------------------------
# What a pass cannot do without.
# ---------------------------------------------------------------------------

def work(case):
    c = case
    size = {"bf16": 2, "fp16": 2, "fp32": 4}
    if c["op"] in ("ffn_fwd", "ffn_bwd"):
        n, H, I = c["rows"], c["H"], c["I"]
        if c["op"] == "ffn_fwd":
            return {"bytes": 2 * (3 * H * I + 2 * n * H + (3 * n * I if c["save"] else 0)), "flops": 6 * n * H * I}
        return {"bytes": 2 * (6 * H * I + 3 * n * H + (3 if c["save"] else 2) * n * I), "flops": 12 * n * H * I}
    if c["op"] == "clip":
        H, I, E, L = c["H"], c["I"], c["E"], c["layers"]
        n, v = L * 3 * H * I, L * (2 * H + E * H)
        return {"bytes": 2 * (n * size[c["mats"]] + 4 * v), "flops": 3 * (n + v)}
    n, H, x, y = c["rows"], c["H"], size[c["x"]], size[c["y"]]
    if c["op"] == "ln_fwd":
        return {"bytes": n * H * (x + y) + 8 * n + 4 * H * (1 + c["bias"]), "flops": 8 * n * H}
    return {"bytes": n * H * ((3 if c["res"] else 2) * x + y) + 8 * n + 4 * H * (2 + c["bias"]), "flops": 16 * n * H}


# ---------------------------------------------------------------------------
# The definitions in 64 bits.
# ---------------------------------------------------------------------------

def _slope64(kind, h):
    """act(h) / h, with h = 0 going by its limit, and act'(h)."""
    if kind == "silu":
        s = torch.sigmoid(h)
        return s, s + h * s * torch.sigmoid(-h)
    if kind == "relu":
        return torch.heaviside(h, torch.zeros((), dtype=h.dtype, device=h.device)), torch.heaviside(h, torch.zeros((), dtype=h.dtype, device=h.device))
    if kind == "gelu":
        s = torch.special.ndtr(h)
        return s, s + h * torch.exp(-h.square() / 2) / math.sqrt(2 * math.pi)
    v = math.sqrt(2 / math.pi) * (h + 0.044715 * h.pow(3))
    s = (1 + torch.tanh(v)) / 2
    return s, s + h / 2 / torch.cosh(v.clamp(-300, 300)).square() * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * h.square())


def _ffn_fwd_exact(s):
    c, w = s["c"], s["W13"].double()
    x, I = s["X"].double(), c["I"]
    h, u = x @ w[:I].t(), x @ w[I:].t()
    a = h * _slope64(c["act"], h)[0] * u
    out = a @ s["W2"].double().t()
    return (out, torch.cat([h, u], 1), a) if c["save"] else out


def _ffn_bwd_exact(s):
    c, I = s["c"], s["c"]["I"]
    hu = s["HU"].double()
    h, u = hu.split(I, 1)
    ratio, slope = _slope64(c["act"], h)
    g = s["dOut"].double()
    a = ratio * h * u if s["A"] is None else s["A"].double()
    up = g @ s["W2"].double()
    dh, du = up * u * slope, up * ratio * h
    w, x = s["W13"].double(), s["X"].double()
    return dh @ w[:I] + du @ w[I:], torch.cat([dh.t() @ x, du.t() @ x]), g.t() @ a


def _ln_rows(s, k):
    x = s["x"][k].double()
    mean = x.mean(1, keepdim=True)
    return x, mean, torch.sqrt(x.var(1, unbiased=False, keepdim=True) + EPS)


def _ln_fwd_exact(s):
    y, stats = [], []
    for i in range(0, s["c"]["rows"], 8192):
        x, mean, std = _ln_rows(s, slice(i, i + 8192))
        v = (x - mean) / std * s["gain"].double()
        y.append(v if s["bias"] is None else v + s["bias"].double())
        stats.append(torch.cat([mean, 1 / std], 1))
    return torch.cat(y), torch.cat(stats)


def _ln_bwd_exact(s):
    c, dx = s["c"], []
    dg, db = (torch.zeros(c["H"], dtype=torch.float64, device=DEV) for _ in range(2))
    for i in range(0, c["rows"], 8192):
        k = slice(i, i + 8192)
        x, mean, std = _ln_rows(s, k)
        xh, dy = (x - mean) / std, s["dy"][k].double()
        dg += torch.sum(dy * xh, 0)
        db += torch.sum(dy, 0)
        t = dy * s["gain"].double()
        t = t - t.mean(1, keepdim=True)
        v = (t - xh * torch.mean(t * xh, 1, keepdim=True)) / std
        dx.append(v if s["dres"] is None else v + s["dres"][k].double())
    return torch.cat(dx), dg, db if c["bias"] else None


def _clip_exact(s):
    c = s["c"]
    if c["kind"] == "l2":
        norm = math.sqrt(sum(float(p.double().square().sum()) for t in s["flat"] for p in t.split(1 << 26)))
    else:
        norm = max(float(t.abs().max()) for t in s["flat"])
    coef = min(1.0, c["max_norm"] / (norm + 1e-6))
    return torch.tensor([norm], dtype=torch.float64), s["flat"][0].double() * coef, s["flat"][1].double() * coef


def exact(case, seed):
    fn = {"ffn_fwd": _ffn_fwd_exact, "ffn_bwd": _ffn_bwd_exact, "ln_fwd": _ln_fwd_exact, "ln_bwd": _ln_bwd_exact, "clip": _clip_exact}
    return fn[case["op"]](prepare(case, seed))
