"""Cases that time the operators around the expert layer, and their plain forms.

  few       the whole MoE layer for a few tokens (bf16 or MXFP8 routed experts,
            optionally with the bf16 shared expert)
  norm_fwd  post-norm, gate, residual scale and next pre-norm in one pass
  norm_bwd  the gradient of norm_fwd
  ckpt      a layer's pre-activations packed to 8 bits and the SwiGLU backward
            that reads them

``run`` makes the framework's calls where ``own`` is true; otherwise it computes
the same operators from elementary torch operations in 32 bits, rounded once.
``exact`` is each operator's definition in 64 bits.
"""
import torch

own = False

DEV = "cuda:0"
EPS = 1e-6
BLOCK = 128  # elements that share one scale of a checkpoint


def listed():
    return [
        # the smallest call: one token of the smoke test's layer, latency alone
        dict(name="few tiny 1 token", op="few", mx=False, P=1, Np=1, K=2, E=8, L=8, base=0, H=256, I=128, Is=0, drop=False),
        # a decode step of the full-size share: one token from each of 8 partitions, about 8 of 48 experts hit
        dict(name="few share 8 tokens", op="few", mx=False, P=8, Np=1, K=8, E=384, L=48, base=48, H=7168, I=2048, Is=0, drop=False),
        # a ragged decode batch of the mid-size layer, every expert local, dropped ids, with a shared expert
        dict(name="few mid 37 tokens shared", op="few", mx=False, P=1, Np=37, K=6, E=64, L=64, base=0, H=2048, I=1024, Is=1024, drop=True),
        # the full-size share with MXFP8 weights, 32 tokens
        dict(name="few share 32 tokens mx", op="few", mx=True, P=8, Np=4, K=8, E=384, L=48, base=0, H=7168, I=2048, Is=0, drop=False),
        # the largest batch of the full-size share, with its shared expert: nearly every expert is hit
        dict(name="few share 128 tokens shared", op="few", mx=False, P=8, Np=16, K=8, E=384, L=48, base=336, H=7168, I=2048, Is=2048, drop=False),
        # one token of a decode step
        dict(name="norm fwd 1 row", op="norm_fwd", rows=1, H=7168, gate="token", res="bf16", post=True, pre=True, alpha=1.0, beta=1.0),
        # the full-size layer's tokens, a gate for each channel
        dict(name="norm fwd 57344 rows", op="norm_fwd", rows=57344, H=7168, gate="elem", res="bf16", post=True, pre=True, alpha=1.0, beta=0.5),
        # an odd number of rows of the mid-size layer, fp32 residual stream, a gate for each token
        dict(name="norm bwd 4095 rows fp32", op="norm_bwd", rows=4095, H=2056, gate="token", res="fp32", post=True, pre=True, alpha=0.9, beta=0.7),
        # a macrobatch of the full-size layer, a gate for each channel
        dict(name="norm bwd 16384 rows", op="norm_bwd", rows=16384, H=7168, gate="elem", res="bf16", post=True, pre=True, alpha=1.0, beta=1.0),
        # the tiny layer's rows
        dict(name="ckpt 301 rows", op="ckpt", n=301, cap=2304, I=128, scaled=True),
        # the mid-size layer's rows in buffers of their worst case
        dict(name="ckpt 26112 rows", op="ckpt", n=26112, cap=40000, I=1024, scaled=True),
        # the full-size share's rows under balanced routing, padding included
        dict(name="ckpt 61440 rows", op="ckpt", n=61440, cap=70000, I=2048, scaled=True),
    ]


def _log(rng, lo, hi):
    import math

    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(("few", "few", "norm_fwd", "norm_bwd", "ckpt"))
    if op == "few":
        tokens = _log(rng, 1, 128)
        P = 8 if tokens % 8 == 0 else 1
        L = _log(rng, 1, 48)
        E = L * rng.choice((1, 2, 8))
        return dict(op=op, mx=rng.random() < 0.4, P=P, Np=tokens // P, K=min(E, rng.choice((1, 2, 4, 6, 8))), E=E, L=L,
                    base=rng.randrange(E - L + 1), H=256 * _log(rng, 1, 28), I=128 * _log(rng, 1, 16),
                    Is=rng.choice((0, 0, 128 * _log(rng, 1, 16))), drop=rng.random() < 0.25)
    if op == "ckpt":
        n, I = _log(rng, 1, 57000), 128 * _log(rng, 1, 16)
        return dict(op=op, n=n, cap=n + rng.randrange(0, 2000), I=I, scaled=rng.random() < 0.7)
    H = 8 * _log(rng, 8, 1024)
    rows = _log(rng, 1, min(50000, (16000 if op == "norm_bwd" else 50000) * 7168 // H))
    return dict(op=op, rows=rows, H=H, gate=rng.choice(("none", "token", "elem")), res=rng.choice(("bf16", "fp32")),
                post=rng.random() < 0.7, pre=rng.random() < 0.8, alpha=rng.choice((1.0, 0.8)), beta=rng.choice((1.0, 0.25)))


# ---------------------------------------------------------------------------
# Inputs.
# ---------------------------------------------------------------------------

def _randn(g, shape, std, dtype=torch.bfloat16):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32).mul_(std).to(dtype)


def _mx_codes(wt):
    """E4M3 codes and one power-of-two scale byte for 32 elements of a row."""
    x = wt.float().unflatten(-1, (-1, 32))
    amax = x.abs().amax(-1, keepdim=True)
    e = torch.where(amax > 0, torch.floor(torch.log2(amax)) - 8, torch.full_like(amax, -127.0))
    q = torch.ldexp(x, -e).clamp_(-448, 448).to(torch.float8_e4m3fn)
    return q.flatten(-2).view(torch.uint8), (e + 127).to(torch.uint8).squeeze(-1)


def _prepare_few(c, g):
    T, E, K, L, H, I, Is = c["P"] * c["Np"], c["E"], c["K"], c["L"], c["H"], c["I"], c["Is"]
    ids = torch.rand((T, E), generator=g, device=DEV).argsort(dim=1)[:, :K].to(torch.int32)
    if c["drop"]:
        ids = torch.where(torch.rand((T, K), generator=g, device=DEV) < 0.05, torch.full_like(ids, -1), ids)
    z = torch.randn((T, K), generator=g, device=DEV).sort(dim=1, descending=True).values
    shape = (c["P"], c["Np"])
    s = dict(c=c, routes=ids.reshape(shape + (K,)).contiguous(), w=torch.softmax(z, 1).reshape(shape + (K,)).contiguous(),
             X=_randn(g, shape + (H,), 1.0))
    w13, w2 = [], []
    for _ in range(L):  # an expert at a time: the 32-bit draws stay small
        a, b = _randn(g, (2 * I, H), H ** -0.5 * 1.5), _randn(g, (H, I), I ** -0.5)
        w13.append(_mx_codes(a) if c["mx"] else a)
        w2.append(_mx_codes(b) if c["mx"] else b)
    if c["mx"]:
        s["W13"], s["W13s"] = (torch.stack(x) for x in zip(*w13))
        s["W2"], s["W2s"] = (torch.stack(x) for x in zip(*w2))
    else:
        s["W13"], s["W2"] = torch.stack(w13), torch.stack(w2)
    s["S13"], s["S2"] = (_randn(g, (2 * Is, H), H ** -0.5 * 1.5), _randn(g, (H, Is), Is ** -0.5)) if Is else (None, None)
    return s


def _prepare_norm(c, g):
    n, H = c["rows"], c["H"]
    res = torch.float32 if c["res"] == "fp32" else torch.bfloat16
    spread = 1.0 + 4.0 * (torch.rand(H, generator=g, device=DEV) < 0.02)  # a few channels are far larger, as in a residual stream
    s = dict(c=c, y=_randn(g, (n, H), 0.3), r=(torch.randn((n, H), generator=g, device=DEV) * spread).to(res),
             z=None if c["gate"] == "none" else _randn(g, (n,), 1.0, torch.float32) if c["gate"] == "token" else _randn(g, (n, H), 1.0),
             g_post=1.0 + 0.2 * _randn(g, (H,), 1.0, torch.float32) if c["post"] else None,
             g_pre=1.0 + 0.2 * _randn(g, (H,), 1.0, torch.float32) if c["pre"] else None,
             r_out=torch.empty((n, H), dtype=res, device=DEV),
             xn=torch.empty((n, H), dtype=torch.bfloat16, device=DEV) if c["pre"] else None)
    s["stats"] = torch.empty((n, 2), dtype=torch.float32, device=DEV)
    if c["op"] == "norm_bwd":
        del s["r_out"], s["xn"]
        _, _, s["stats"] = _norm_fwd_plain(s)  # the forward's, which a training step keeps
        s["dr_out"] = _randn(g, (n, H), 0.01, res)
        s["dxn"] = _randn(g, (n, H), 0.01) if c["pre"] else None
    return s


def _prepare_ckpt(c, g):
    n, cap, I = c["n"], c["cap"], c["I"]
    hu = torch.zeros((cap, 2 * I), dtype=torch.bfloat16, device=DEV)
    hu[:n] = _randn(g, (n, 2 * I), 1.5)
    hu[:n][torch.rand(n, generator=g, device=DEV) < 0.05] = 0  # padding rows of the expert segments
    z = torch.rand(cap, generator=g, device=DEV)
    return dict(c=c, HU=hu, dA=_randn(g, (cap, I), 0.02), wrow=z if c["scaled"] else None,
                nrows=torch.tensor([n], dtype=torch.int32, device=DEV),
                q=torch.zeros((cap, 2 * I), dtype=torch.int8, device=DEV),
                scales=torch.zeros((cap, 2 * I // BLOCK), dtype=torch.float32, device=DEV),
                dHU=torch.zeros((cap, 2 * I), dtype=torch.bfloat16, device=DEV),
                A=torch.zeros((cap, I), dtype=torch.bfloat16, device=DEV), dw=torch.zeros(cap, device=DEV))


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    make = {"few": _prepare_few, "norm_fwd": _prepare_norm, "norm_bwd": _prepare_norm, "ckpt": _prepare_ckpt}
    return make[case["op"]](dict(case), g)


# ---------------------------------------------------------------------------
# Plain forms.
# ---------------------------------------------------------------------------

def _values(codes, scales, dtype):
    """What MX codes and their scale bytes stand for."""
    v = codes.view(torch.float8_e4m3fn).to(dtype).unflatten(-1, (-1, 32))
    return torch.ldexp(v, scales.to(dtype).unsqueeze(-1) - 127).flatten(-2)


def _few_plain(s):
    c = s["c"]
    T, K, L, H, I = c["P"] * c["Np"], c["K"], c["L"], c["H"], c["I"]
    x = s["X"].reshape(T, H).float()
    lid = s["routes"].reshape(T, K).long() - c["base"]
    local = (lid >= 0) & (lid < L) & (s["routes"].reshape(T, K) >= 0)
    hit = torch.unique(lid[local])
    n = hit.numel()
    if c["mx"]:
        w13, w2 = _values(s["W13"][hit], s["W13s"][hit], torch.float32), _values(s["W2"][hit], s["W2s"][hit], torch.float32)
    else:
        w13, w2 = s["W13"][hit].float(), s["W2"][hit].float()
    hu = torch.matmul(x, w13.reshape(n * 2 * I, H).t()).reshape(T, n, 2 * I)
    a = hu[..., :I] / (1 + torch.exp(-hu[..., :I])) * hu[..., I:]
    weight = (s["w"].reshape(T, K, 1) * ((lid.unsqueeze(-1) == hit) & local.unsqueeze(-1))).sum(1)  # [T][n]
    a = (a * weight.unsqueeze(-1)).permute(1, 2, 0).contiguous()  # [n][I][T]
    out = torch.bmm(w2, a).sum(0).t()
    if c["Is"]:
        hs = torch.matmul(x, s["S13"].float().t())
        out = out + torch.matmul(hs[:, :c["Is"]] / (1 + torch.exp(-hs[:, :c["Is"]])) * hs[:, c["Is"]:], s["S2"].float().t())
    return out.to(torch.bfloat16).reshape(c["P"], c["Np"], H).contiguous()


def _gate(s):
    if s["z"] is None:
        return None
    v = 1 / (1 + torch.exp(-s["z"].float()))
    return v.unsqueeze(1) if s["c"]["gate"] == "token" else v


def _norm_fwd_plain(s):
    c = s["c"]
    p, stats = s["y"].float(), torch.zeros((c["rows"], 2), device=DEV)
    if c["post"]:
        stats[:, 0] = torch.rsqrt(p.square().mean(1) + EPS)
        p = p * stats[:, :1] * s["g_post"]
    v = _gate(s)
    r = c["alpha"] * s["r"].float() + c["beta"] * (p if v is None else v * p)
    xn = None
    if c["pre"]:
        stats[:, 1] = torch.rsqrt(r.square().mean(1) + EPS)
        xn = (r * stats[:, 1:] * s["g_pre"]).to(torch.bfloat16)
    return r.to(s["r"].dtype), xn, stats


def _norm_bwd_plain(s):
    c = s["c"]
    v, y = _gate(s), s["y"].float()
    ys, rs = s["stats"][:, :1], s["stats"][:, 1:]
    yh = y * ys if c["post"] else y
    p = yh * s["g_post"] if c["post"] else y
    grad, dg_pre = s["dr_out"].float(), None
    if c["pre"]:
        r = c["alpha"] * s["r"].float() + c["beta"] * (p if v is None else v * p)
        dx, xh = s["dxn"].float(), r * rs
        dg_pre = (dx * xh).sum(0)
        dx = dx * s["g_pre"]
        grad = grad + rs * (dx - xh * (dx * xh).mean(1, keepdim=True))
    dr = (c["alpha"] * grad).to(s["r"].dtype)
    dz = None
    if v is not None:
        dz = c["beta"] * p * grad * v * (1 - v)
        dz = dz.sum(1) if c["gate"] == "token" else dz.to(torch.bfloat16)
    dp = c["beta"] * grad if v is None else c["beta"] * grad * v
    dg_post = None
    if c["post"]:
        dg_post = (dp * yh).sum(0)
        dp = dp * s["g_post"]
        dp = ys * (dp - yh * (dp * yh).mean(1, keepdim=True))
    return dp.to(torch.bfloat16), dr, dz, dg_post, dg_pre


def _pack_plain(hu):
    x = hu.float().unflatten(-1, (-1, BLOCK))
    amax = x.abs().amax(-1, keepdim=True)
    q = torch.where(amax > 0, torch.round(x * (127.0 / amax)), torch.zeros_like(x)).to(torch.int8)
    return q.flatten(-2), (amax / 127.0).squeeze(-1)


def _ckpt_plain(s):
    c = s["c"]
    n, I = c["n"], c["I"]
    s["q"][:n], s["scales"][:n] = _pack_plain(s["HU"][:n])
    hu = (s["q"][:n].float().unflatten(-1, (-1, BLOCK)) * s["scales"][:n].unsqueeze(-1)).flatten(-2)
    h, u, dA = hu[:, :I], hu[:, I:], s["dA"][:n].float()
    sg = 1 / (1 + torch.exp(-h))
    a = h * sg * u
    s["A"][:n], s["dw"][:n] = a.to(torch.bfloat16), (dA * a).sum(1)
    if s["wrow"] is not None:
        dA = dA * s["wrow"][:n].unsqueeze(1)
    s["dHU"][:n, :I] = (dA * u * sg * (1 + h * (1 - sg))).to(torch.bfloat16)
    s["dHU"][:n, I:] = (dA * h * sg).to(torch.bfloat16)
    return s["dHU"], s["A"], s["dw"]


# ---------------------------------------------------------------------------
# The framework's calls.
# ---------------------------------------------------------------------------

def _few_own(s):
    from routing_schedule_expert_amd import ops

    c = s["c"]
    if "bufs" not in s:  # the output and the workspace, which a decode loop keeps
        s["d"] = ops.make_desc(c["P"], c["Np"], c["K"], c["E"], c["L"], expert_base=c["base"], H=c["H"], I=c["I"])
        s["bufs"] = ops.alloc_few(s["d"], DEV, c["Is"])
    if c["mx"]:
        ops.layer_fwd_few_mx(s["d"], s["routes"], s["w"], s["X"], s["W13"], s["W13s"], s["W2"], s["W2s"], s["bufs"], s["S13"], s["S2"])
    else:
        ops.layer_fwd_few(s["d"], s["routes"], s["w"], s["X"], s["W13"], s["W2"], s["bufs"], s["S13"], s["S2"])
    return s["bufs"].out


def _norm_desc(s):
    from routing_schedule_expert_amd import ops

    c = s["c"]
    if "n" not in s:
        gate = {"none": ops.MOE_GATE_NONE, "token": ops.MOE_GATE_TOKEN, "elem": ops.MOE_GATE_ELEM}[c["gate"]]
        s["n"] = ops.make_norm_desc(c["rows"], c["H"], gate=gate, res_fp32=c["res"] == "fp32", alpha=c["alpha"], beta=c["beta"], eps=EPS)
    return s["n"]


def _norm_fwd_own(s):
    from routing_schedule_expert_amd import ops

    ops.moe_block_norm_fwd(_norm_desc(s), s["y"], s["r"], s["z"], s["g_post"], s["g_pre"], s["r_out"], s["xn"], s["stats"])
    return s["r_out"], s["xn"], s["stats"]


def _norm_bwd_own(s):
    from routing_schedule_expert_amd import ops

    n = _norm_desc(s)
    if "grads" not in s:
        s["grads"] = ops.alloc_norm_bwd(n, DEV, post=s["c"]["post"], pre=s["c"]["pre"])
    b = s["grads"]
    ops.block_norm_bwd(n, s["y"], s["r"], s["z"], s["g_post"], s["g_pre"], s["stats"], s["dr_out"], s["dxn"], b)
    return b.dy, b.dr, b.dz, b.dg_post, b.dg_pre


def _ckpt_own(s):
    from routing_schedule_expert_amd import ops

    ops.moe_ckpt_pack(s["HU"], s["q"], s["scales"], s["nrows"])
    ops.moe_ckpt_swiglu_bwd(s["q"], s["scales"], s["dA"], s["wrow"], s["dHU"], s["A"], s["dw"], s["nrows"])
    return s["dHU"], s["A"], s["dw"]


def run(state):
    op = state["c"]["op"]
    if own:
        return {"few": _few_own, "norm_fwd": _norm_fwd_own, "norm_bwd": _norm_bwd_own, "ckpt": _ckpt_own}[op](state)
    return {"few": _few_plain, "norm_fwd": _norm_fwd_plain, "norm_bwd": _norm_bwd_plain, "ckpt": _ckpt_plain}[op](state)


# ---------------------------------------------------------------------------
# What a pass cannot do without.
# ---------------------------------------------------------------------------

def work(case):
    c = case
    if c["op"] == "few":
        T, K, E, L, H, I, Is = c["P"] * c["Np"], c["K"], c["E"], c["L"], c["H"], c["I"], c["Is"]
        keep = 0.95 if c["drop"] else 1.0
        hit = L * (1 - (1 - keep * K / E) ** T)  # the experts that uniform routes are expected to hit
        routes = T * K * keep * L / E
        per = 3 * H * I * (33 / 32 if c["mx"] else 2)
        return {"bytes": hit * per + 6 * H * Is + 4 * T * H + 8 * T * K, "flops": 6 * H * (I * routes + Is * T)}
    if c["op"] == "ckpt":
        n, I = c["n"], c["I"]
        code = 2 * I * (1 + 4 / BLOCK)
        return {"bytes": n * (4 * I + 2 * code + 2 * I + 4 * I + 2 * I + 8), "flops": n * I * 30}
    n, H, res = c["rows"], c["H"], 4 if c["res"] == "fp32" else 2
    z = {"none": 0, "token": 4 * n, "elem": 2 * n * H}[c["gate"]]
    if c["op"] == "norm_fwd":
        return {"bytes": n * H * (2 + 2 * res + 2 * c["pre"]) + z + 8 * n + 8 * H, "flops": 10 * n * H}
    return {"bytes": n * H * (4 + 3 * res + 2 * c["pre"]) + 2 * z + 8 * n + 16 * H, "flops": 25 * n * H}


# ---------------------------------------------------------------------------
# The definitions in 64 bits.
# ---------------------------------------------------------------------------

def _few_exact(s):
    c = s["c"]
    T, K, H, I = c["P"] * c["Np"], c["K"], c["H"], c["I"]
    x, ids, w = s["X"].reshape(T, H).double(), s["routes"].reshape(T, K).tolist(), s["w"].reshape(T, K).double()
    out = torch.zeros((T, H), dtype=torch.float64, device=DEV)

    def expert(rows, w13, w2, inner):
        g, u = rows @ w13[:inner].t(), rows @ w13[inner:].t()
        return (g * torch.sigmoid(g) * u) @ w2.t()

    for e in range(c["L"]):
        at = [(t, j) for t in range(T) for j in range(K) if ids[t][j] == e + c["base"]]
        if not at:
            continue
        t, j = (torch.tensor(v, device=DEV) for v in zip(*at))
        if c["mx"]:
            w13, w2 = _values(s["W13"][e], s["W13s"][e], torch.float64), _values(s["W2"][e], s["W2s"][e], torch.float64)
        else:
            w13, w2 = s["W13"][e].double(), s["W2"][e].double()
        out.index_add_(0, t, w[t, j].unsqueeze(1) * expert(x[t], w13, w2, I))
    if c["Is"]:
        out += expert(x, s["S13"].double(), s["S2"].double(), c["Is"])
    return out.reshape(c["P"], c["Np"], H)


def _norm_exact_rows(s, k):
    """norm_fwd's r', xn and what norm_bwd needs of it, for the rows of the slice k."""
    c = s["c"]
    y, r = s["y"][k].double(), s["r"][k].double()
    ystd = torch.sqrt(torch.mean(y * y, 1, keepdim=True) + EPS) if c["post"] else None
    p = y / ystd * s["g_post"].double() if c["post"] else y
    v = torch.ones_like(y)
    if c["gate"] != "none":
        v = torch.sigmoid(s["z"][k].double()).reshape(y.shape[0], -1).expand_as(y)
    new = c["alpha"] * r + c["beta"] * v * p
    rstd = torch.sqrt(torch.mean(new * new, 1, keepdim=True) + EPS)
    return y, ystd, p, v, new, rstd


def _norm_fwd_exact(s):
    c, r_out, xn = s["c"], [], []
    stats = torch.zeros((c["rows"], 2), dtype=torch.float64, device=DEV)
    for i in range(0, c["rows"], 4096):
        _, ystd, _, _, new, rstd = _norm_exact_rows(s, slice(i, i + 4096))
        r_out.append(new)
        if c["post"]:
            stats[i:i + 4096, :1] = 1 / ystd
        if c["pre"]:
            stats[i:i + 4096, 1:] = 1 / rstd
            xn.append(new / rstd * s["g_pre"].double())
    return torch.cat(r_out), torch.cat(xn) if c["pre"] else None, stats


def _norm_bwd_exact(s):
    c, dy, dr, dz = s["c"], [], [], []
    H = c["H"]
    dg_post, dg_pre = (torch.zeros(H, dtype=torch.float64, device=DEV) for _ in range(2))
    for i in range(0, c["rows"], 4096):
        k = slice(i, i + 4096)
        y, ystd, p, v, new, rstd = _norm_exact_rows(s, k)
        up = s["dr_out"][k].double()
        if c["pre"]:
            dx = s["dxn"][k].double()
            dg_pre += torch.sum(dx * new / rstd, 0)
            t = dx * s["g_pre"].double()
            up = up + t / rstd - new * torch.sum(t * new, 1, keepdim=True) / (H * rstd ** 3)
        dr.append(c["alpha"] * up)
        t = c["beta"] * up * p * v * (1 - v)
        dz.append(t.sum(1) if c["gate"] == "token" else t)
        t = c["beta"] * up * v
        if c["post"]:
            dg_post += torch.sum(t * y / ystd, 0)
            t = t * s["g_post"].double()
            t = t / ystd - y * torch.sum(t * y, 1, keepdim=True) / (H * ystd ** 3)
        dy.append(t)
    return (torch.cat(dy), torch.cat(dr), torch.cat(dz) if c["gate"] != "none" else None, dg_post if c["post"] else None,
            dg_pre if c["pre"] else None)


def _ckpt_exact(s):
    # the codes and scales are 32-bit operations by the format's definition; the rest is in 64 bits
    c = s["c"]
    I, cap = c["I"], c["cap"]
    dhu, a_out = (torch.zeros((cap, m * I), dtype=torch.float64, device=DEV) for m in (2, 1))
    dw = torch.zeros(cap, dtype=torch.float64, device=DEV)
    for i in range(0, c["n"], 8192):
        k = slice(i, min(c["n"], i + 8192))
        x = s["HU"][k].float().reshape(-1, 2 * I // BLOCK, BLOCK)
        top = x.abs().max(dim=-1, keepdim=True).values
        inv = 127.0 / torch.where(top > 0, top, torch.ones_like(top))
        v = (torch.round(x * inv).double() * (top / 127.0).double()).reshape(-1, 2 * I)
        h, u, d = v[:, :I], v[:, I:], s["dA"][k].double()
        sg = torch.sigmoid(h)
        a_out[k] = h * sg * u
        dw[k] = (d * a_out[k]).sum(1)
        if s["wrow"] is not None:
            d = d * s["wrow"][k].double().unsqueeze(1)
        dhu[k, :I], dhu[k, I:] = d * u * (sg + h * sg * (1 - sg)), d * h * sg
    return dhu, a_out, dw


def exact(case, seed):
    fn = {"few": _few_exact, "norm_fwd": _norm_fwd_exact, "norm_bwd": _norm_bwd_exact, "ckpt": _ckpt_exact}
    return fn[case["op"]](prepare(case, seed))
