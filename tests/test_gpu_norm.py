"""The block norms and their gradient against the formulas in 64 bits.

Bounds.  A bf16 output is rounded once: 2^-8 of its value.  Besides that, every
output is a short chain of 32-bit operations: each rounds by 2^-24 of its
result, a mean of H products adds at most 32 (in a thread) + 6 (in a wave) + 16
(waves) = 54 additions in a row, an exponential of |z| <= 8 loses |z| + 2 steps.
One stage (a mean, its use, the gate) is so below 80 * 2^-24 < 2^-17 of the sum
of the magnitudes that enter it, and there are at most four stages: F = 2^-15.
`mags` follows the formulas with magnitudes in place of signed terms.  A column
sum adds at most rows / 512 + 1 + 32 + 4 terms in a row on top.
"""
import itertools

import pytest
import torch

from routing_schedule_expert_amd import ops
from tests.helpers import dev

pytestmark = pytest.mark.gpu

F, EPS = 2.0 ** -15, 1e-5
GATES = {"none": ops.MOE_GATE_NONE, "token": ops.MOE_GATE_TOKEN, "elem": ops.MOE_GATE_ELEM}


def make(rows, H, gate="none", res="bf16", post=True, pre=True, alpha=0.9, beta=0.7, y=True, seed=1):
    g = torch.Generator(device=dev())
    g.manual_seed(seed)

    def rnd(shape, std, dtype=torch.bfloat16):
        return (torch.randn(shape, generator=g, device=dev()) * std).to(dtype)

    rt = torch.float32 if res == "fp32" else torch.bfloat16
    c = dict(n=ops.make_norm_desc(rows, H, GATES[gate], res == "fp32", alpha, beta, EPS), gate=gate)
    c["y"] = rnd((rows, H), 0.4) if y else None
    c["r"] = rnd((rows, H), 1.5, rt)
    c["z"] = None if gate == "none" else rnd((rows,), 2.0, torch.float32).clamp(-8, 8) if gate == "token" else rnd((rows, H), 2.0).clamp(-8, 8)
    c["g_post"] = 1 + rnd((H,), 0.3, torch.float32) if post else None
    c["g_pre"] = 1 + rnd((H,), 0.3, torch.float32) if pre else None
    c["r_out"] = torch.full((rows, H), 7.0, dtype=rt, device=dev()) if y else None
    c["xn"] = torch.full((rows, H), 7.0, dtype=torch.bfloat16, device=dev()) if pre else None
    c["stats"] = torch.full((rows, 2), 7.0, device=dev())
    c["dr_out"], c["dxn"] = rnd((rows, H), 0.1, rt), rnd((rows, H), 0.1) if pre else None
    return c


def fwd(c, stream=None):
    ops.moe_block_norm_fwd(c["n"], c["y"], c["r"], c["z"], c["g_post"], c["g_pre"], c["r_out"], c["xn"], c["stats"], stream)


def bwd(c, stream=None):
    b = ops.alloc_norm_bwd(c["n"], dev(), c["g_post"] is not None, c["g_pre"] is not None, c["y"] is not None)
    for t in (b.dy, b.dr, b.dz, b.dg_post, b.dg_pre):
        if t is not None:
            t.fill_(7)
    ops.block_norm_bwd(c["n"], c["y"], c["r"], c["z"], c["g_post"], c["g_pre"], c["stats"], c["dr_out"], c["dxn"], b, stream)
    return b


def dbl(t):
    return None if t is None else t.double()


def formula(c, y, r, z, g_post, g_pre):
    """r', xn (None where absent), in the type of its arguments."""
    n = c["n"]
    if y is None:
        new = r
    else:
        p = y if g_post is None else y * torch.rsqrt(y.square().mean(1, keepdim=True) + n.eps) * g_post
        s = 1.0 if z is None else torch.sigmoid(z if c["gate"] == "elem" else z.unsqueeze(1))
        new = n.alpha * r + n.beta * s * p
    return new, None if g_pre is None else new * torch.rsqrt(new.square().mean(1, keepdim=True) + n.eps) * g_pre


def mags(c):
    """Sums of the magnitudes that enter each output."""
    n = c["n"]
    y, r, z, g_post, g_pre = (dbl(c[k]) for k in ("y", "r", "z", "g_post", "g_pre"))
    new, _ = formula(c, y, r, z, g_post, g_pre)
    m = {}
    s = torch.ones_like(r)
    if y is None:
        rm = r.abs()
    else:
        ystd = torch.ones_like(r[:, :1]) if g_post is None else torch.rsqrt(y.square().mean(1, keepdim=True) + n.eps)
        yh = y * ystd
        p = yh if g_post is None else yh * g_post
        if z is not None:
            s = torch.sigmoid(z if c["gate"] == "elem" else z.unsqueeze(1)).expand_as(r)
        rm = (n.alpha * r).abs() + (n.beta * s * p).abs()
    m["r_out"] = rm
    up = 0 if c["dr_out"] is None else dbl(c["dr_out"]).abs()
    if g_pre is not None:
        rstd = torch.rsqrt(new.square().mean(1, keepdim=True) + n.eps)
        m["xn"] = rm * rstd * g_pre.abs()
        dx, xm = dbl(c["dxn"]).abs(), rm * rstd
        m["dg_pre"] = (dx * xm).sum(0)
        t = dx * g_pre.abs()
        up = up + rstd * (t + xm * (t * xm).mean(1, keepdim=True))
    m["dr"] = (n.alpha if y is not None else 1.0) * up
    if y is not None:
        dz = n.beta * up * p.abs() * s  # s (1 - s) <= s: 1 - s is itself a rounded difference
        m["dz"] = dz.sum(1) if c["gate"] == "token" else dz
        q = n.beta * up * s
        m["dg_post"] = (q * yh.abs()).sum(0)
        if g_post is not None:
            q = q * g_post.abs()
            q = ystd * (q + yh.abs() * (q * yh.abs()).mean(1, keepdim=True))
        m["dy"] = q
    return m


def near(name, got, ref, mag, extra=0.0):
    half = 2.0 ** -8 if got.dtype == torch.bfloat16 else 2.0 ** -24
    bound = half * ref.abs() + (F + extra) * mag + 1e-30
    err = (got.double() - ref).abs()
    assert bool((err <= bound).all()), f"{name}: worst error {float((err / bound).max()):.3g} of its bound"


def check(c):
    n = c["n"]
    ins = {k: dbl(c[k]) for k in ("y", "r", "z", "g_post", "g_pre")}
    for v in ins.values():
        if v is not None:
            v.requires_grad_(True)
    new, xn = formula(c, **ins)
    fwd(c)
    m = mags(c)
    if c["y"] is not None:
        near("r_out", c["r_out"], new.detach(), m["r_out"])
    if xn is not None:
        near("xn", c["xn"], xn.detach(), m["xn"])
    one = torch.ones((n.rows, 1), dtype=torch.float64, device=dev())
    for k, (v, g) in enumerate(((ins["y"], c["g_post"]), (new, c["g_pre"]))):
        want = 0 * one if g is None else torch.rsqrt(v.detach().square().mean(1, keepdim=True) + n.eps)
        near("stats", c["stats"][:, k:k + 1], want, want)
    loss = 0 if c["dr_out"] is None else (new * dbl(c["dr_out"])).sum()
    if xn is not None:
        loss = loss + (xn * dbl(c["dxn"])).sum()
    loss.backward()
    b = bwd(c)
    extra = (n.rows / 512 + 37) * 2.0 ** -24
    for name, got, leaf, e in (("dy", b.dy, "y", 0), ("dr", b.dr, "r", 0), ("dz", b.dz, "z", 0), ("dg_post", b.dg_post, "g_post", extra),
                               ("dg_pre", b.dg_pre, "g_pre", extra)):
        assert (got is None) == (c[leaf] is None)
        if got is not None:
            near(name, got, ins[leaf].grad, m[name], e)
    return b


SHAPES = [(1, 8), (3, 64), (5, 520), (2, 2048), (7, 2056), (3, 4104), (4, 7168), (2, 8192), (3, 8200), (2, 16384), (2, 32768)]


@pytest.mark.parametrize("rows,H", SHAPES)
def test_norm_shapes(rows, H):
    check(make(rows, H, "elem", "bf16"))
    check(make(rows, H, "token", "fp32", seed=2))


@pytest.mark.parametrize("gate,res,post,pre", itertools.product(GATES, ("bf16", "fp32"), (True, False), (True, False)))
def test_norm_forms(gate, res, post, pre):
    check(make(9, 776, gate, res, post, pre))


@pytest.mark.parametrize("res", ["bf16", "fp32"])
@pytest.mark.parametrize("rows,H", [(6, 512), (3, 2304), (2, 9000)])
def test_norm_before_the_first_block(res, rows, H):
    # no block output yet: the pre-norm of the residual stream alone
    c = make(rows, H, res=res, y=False, post=False)
    check(c)
    c["dr_out"] = None  # nothing else uses the stream (the last norm of a model)
    check(c)


@pytest.mark.parametrize("rows", [511, 512, 513, 2500, 9001])
def test_norm_many_rows(rows):
    # more rows than workgroups of the backward; every column sum in its order
    check(make(rows, 256, "token"))
    check(make(rows, 1032, "none", seed=3))


def test_norm_repeats_bitwise():
    c = make(700, 1032, "elem")
    fwd(c)
    first = (c["r_out"].clone(), c["xn"].clone(), c["stats"].clone())
    g = bwd(c)
    for _ in range(3):
        fwd(c)
        assert all(torch.equal(a, b) for a, b in zip(first, (c["r_out"], c["xn"], c["stats"])))
        h = bwd(c)
        assert all(torch.equal(getattr(g, k), getattr(h, k)) for k in ("dy", "dr", "dz", "dg_post", "dg_pre"))


def test_norm_gradient_against_differences():
    # directional derivatives of the 64-bit formula; the kernel's gradient may be off by its own rounding
    c = make(6, 264, "elem", "fp32")
    fwd(c)
    b = bwd(c)
    m = mags(c)
    ins = {k: dbl(c[k]) for k in ("y", "r", "z", "g_post", "g_pre")}

    def loss(**kw):
        new, xn = formula(c, **(ins | kw))
        return float((new * dbl(c["dr_out"])).sum() + (xn * dbl(c["dxn"])).sum())

    for name, grad in (("y", b.dy), ("r", b.dr), ("z", b.dz), ("g_post", b.dg_post), ("g_pre", b.dg_pre)):
        v = torch.randn_like(ins[name])
        h = 1e-5
        num = (loss(**{name: ins[name] + h * v}) - loss(**{name: ins[name] - h * v})) / (2 * h)
        half = 2.0 ** -8 if grad.dtype == torch.bfloat16 else 2.0 ** -24
        tol = float((v.abs() * (half * grad.double().abs() * 1.01 + 2 * F * m["d" + name])).sum()) + 1e-6
        assert abs(num - float((grad.double() * v).sum())) <= tol, name


def test_norm_in_place():
    c = make(40, 2056, "elem")
    fwd(c)
    want = (c["r_out"].clone(), c["xn"].clone())
    r, y, z = c["r"].clone(), c["y"].clone(), c["z"].clone()
    ops.moe_block_norm_fwd(c["n"], y, r, z, c["g_post"], c["g_pre"], r, y, c["stats"])
    assert torch.equal(r, want[0]) and torch.equal(y, want[1])
    b = bwd(c)
    want = [t.clone() for t in (b.dy, b.dr, b.dz)]
    y, dr = c["y"].clone(), c["dr_out"].clone()
    ops.moe_block_norm_bwd(c["n"], y, c["r"], z, c["g_post"], c["g_pre"], c["stats"], dr, c["dxn"], y, dr, z, b.dg_post, b.dg_pre, b.ws)
    assert all(torch.equal(a, w) for a, w in zip((y, dr, z), want))


def test_norm_rows_stand_alone():
    # a row with an infinity or NaN, one of zeros, and the rest untouched by them
    c = make(12, 520, "token")
    fwd(c)
    clean, g = c["r_out"].clone(), bwd(c)
    c["y"][3, 5] = float("nan")
    c["r"][7, 9] = float("inf")
    c["y"][9] = 0
    c["r"][10], c["y"][10] = 0, 0
    fwd(c)
    keep = [i for i in range(12) if i not in (3, 7, 9, 10)]
    assert torch.equal(c["r_out"][keep], clean[keep])
    assert torch.equal(c["xn"][10], torch.zeros_like(c["xn"][10]))
    assert bool(c["xn"][3].isnan().all()) and not bool(c["r_out"][[9, 10]].isnan().any())
    h = bwd(c)
    assert torch.equal(h.dr[keep], g.dr[keep]) and torch.equal(h.dy[keep], g.dy[keep]) and torch.equal(h.dz[keep], g.dz[keep])


def test_norm_without_rows():
    c = make(0, 512, "token")
    fwd(c)
    b = bwd(c)
    assert not b.dg_post.any() and not b.dg_pre.any()


def test_norm_captured_and_replayed():
    c = make(600, 1032, "token")
    fwd(c)
    b = bwd(c)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        fwd(c)
        ops.block_norm_bwd(c["n"], c["y"], c["r"], c["z"], c["g_post"], c["g_pre"], c["stats"], c["dr_out"], c["dxn"], b)
    for seed in range(4):
        other = make(600, 1032, "token", seed=20 + seed)
        for k in ("y", "r", "z", "dr_out", "dxn", "g_post", "g_pre"):
            c[k].copy_(other[k])
        g.replay()
        torch.cuda.synchronize()
        fwd(other)
        want = bwd(other)
        assert torch.equal(c["r_out"], other["r_out"]) and torch.equal(c["xn"], other["xn"])
        assert all(torch.equal(getattr(b, k), getattr(want, k)) for k in ("dy", "dr", "dz", "dg_post", "dg_pre"))


def test_norm_binding_refuses_wrong_buffers():
    c = make(4, 512, "token")
    with pytest.raises(ValueError):
        ops.moe_block_norm_fwd(c["n"], c["y"], c["r"].float(), c["z"], c["g_post"], c["g_pre"], c["r_out"], c["xn"], c["stats"])
    with pytest.raises(ValueError):
        ops.moe_block_norm_fwd(c["n"], c["y"], c["r"], c["z"], c["g_post"], c["g_pre"], c["r_out"], c["xn"][:3].contiguous(), c["stats"])
    with pytest.raises(ops.MoeError):
        ops.moe_block_norm_fwd(c["n"], c["y"], c["r"], None, c["g_post"], c["g_pre"], c["r_out"], c["xn"], c["stats"])


@pytest.mark.parametrize("H", [1024, 9000, 20000])
def test_norm_gradient_without_a_pre_norm_ignores_r(H):
    # dr and dy do not depend on the residual where nothing norms it, whatever it holds
    g = torch.Generator(device=dev()).manual_seed(H)
    n = ops.make_norm_desc(3, H, gate=ops.MOE_GATE_TOKEN, alpha=0.5)
    y, r, up = (torch.randn((3, H), generator=g, device=dev()).to(torch.bfloat16) for _ in range(3))
    z, gp = torch.randn(3, generator=g, device=dev()), torch.rand(H, generator=g, device=dev())
    out, stats = torch.empty_like(r), torch.empty((3, 2), device=dev())

    def run():
        b = ops.alloc_norm_bwd(n, dev(), pre=False)
        ops.moe_block_norm_fwd(n, y, r, z, gp, None, out, None, stats)
        ops.block_norm_bwd(n, y, r, z, gp, None, stats, up, None, b)
        return [b.dy, b.dr, b.dz, b.dg_post]

    want = run()
    r[1, 5], r[2, H - 1] = float("inf"), float("nan")
    got = run()
    assert all(torch.equal(a, c) and bool(a.isfinite().all()) for a, c in zip(got, want))


@pytest.mark.parametrize("gate,res", [("elem", "bf16"), ("token", "fp32"), ("none", "bf16")])
@pytest.mark.parametrize("rows,H", [(257, 8200), (600, 12296), (5, 16392), (520, 24584)])
def test_norm_long_rows(rows, H, gate, res):
    # rows that the backward reads twice, several a workgroup
    c = make(rows, H, gate, res, seed=4)
    check(c)
    b = bwd(c)
    first = [None if t is None else t.clone() for t in (b.dy, b.dr, b.dz, b.dg_post, b.dg_pre)]
    b = bwd(c)
    assert all(a is None or torch.equal(a, t) for a, t in zip(first, (b.dy, b.dr, b.dz, b.dg_post, b.dg_pre)))
    # in place: dy over y, dr over what arrives for r', dz over z; then dy over dxn, dr over r
    y, up, z, dxn, r = (None if c[k] is None else c[k].clone() for k in ("y", "dr_out", "z", "dxn", "r"))
    ops.moe_block_norm_bwd(c["n"], y, c["r"], z, c["g_post"], c["g_pre"], c["stats"], up, c["dxn"], y, up, z, b.dg_post, b.dg_pre, b.ws)
    assert all(a is None or torch.equal(a, t) for a, t in zip(first, (y, up, z, b.dg_post, b.dg_pre)))
    ops.moe_block_norm_bwd(c["n"], c["y"], r, c["z"], c["g_post"], c["g_pre"], c["stats"], c["dr_out"], dxn, dxn, r, b.dz, b.dg_post, b.dg_pre, b.ws)
    assert torch.equal(dxn, first[0]) and torch.equal(r, first[1])


@pytest.mark.parametrize("gate", GATES)
@pytest.mark.parametrize("H", [1024, 9000, 20000])
def test_norm_gradient_without_norms_ignores_y(H, gate):
    # dr and dy do not depend on the block's output where nothing norms it, whatever it holds; the gate's gradient alone does
    c = make(4, H, gate, post=False, pre=False, seed=H)
    c["dr_out"][1, 5] = 1
    fwd(c)
    want = bwd(c)
    c["y"][1, 5], c["y"][2, H - 1] = float("inf"), float("nan")
    fwd(c)
    got = bwd(c)
    assert torch.equal(got.dr, want.dr) and torch.equal(got.dy, want.dy) and bool(got.dy.isfinite().all())
    if gate == "token":
        assert torch.equal(got.dz[[0, 3]], want.dz[[0, 3]]) and bool(got.dz[1].isinf()) and bool(got.dz[2].isnan())
    if gate == "elem":
        assert bool(got.dz[1, 5].isinf()) and bool(got.dz[2, H - 1].isnan())
        got.dz[1, 5], got.dz[2, H - 1] = want.dz[1, 5], want.dz[2, H - 1]
        assert torch.equal(got.dz, want.dz)


def column_steps(n):
    """Additions in a row of the backward's column sums: a workgroup's rows, the partial rows that one thread of
    the second launch takes, and its tree over the threads of a column (16 columns a workgroup below H = 2048, or 64)."""
    groups = ops.block_norm_workspace_bytes(n) // (8 * n.H)
    cols = 16 if n.H < 2048 else 64
    return -(-n.rows // groups) + -(-groups * cols // 1024) + (1024 // cols).bit_length() - 1


@pytest.mark.parametrize("gate,res", [("elem", "bf16"), ("elem", "fp32"), ("token", "bf16"), ("token", "fp32")])
@pytest.mark.parametrize("rows,H", [(61, 776), (1030, 1032), (24, 8192), (19, 9000), (7, 20000)])
def test_norm_gradient_of_open_and_closed_gates(rows, H, gate, res):
    """Gates up to 10^-13 from open or closed.  s (1 - s) is what the gate's gradient scales with, so its error is
    counted relative to that: exponentials of |z| <= 30 are off by 32 steps of 2^-24 each, in s and in 1 - s,
    64 * 2^-24 = 2^-18 beside the other stages.  dz is compared with the formula itself (64 bits lose 1 - s too)."""
    c = make(rows, H, gate, res, seed=H)
    z = torch.linspace(-30, 30, c["z"].numel(), device=dev())[torch.randperm(c["z"].numel(), device=dev())]
    c["z"] = z.reshape(c["z"].shape).to(c["z"].dtype)
    n = c["n"]
    ins = {k: dbl(c[k]) for k in ("y", "r", "z", "g_post", "g_pre")}
    for k in ("y", "r", "g_post", "g_pre"):
        ins[k].requires_grad_(True)
    new, xn = formula(c, **ins)
    ((new * dbl(c["dr_out"])).sum() + (xn * dbl(c["dxn"])).sum()).backward()
    fwd(c)
    b, m = bwd(c), mags(c)
    more, sums = 2.0 ** -18, column_steps(n) * 2.0 ** -24
    near("xn", c["xn"], xn.detach(), m["xn"], more)
    near("dy", b.dy, ins["y"].grad, m["dy"], more)
    near("dr", b.dr, ins["r"].grad, m["dr"], more)
    near("dg_post", b.dg_post, ins["g_post"].grad, m["dg_post"], more + sums)
    near("dg_pre", b.dg_pre, ins["g_pre"].grad, m["dg_pre"], more + sums)
    z = ins["z"] if gate == "elem" else ins["z"].unsqueeze(1)
    y = dbl(c["y"])
    p = y * torch.rsqrt(y.square().mean(1, keepdim=True) + n.eps) * dbl(c["g_post"])
    slope = n.beta * p * torch.sigmoid(z) * torch.sigmoid(-z)
    want, mag = slope * ins["r"].grad / n.alpha, slope.abs() * m["dr"] / n.alpha
    if gate == "token":
        want, mag = want.sum(1), mag.sum(1)
    near("dz", b.dz, want, mag, more)


@pytest.mark.parametrize("gate", ["token", "elem"])
@pytest.mark.parametrize("H", [1032, 9000])
def test_norm_gates_shut_and_open_for_good(H, gate):
    # gates of minus and plus infinity are those of -200 and 200: nothing passes, or all of it, and no gradient reaches them
    c = make(6, H, gate, seed=H)
    out = []
    for far in (200.0, float("inf")):
        c["z"][0], c["z"][1] = -far, far
        if gate == "elem":
            c["z"][3, 7], c["z"][3, H - 1] = far, -far
        fwd(c)
        b = bwd(c)
        out.append([t.clone() for t in (c["r_out"], c["xn"], b.dr, b.dy, b.dz, b.dg_post, b.dg_pre)])
    for a, t in zip(*out):
        assert torch.equal(a, t) and bool(t.isfinite().all())
    dz = out[1][4]
    assert not dz[:2].any() and not out[1][3][0].any() and bool(dz[2:].any())
    if gate == "elem":
        assert not dz[3, 7] and not dz[3, H - 1]
