"""The gated feed-forward block and its gradient against the formulas in 64 bits.

Bounds, element by element.  A product's sum of K terms is off by at most
(K + 32) 2^-24 of the sum of the terms' magnitudes (K - 1 additions and, where K
is cut into parts, up to 16 more).  An activation and its slope are a short chain
of 32-bit operations on arguments below 16: off by 2^-17 of (1 + |h|), their own
scale, at most; an error dh of h moves either by at most 1.2 dh (the slopes of
the activations stay below 1.2, those of the slopes below 1.2 too; ReLU's slope,
which jumps, is compared where |h| is above its error).  A rounding to 16 bits is
off by half a step, 2^-8 (bf16) or 2^-11 (fp16) of the value; fp16 loses up to
2^-25 more below its normal range.  These errors go through the products that
follow with the magnitudes of the other operand.
"""
import pytest
import torch

from routing_schedule_expert_amd import ops
from tests.helpers import dev

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
ACT = 2.0 ** -17
ACTS = {"silu": ops.MOE_ACT_SILU, "gelu": ops.MOE_ACT_GELU, "gelu_tanh": ops.MOE_ACT_GELU_TANH, "relu": ops.MOE_ACT_RELU}
HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: U}
TINY = {torch.bfloat16: 1e-37, torch.float16: 2.0 ** -25, torch.float32: 1e-37}


def act(kind, h):
    f = torch.nn.functional
    return {"silu": f.silu, "relu": torch.relu, "gelu": f.gelu, "gelu_tanh": lambda v: f.gelu(v, approximate="tanh")}[kind](h)


def slope(kind, h):
    h = h.detach().clone().requires_grad_(True)
    return torch.autograd.grad(act(kind, h).sum(), h)[0]


def make(rows, H, I, kind="silu", dtype=torch.bfloat16, ldx=0, ldo=0, seed=1):
    g = torch.Generator(device=dev())
    g.manual_seed(seed)

    def rnd(shape, std):
        return (torch.randn(shape, generator=g, device=dev()) * std).to(dtype)

    def spread(t, ld):  # the same rows ld apart, NaN between them
        if not ld:
            return t
        wide = torch.full((rows, ld), float("nan"), dtype=dtype, device=dev())
        wide[:, :H] = t
        return wide[:, :H]

    c = dict(n=ops.make_ffn_desc(rows, H, I, ACTS[kind], dtype, ldx, ldo), kind=kind, dtype=dtype, I=I, H=H, rows=rows)
    c["X"] = spread(rnd((rows, H), 1.0), ldx)
    c["W13"], c["W2"] = rnd((2 * I, H), 1.5 * H ** -0.5), rnd((H, I), I ** -0.5)
    c["dOut"] = spread(rnd((rows, H), 0.1), ldo)
    return c


def fwd(c, save=True, stream=None):
    b = ops.alloc_gated_ffn(c["n"], dev(), save_hu=save)
    for t in (b.out, b.HU, b.A):
        if t is not None:
            t.fill_(7)
    ops.gated_ffn_fwd(c["n"], c["X"], c["W13"], c["W2"], b, stream)
    return b


def near(name, got, ref, err, c=None):
    t = got.dtype
    bound = HALF[t] * (ref.abs() + err) + err + TINY[t]
    off = (got.double() - ref).abs()
    worst = float((off / bound).max()) if off.numel() else 0.0
    print(f"    {name}: worst error {worst:.2f} of its bound", flush=True)
    assert bool((off <= bound).all()), f"{name}: worst error {worst:.3g} of its bound"


def sums(K):
    return (K + 32) * U


def forward64(c):
    """out, HU, a and the bounds of their errors before they are rounded."""
    I, H, half = c["I"], c["H"], HALF[c["dtype"]]
    X, W13, W2 = c["X"].double(), c["W13"].double(), c["W2"].double()
    hu = X @ W13.t()
    ehu = sums(H) * (X.abs() @ W13.abs().t())
    h, u = hu[:, :I], hu[:, I:]
    v = act(c["kind"], h)
    a = v * u
    ev = 1.2 * ehu[:, :I] + ACT * (1 + h.abs())
    ea = ev * (u.abs() + ehu[:, I:]) + v.abs() * ehu[:, I:] + 2 * U * a.abs()
    round_a = ea + half * (a.abs() + ea) + TINY[c["dtype"]]
    out = a @ W2.t()
    eout = round_a @ W2.abs().t() + sums(I) * ((a.abs() + round_a) @ W2.abs().t())
    return (out, hu, a), (eout, ehu, ea)


SHAPES = [(1, 8, 8), (1, 256, 128), (3, 72, 40), (8, 264, 1032), (16, 2048, 264), (17, 136, 8), (33, 512, 520), (64, 1032, 64), (65, 64, 64),
          (130, 8, 264), (200, 520, 72), (257, 264, 328), (333, 1032, 520), (1021, 1288, 392), (8200, 1544, 776)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("rows,H,I", SHAPES)
def test_forward(rows, H, I, dtype):
    c = make(rows, H, I, dtype=dtype, kind="silu" if dtype == torch.bfloat16 else "gelu_tanh")
    b = fwd(c)
    (out, hu, a), (eout, ehu, ea) = forward64(c)
    near("HU", b.HU, hu, ehu)
    near("A", b.A, a, ea)
    near("out", b.out, out, eout)


@pytest.mark.parametrize("kind", list(ACTS))
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_activations(kind, dtype):
    c = make(70, 136, 200, kind, dtype)
    c["W13"] *= 3  # arguments far into the tails
    b = fwd(c)
    (out, hu, a), (eout, ehu, ea) = forward64(c)
    near("A", b.A, a, ea)
    near("out", b.out, out, eout)
    plain = fwd(c, save=False)
    assert plain.HU is None and torch.equal(plain.out, b.out) and torch.equal(plain.A, b.A)


def backward64(c, HU, A, given):
    """dX, dW13, dW2 of the HU and a that the call reads, and their error bounds."""
    I, H, rows, half, kind = c["I"], c["H"], c["rows"], HALF[c["dtype"]], c["kind"]
    X, W13, W2, g = c["X"].double(), c["W13"].double(), c["W2"].double(), c["dOut"].double()
    h, u = HU[:, :I].double(), HU[:, I:].double()
    v, s = act(kind, h), slope(kind, h)
    ev = ACT * (1 + h.abs())
    dA = g @ W2
    eA = sums(H) * (g.abs() @ W2.abs())
    dhu = torch.cat([dA * u * s, dA * v], 1)
    e = torch.cat([u.abs() * ((dA.abs() + eA) * ev + eA * s.abs()), (dA.abs() + eA) * ev + eA * v.abs()], 1) + 3 * U * dhu.abs()
    e = e + half * (dhu.abs() + e) + TINY[c["dtype"]]
    a = A.double() if given else v * u
    ea = torch.zeros_like(a) if given else (ev * u.abs() + U * a.abs()) * (1 + half) + half * a.abs() + TINY[c["dtype"]]
    m = dhu.abs() + e
    return ((dhu @ W13, e @ W13.abs() + sums(2 * I) * (m @ W13.abs())),
            (dhu.t() @ X, e.t() @ X.abs() + sums(rows) * (m.t() @ X.abs())),
            (g.t() @ a, g.abs().t() @ ea + sums(rows) * (g.abs().t() @ (a.abs() + ea))))


def kept(c):
    """HU and a as a forward leaves them, from the 64-bit values."""
    (_, hu, a), _ = forward64(c)
    return hu.to(c["dtype"]), a.to(c["dtype"])


@pytest.mark.parametrize("given", [True, False])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("rows,H,I", SHAPES + [(300, 4104, 2056)])
def test_backward(rows, H, I, dtype, given):
    kind = ("silu", "gelu", "gelu_tanh", "relu")[(rows + H + I // 8 + given) % 4]
    c = make(rows, H, I, kind, dtype)
    HU, A = kept(c)
    b = ops.alloc_gated_ffn_bwd(c["n"], dev(), dw_dtype=torch.float32 if (rows + given) % 2 else dtype)
    for t in (b.dX, b.dW13, b.dW2):
        t.fill_(7)
    ops.gated_ffn_bwd(c["n"], c["dOut"], c["X"], HU, A if given else None, c["W13"], c["W2"], b)
    for name, got, (ref, err) in zip(("dX", "dW13", "dW2"), (b.dX, b.dW13, b.dW2), backward64(c, HU, A, given)):
        near(name, got, ref, err)


@pytest.mark.parametrize("kind", list(ACTS))
def test_gradient_against_differences(kind):
    # the whole block in 64 bits, moved along a direction by t = 1e-5: differences are off by t^2 and the noise of 1e-16 / t;
    # the call's roundings (fp16: four of 2^-11 in a row) put its own directional derivative within 2e-3 of the sum of magnitudes
    c = make(40, 72, 48, kind, torch.float16)
    if kind == "relu":  # no argument near the jump
        c["W13"][: c["I"]].abs_(), c["X"].abs_()
    HU, A = kept(c)
    b = ops.alloc_gated_ffn_bwd(c["n"], dev())
    ops.gated_ffn_bwd(c["n"], c["dOut"], c["X"], HU, A, c["W13"], c["W2"], b)

    def value(X, W13, W2):
        hu = X @ W13.t()
        return ((act(kind, hu[:, : c["I"]]) * hu[:, c["I"]:]) @ W2.t() * c["dOut"].double()).sum()

    at = [c[k].double() for k in ("X", "W13", "W2")]
    for i, got in enumerate((b.dX, b.dW13, b.dW2)):
        d = torch.randn_like(at[i])
        lo, hi = ([t + k * 1e-5 * d if j == i else t for j, t in enumerate(at)] for k in (-1, 1))
        want = float(value(*hi) - value(*lo)) / 2e-5
        assert abs(float((got.double() * d).sum()) - want) <= 2e-3 * float((got.double() * d).abs().sum()) + 1e-6


def test_accumulate_and_absent():
    c = make(77, 136, 72)
    HU, A = kept(c)
    n = c["n"]
    full = ops.alloc_gated_ffn_bwd(n, dev())
    ops.gated_ffn_bwd(n, c["dOut"], c["X"], HU, A, c["W13"], c["W2"], full)
    acc = ops.alloc_gated_ffn_bwd(n, dev())
    w13, w2 = torch.randn_like(acc.dW13), torch.randn_like(acc.dW2)
    acc.dW13.copy_(w13), acc.dW2.copy_(w2)
    ops.gated_ffn_bwd(n, c["dOut"], c["X"], HU, A, c["W13"], c["W2"], acc, accumulate=True)
    assert torch.equal(acc.dW13, w13 + full.dW13) and torch.equal(acc.dW2, w2 + full.dW2) and torch.equal(acc.dX, full.dX)
    args = (n, c["dOut"], c["X"], HU, A, c["W13"], c["W2"])
    only = ops.alloc_gated_ffn_bwd(n, dev())
    ops.moe_gated_ffn_bwd(*args, only.dX, None, None, only.ws)
    ops.moe_gated_ffn_bwd(*args, None, only.dW13, None, only.ws)
    ops.moe_gated_ffn_bwd(*args, None, None, only.dW2, only.ws)
    assert torch.equal(only.dX, full.dX) and torch.equal(only.dW13, full.dW13) and torch.equal(only.dW2, full.dW2)


def test_accumulate_in_parts():
    # many rows of a narrow block: the weights' gradients are cut along the rows
    c = make(5000, 64, 40)
    HU, A = kept(c)
    b = ops.alloc_gated_ffn_bwd(c["n"], dev())
    b.dW13.fill_(1), b.dW2.fill_(1)
    ops.gated_ffn_bwd(c["n"], c["dOut"], c["X"], HU, A, c["W13"], c["W2"], b, accumulate=True)
    _, (dW13, e13), (dW2, e2) = backward64(c, HU, A, True)
    near("dW13", b.dW13, 1 + dW13, e13)
    near("dW2", b.dW2, 1 + dW2, e2)


@pytest.mark.parametrize("rows", [5, 300])
def test_strides(rows):
    H, I = 136, 72
    a, c = make(rows, H, I), make(rows, H, I, ldx=168, ldo=264)
    assert torch.equal(a["X"], c["X"])
    want, b = fwd(a), fwd(c)
    assert torch.equal(want.out, b.out) and torch.equal(want.A, b.A)
    gap = torch.as_strided(b.out, (rows - 1, 264 - H), (264, 1), b.out.storage_offset() + H)
    whole = torch.full((rows, 264), 3.0, dtype=torch.bfloat16, device=dev())
    ops.moe_gated_ffn_fwd(c["n"], c["X"], c["W13"], c["W2"], None, b.A, whole[:, :H], b.ws)
    assert torch.equal(whole[:, :H], want.out) and bool((whole[:, H:] == 3).all()) and gap.numel()
    g, d = (ops.alloc_gated_ffn_bwd(k["n"], dev()) for k in (a, c))
    wide = torch.full((rows, 168), 3.0, dtype=torch.bfloat16, device=dev())
    ops.gated_ffn_bwd(a["n"], a["dOut"], a["X"], want.HU, want.A, a["W13"], a["W2"], g)
    ops.moe_gated_ffn_bwd(c["n"], c["dOut"], c["X"], want.HU, want.A, c["W13"], c["W2"], wide[:, :H], d.dW13, d.dW2, d.ws)
    assert torch.equal(wide[:, :H], g.dX) and bool((wide[:, H:] == 3).all())
    assert torch.equal(d.dW13, g.dW13) and torch.equal(d.dW2, g.dW2)


@pytest.mark.parametrize("rows,H,I", [(1, 264, 136), (63, 264, 136), (200, 264, 136), (300, 1032, 520)])
def test_rows_behind_the_last_stay(rows, H, I):
    c = make(rows, H, I)
    big = {k: torch.full((rows + 300, w), 5.0, dtype=torch.bfloat16, device=dev()) for k, w in (("out", H), ("HU", 2 * I), ("A", I), ("dX", H))}
    b = ops.alloc_gated_ffn(c["n"], dev())
    ops.moe_gated_ffn_fwd(c["n"], c["X"], c["W13"], c["W2"], big["HU"], big["A"], big["out"], b.ws)
    g = ops.alloc_gated_ffn_bwd(c["n"], dev())
    ops.moe_gated_ffn_bwd(c["n"], c["dOut"], c["X"], big["HU"], big["A"], c["W13"], c["W2"], big["dX"], g.dW13, g.dW2, g.ws)
    for t in big.values():
        assert bool((t[rows:] == 5).all()) and not bool((t[:rows] == 5).all())


@pytest.mark.parametrize("rows", [9, 150, 1500])
def test_a_bad_row_stays_alone(rows):
    c = make(rows, 264, 136)
    clean = fwd(c)
    r = rows // 2
    bad = dict(c, X=c["X"].clone())
    bad["X"][r, 5], bad["X"][r, 6] = float("nan"), float("inf")
    b = fwd(bad)
    rest = torch.arange(rows, device=dev()) != r
    assert bool(b.out[r].isnan().all()) and torch.equal(b.out[rest], clean.out[rest]) and torch.equal(b.HU[rest], clean.HU[rest])
    g = ops.alloc_gated_ffn_bwd(c["n"], dev())
    ops.gated_ffn_bwd(c["n"], c["dOut"], c["X"], clean.HU, clean.A, c["W13"], c["W2"], g)
    d = c["dOut"].clone()
    d[r, 3] = float("nan")
    gb = ops.alloc_gated_ffn_bwd(c["n"], dev())
    ops.gated_ffn_bwd(c["n"], d, c["X"], clean.HU, clean.A, c["W13"], c["W2"], gb)
    assert bool(gb.dX[r].isnan().all()) and torch.equal(gb.dX[rest], g.dX[rest])
    assert bool(gb.dW2[3].isnan().all()) and torch.equal(gb.dW2[4:], g.dW2[4:]) and torch.equal(gb.dW2[:3], g.dW2[:3])


def test_a_row_does_not_depend_on_the_others():
    # rows of one call of 64 rows or fewer, and of one of many, each against the row by itself, to the bound of sums in another order
    c = make(600, 264, 136)
    b = fwd(c)
    (out, _, _), (eout, _, _) = forward64(c)
    one = dict(c, n=ops.make_ffn_desc(1, 264, 136), X=c["X"][77:78].clone(), rows=1)
    near("out", fwd(one).out, out[77:78], eout[77:78])
    swapped = dict(c, X=c["X"].clone())
    swapped["X"][100:] = swapped["X"][100:].flip(0)
    assert torch.equal(fwd(swapped).out[:100], b.out[:100])


@pytest.mark.parametrize("rows", [0])
def test_no_rows(rows):
    n = ops.make_ffn_desc(0, 136, 72)
    e = torch.empty((0, 136), dtype=torch.bfloat16, device=dev())
    W13, W2 = torch.zeros((144, 136), dtype=torch.bfloat16, device=dev()), torch.zeros((136, 72), dtype=torch.bfloat16, device=dev())
    b = ops.alloc_gated_ffn(n, dev())
    ops.gated_ffn_fwd(n, e, W13, W2, b)
    for dt in (torch.float32, torch.bfloat16):
        g = ops.alloc_gated_ffn_bwd(n, dev(), dw_dtype=dt)
        g.dW13.fill_(7), g.dW2.fill_(7)
        if dt == torch.float32:
            ops.gated_ffn_bwd(n, e, e, b.HU, b.A, W13, W2, g, accumulate=True)
            assert bool((g.dW13 == 7).all()) and bool((g.dW2 == 7).all())
        ops.gated_ffn_bwd(n, e, e, b.HU, b.A, W13, W2, g)
        assert not bool(g.dW13.any()) and not bool(g.dW2.any())


@pytest.mark.parametrize("rows", [4, 500])
def test_repeats_streams_and_graphs(rows):
    c = make(rows, 520, 264)
    HU, A = kept(c)
    want = fwd(c)
    grads = [ops.alloc_gated_ffn_bwd(c["n"], dev()) for _ in range(2)]
    step = lambda b, g, stream=None: (ops.gated_ffn_fwd(c["n"], c["X"], c["W13"], c["W2"], b, stream),  # noqa: E731
                                      ops.gated_ffn_bwd(c["n"], c["dOut"], c["X"], b.HU, None, c["W13"], c["W2"], g, stream=stream))
    bufs = [fwd(c) for _ in range(2)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    step(bufs[0], grads[0])
    ref = [t.clone() for t in (bufs[0].out, grads[0].dX, grads[0].dW13, grads[0].dW2)]
    assert torch.equal(ref[0], want.out)
    torch.cuda.synchronize()
    for _ in range(10):
        for b, g, s in zip(bufs, grads, streams):
            step(b, g, s)
    torch.cuda.synchronize()
    for b, g in zip(bufs, grads):
        assert all(torch.equal(x, y) for x, y in zip(ref, (b.out, g.dX, g.dW13, g.dW2)))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(bufs[0], grads[0])
    for k in range(3):
        c["X"].copy_(make(rows, 520, 264, seed=10 + k)["X"])
        graph.replay()
        step(bufs[1], grads[1])
        torch.cuda.synchronize()
        assert torch.equal(bufs[0].out, bufs[1].out) and torch.equal(grads[0].dX, grads[1].dX)
        assert torch.equal(grads[0].dW13, grads[1].dW13) and torch.equal(grads[0].dW2, grads[1].dW2)


def test_offsets_past_4_gib():
    rows, H, I, ld = 2500, 64, 40, 1 << 20
    a = make(rows, H, I)
    X = torch.empty((rows, ld), dtype=torch.bfloat16, device=dev())[:, :H]
    X.copy_(a["X"])
    c = dict(a, n=ops.make_ffn_desc(rows, H, I, ldx=ld, ldo=ld), X=X)
    want, b = fwd(a), ops.alloc_gated_ffn(c["n"], dev())
    ops.gated_ffn_fwd(c["n"], X, a["W13"], a["W2"], b)
    assert torch.equal(b.out, want.out)
    dOut = X.new_empty((rows, ld))[:, :H]
    dOut.copy_(a["dOut"])
    g, d = ops.alloc_gated_ffn_bwd(a["n"], dev()), ops.alloc_gated_ffn_bwd(c["n"], dev())
    ops.gated_ffn_bwd(a["n"], a["dOut"], a["X"], want.HU, want.A, a["W13"], a["W2"], g)
    ops.gated_ffn_bwd(c["n"], dOut, X, want.HU, want.A, a["W13"], a["W2"], d)
    assert torch.equal(d.dX, g.dX) and torch.equal(d.dW13, g.dW13) and torch.equal(d.dW2, g.dW2)


def test_tensors_that_do_not_fit():
    c = make(8, 64, 40)
    b, n = ops.alloc_gated_ffn(c["n"], dev()), c["n"]
    for kw in (dict(X=c["X"][:7]), dict(X=c["X"].float()), dict(W13=c["W13"][:-1]), dict(W2=c["W2"].cpu()), dict(HU=c["X"]), dict(A=b.A[:3]),
               dict(out=c["W2"].t())):
        a = dict(X=c["X"], W13=c["W13"], W2=c["W2"], HU=b.HU, A=b.A, out=b.out) | kw
        with pytest.raises((ValueError, TypeError)):
            ops.moe_gated_ffn_fwd(n, *a.values(), b.ws)
    g = ops.alloc_gated_ffn_bwd(n, dev())
    with pytest.raises(ValueError):
        ops.moe_gated_ffn_bwd(n, c["dOut"], c["X"], b.HU, b.A, c["W13"], c["W2"], g.dX, g.dW13, g.dW2.bfloat16(), g.ws)
    with pytest.raises(ops.MoeError):
        ops.moe_gated_ffn_bwd(n, c["dOut"], c["X"], b.HU, b.A, c["W13"], c["W2"], g.dX, g.dW13.bfloat16(), g.dW2.bfloat16(), g.ws, True)
    with pytest.raises(ops.MoeError):
        ops.moe_gated_ffn_bwd(n, c["dOut"], c["X"], b.HU, b.A, c["W13"], c["W2"], g.dX, g.dW13, g.dW2, g.ws[:16])


@pytest.mark.parametrize("given", [True, False])
@pytest.mark.parametrize("kind", list(ACTS))
def test_fp16_values_kept_as_infinities(kind, given):
    # h and u past 65504 lie in HU as infinities, which stand for numbers: where the slope or the value is 0, or nothing
    # arrives, their products are 0.  The reference has 200 in their place, where each activation is at its limits in 64 bits.
    I, f16 = 40, torch.float16
    c = make(80, 72, I, kind, f16)
    HU, A = kept(c)
    inf = float("inf")
    HU[3, 5], HU[3, I + 5] = -inf, 0.01
    HU[4, 6], HU[4, I + 6] = -inf, -inf
    HU[5, 7], HU[5, I + 7] = -inf, inf
    HU[6, 8], HU[6, I + 8] = inf, 0.01
    HU[7, 9], HU[7, I + 9] = inf, inf  # a row that nothing arrives for
    HU[7, 10], HU[7, I + 10] = 1.0, inf
    A[torch.tensor([3, 4, 5], device=dev()), torch.tensor([5, 6, 7], device=dev())] = 0.0
    A[6, 8], A[7, 9:11] = 700.0, 3.0
    c["dOut"][7] = 0.0
    b = ops.alloc_gated_ffn_bwd(c["n"], dev())
    ops.gated_ffn_bwd(c["n"], c["dOut"], c["X"], HU, A if given else None, c["W13"], c["W2"], b)
    ref = HU.double().nan_to_num(posinf=200.0, neginf=-200.0)
    (dX, eX), (dW13, e13), (dW2, e2) = backward64(c, ref, A, given)
    rows = torch.arange(80, device=dev()) != 6  # du there is infinite, as h is
    near("dX", b.dX[rows], dX[rows], eX[rows])
    rows = torch.arange(2 * I, device=dev()) != I + 8
    near("dW13", b.dW13[rows], dW13[rows], e13[rows])
    assert not bool(b.dX[6].isfinite().any()) and not bool(b.dW13[I + 8].isfinite().any())
    cols = torch.tensor([k for k in range(I) if given or k not in (8, 9, 10)], device=dev())  # a there is infinite too
    near("dW2", b.dW2[:, cols], dW2[:, cols], e2[:, cols])
    # NaN is no such number
    HU[9, 5], HU[10, I + 5], HU[10, 5] = float("nan"), float("nan"), -inf
    ops.gated_ffn_bwd(c["n"], c["dOut"], c["X"], HU, A if given else None, c["W13"], c["W2"], b)
    assert bool(b.dX[10].isnan().all()) and (kind == "relu" or bool(b.dX[9].isnan().all()))


@pytest.mark.parametrize("kind", list(ACTS))
def test_fp16_gradient_of_a_finite_forward(kind):
    # one gate argument of -70,000: the forward's outputs are finite, and so is what its HU gives
    c = make(70, 72, 40, kind, torch.float16)
    c["X"][11, 3], c["W13"][17, 3] = 250.0, -280.0
    b = fwd(c)
    assert float(b.HU[11, 17]) == -float("inf") and float(b.A[11, 17]) == 0.0 and bool(b.out.isfinite().all())
    c["dOut"][11] /= 64
    for A in (b.A, None):
        g = ops.alloc_gated_ffn_bwd(c["n"], dev())
        ops.gated_ffn_bwd(c["n"], c["dOut"], c["X"], b.HU, A, c["W13"], c["W2"], g)
        for name, got, (ref, err) in zip(("dX", "dW13", "dW2"), (g.dX, g.dW13, g.dW2), backward64(c, b.HU.double().nan_to_num(neginf=-200.0), b.A, A is not None)):
            near(name, got, ref, err)


@pytest.mark.parametrize("rows", [5, 300])
def test_out_in_the_place_of_x(rows):
    c = make(rows, 264, 136)
    want, b, x = fwd(c), ops.alloc_gated_ffn(c["n"], dev()), c["X"].clone()
    ops.moe_gated_ffn_fwd(c["n"], x, c["W13"], c["W2"], b.HU, b.A, x, b.ws)
    assert torch.equal(x, want.out) and torch.equal(b.A, want.A)
    g = ops.alloc_gated_ffn_bwd(c["n"], dev(), dw_dtype=torch.bfloat16)
    for dX, dW13, dW2 in ((c["X"], None, None), (c["dOut"], None, None), (None, c["W13"], None), (None, None, c["W2"]), (None, c["X"].new_empty(0), None)):
        with pytest.raises((ops.MoeError, ValueError)):
            ops.moe_gated_ffn_bwd(c["n"], c["dOut"], c["X"], b.HU, b.A, c["W13"], c["W2"], dX, dW13, dW2, g.ws)


@pytest.mark.parametrize("sign", [1, -1])
def test_fp16_infinite_u_where_nothing_arrives(sign):
    # a column of W2 without weights: nothing arrives at dA, but a, made again from an infinite u, is infinite
    I = 40
    c = make(80, 72, I, "silu", torch.float16)
    c["W2"][:, 10] = 0.0
    HU, A = kept(c)
    HU[7, 10], HU[7, I + 10] = 1.0, sign * float("inf")
    b = ops.alloc_gated_ffn_bwd(c["n"], dev())
    ops.gated_ffn_bwd(c["n"], c["dOut"], c["X"], HU, None, c["W13"], c["W2"], b)
    assert torch.equal(b.dW2[:, 10], torch.where(c["dOut"][7] > 0, sign, -sign) * float("inf"))
    ref = HU.double().nan_to_num(posinf=200.0, neginf=-200.0)
    (dX, eX), (dW13, e13), (dW2, e2) = backward64(c, ref, A, False)
    rest = torch.arange(I, device=dev()) != 10
    near("dX", b.dX, dX, eX)
    near("dW13", b.dW13, dW13, e13)
    near("dW2", b.dW2[:, rest], dW2[:, rest], e2[:, rest])
