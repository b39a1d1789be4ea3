"""Layer norm and its gradient against the formulas in 64 bits.

Bounds.  A row's mean adds at most 4 * 8 (in a thread) + 6 (in a wave) + 16
(waves) = 54 terms in a row, each addition off by 2^-24 of the magnitudes summed,
and the second sum, over the differences, corrects what the first lost; with the
few operations that use it every stage is below 80 * 2^-24 < 2^-17 of the sum of
the magnitudes that enter it, and there are at most four: F = 2^-15.  The mean
itself is kept in 32 bits (half a step of it).  A column sum adds rows / (teams)
+ waves + parts terms in a row: below (rows / 64 + 64) 2^-24 on top.  16-bit outputs are
rounded once, half a step.
"""
import pytest
import torch

from routing_schedule_expert_amd import ops
from tests.helpers import dev

pytestmark = pytest.mark.gpu

F, EPS, U = 2.0 ** -15, 1e-5, 2.0 ** -24
B, H16, F32 = torch.bfloat16, torch.float16, torch.float32
HALF = {B: 2.0 ** -8, H16: 2.0 ** -11, F32: U}
TYPES = [(B, B), (H16, H16), (F32, F32), (F32, B), (F32, H16)]
WIDTHS = [1, 2, 7, 8, 9, 64, 100, 257, 512, 520, 1000, 1024, 1031, 2048, 2049, 4096, 7168, 8192, 8193, 12288, 16400, 32768]


def make(rows, H, tx=B, ty=B, ldx=0, ldy=0, off=0, seed=1, shift=0.4):
    g = torch.Generator(device=dev())
    g.manual_seed(seed)

    def rows_of(std, t, ld, mean=0.0):
        flat = torch.full((rows * (ld or H) + 16,), float("nan"), dtype=t, device=dev())
        v = torch.as_strided(flat, (rows, H), (ld or H, 1), off)
        v.copy_((torch.randn((rows, H), generator=g, device=dev()) * std + mean).to(t))
        return v

    c = dict(n=ops.make_layer_norm_desc(rows, H, tx, ty, EPS, ldx, ldy), x=rows_of(1.5, tx, ldx, shift), dy=rows_of(0.1, ty, ldy),
             dres=rows_of(0.1, tx, ldx), rows=rows, H=H)
    c["g"] = 1 + 0.3 * torch.randn(H, generator=g, device=dev())
    c["b"] = 0.2 * torch.randn(H, generator=g, device=dev())
    return c


def near(name, got, ref, mag):
    bound = HALF[got.dtype] * ref.abs() + mag + (2.0 ** -25 if got.dtype == H16 else 1e-30)
    off = (got.double() - ref).abs()
    worst = float((off / bound).max()) if off.numel() else 0.0
    print(f"    {name}: worst error {worst:.2f} of its bound", flush=True)
    assert bool((off <= bound).all()), f"{name}: worst error {worst:.3g} of its bound"


def formula(c, g, b):
    x = c["x"].double()
    m = x.mean(1, keepdim=True)
    s = torch.rsqrt((x - m).square().mean(1, keepdim=True) + EPS)
    return x, m, s, (x - m) * s * (1 if g is None else g.double()) + (0 if b is None else b.double())


def check_fwd(c, g, b):
    bufs = ops.alloc_layer_norm(c["n"], dev())
    ops.layer_norm_fwd(c["n"], c["x"], g, b, bufs)
    x, m, s, y = formula(c, g, b)
    # what a value's distance from the mean is off by: half a step of the mean and F of the magnitudes
    em = U * m.abs() + F * ((x - m).abs() + (x - m).abs().mean(1, keepdim=True)) + U * x.abs()
    near("mean", bufs.stats[:, :1], m, F * (x - m).abs().mean(1, keepdim=True) + U * x.abs().mean(1, keepdim=True))
    near("rstd", bufs.stats[:, 1:], s, F * s + s * s * em.mean(1, keepdim=True) * 2)
    mag = em * s * (1 if g is None else g.double().abs()) * 2 + F * y.abs() + (0 if b is None else F * b.double().abs())
    near("y", bufs.y, y, mag)
    return bufs


def check_bwd(c, g, res, weight=True):
    x, m, s, _ = formula(c, None, None)
    stats = torch.cat([m, s], 1).float()
    dres = c["dres"] if res else None
    grads = ops.alloc_layer_norm_bwd(c["n"], dev(), weight=weight, bias=weight)
    ops.layer_norm_bwd(c["n"], c["x"], g, stats, c["dy"], dres, grads)
    m, s, dy = stats[:, :1].double(), stats[:, 1:].double(), c["dy"].double()
    xh = (x - m) * s
    t = dy * (1 if g is None else g.double())
    dx = s * (t - t.mean(1, keepdim=True) - xh * (t * xh).mean(1, keepdim=True))
    ta, xa = t.abs(), xh.abs() + U / F * (x.abs() + m.abs()) * s
    mag = F * s * (ta + ta.mean(1, keepdim=True) + xa * (ta * xa).mean(1, keepdim=True))
    if res:
        dx, mag = dx + dres.double(), mag + F * dres.double().abs()
    near("dx", grads.dx, dx, mag)
    if weight:
        k = F + (c["rows"] / 64 + 64) * U
        near("dg", grads.dg, (dy * xh).sum(0), k * (dy.abs() * xa).sum(0))
        near("db", grads.db, dy.sum(0), k * dy.abs().sum(0))
    return grads


@pytest.mark.parametrize("tx,ty", TYPES)
@pytest.mark.parametrize("H", WIDTHS)
def test_forward(H, tx, ty):
    for rows in (1, 5, 67):
        c = make(rows, H, tx, ty)
        check_fwd(c, c["g"], c["b"])


@pytest.mark.parametrize("tx,ty", TYPES)
@pytest.mark.parametrize("H", WIDTHS)
def test_backward(H, tx, ty):
    for rows, res in ((1, True), (37, False), (300, True)):
        c = make(rows, H, tx, ty)
        check_bwd(c, c["g"], res)


@pytest.mark.parametrize("H", [100, 1031, 2056, 7168, 12288])
def test_without_gain_and_bias(H):
    c = make(9, H)
    check_fwd(c, None, None)
    check_fwd(c, c["g"], None)
    check_fwd(c, None, c["b"])
    check_bwd(c, None, False)
    check_bwd(c, c["g"], True, weight=False)


def test_no_stats():
    c = make(40, 520)
    want = check_fwd(c, c["g"], c["b"])
    b = ops.alloc_layer_norm(c["n"], dev(), stats=False)
    ops.layer_norm_fwd(c["n"], c["x"], c["g"], c["b"], b)
    assert torch.equal(b.y, want.y)


@pytest.mark.parametrize("tx,ty", TYPES)
@pytest.mark.parametrize("H,ldx,ldy,off", [(64, 72, 80, 0), (64, 67, 71, 0), (64, 0, 0, 3), (513, 520, 528, 0), (1024, 1032, 0, 8), (1000, 1001, 1003, 1),
                                           (4096, 4104, 4097, 0), (2049, 2049, 2056, 5)])
def test_strides_and_starts(H, ldx, ldy, off, tx, ty):
    c = make(21, H, tx, ty, ldx, ldy, off)
    even = dict(c, n=ops.make_layer_norm_desc(21, H, tx, ty, EPS))
    for k in ("x", "dy", "dres"):
        even[k] = c[k].clone(memory_format=torch.contiguous_format)
    want, got = (ops.alloc_layer_norm(k["n"], dev()) for k in (even, c))
    flat = torch.full((21 * (ldy or H) + 16,), 3.0, dtype=ty, device=dev())
    got.y = torch.as_strided(flat, (21, H), (ldy or H, 1), off)
    for k, b in ((even, want), (c, got)):
        ops.layer_norm_fwd(k["n"], k["x"], k["g"], k["b"], b)
    x, m, s, y = formula(c, c["g"], c["b"])
    near("y", got.y, y, 4 * F * s * c["g"].double().abs() * ((x - m).abs() + x.abs().mean(1, keepdim=True)) + F * (y.abs() + c["b"].double().abs()))
    touched = torch.zeros_like(flat, dtype=torch.bool)
    torch.as_strided(touched, (21, H), (ldy or H, 1), off).fill_(True)
    assert bool((flat[~touched] == 3).all())
    check_bwd(c, c["g"], True)


@pytest.mark.parametrize("H", [5, 72, 1031, 4096, 7168, 7171, 12288, 12299, 20001])
def test_in_place(H):
    c = make(50, H)
    want = check_fwd(c, c["g"], c["b"])
    grads = check_bwd(c, c["g"], True)
    x = c["x"].clone()
    ops.moe_layer_norm_fwd(c["n"], x, c["g"], c["b"], x, None)
    assert torch.equal(x, want.y)
    m = c["x"].double().mean(1, keepdim=True)
    stats = torch.cat([m, torch.rsqrt((c["x"].double() - m).square().mean(1, keepdim=True) + EPS)], 1).float()
    for k in ("x", "dres", "dy"):
        a = {n: c[n].clone() for n in ("x", "dres", "dy")}
        both = torch.empty((2, H), device=dev())
        ops.moe_layer_norm_bwd(c["n"], a["x"], c["g"], stats, a["dy"], a["dres"], a[k], both[0], both[1], grads.ws)
        assert torch.equal(a[k], grads.dx) and torch.equal(both[0], grads.dg) and torch.equal(both[1], grads.db)


@pytest.mark.parametrize("H", [64, 1000, 5000])
def test_far_mean_and_equal_values(H):
    # a mean 1000 times the spread: the differences keep what 32-bit values hold of it
    c = make(20, H, F32, F32, shift=1500.0)
    check_fwd(c, c["g"], c["b"])
    c["x"].fill_(3.0)  # no spread at all: s = 1 / sqrt(eps), y = b
    b = ops.alloc_layer_norm(c["n"], dev())
    ops.layer_norm_fwd(c["n"], c["x"], c["g"], c["b"], b)
    near("rstd", b.stats[:, 1:], torch.full((20, 1), EPS, dtype=torch.float64, device=dev()).float().double().rsqrt(), torch.tensor(F * EPS ** -0.5, device=dev()))
    assert torch.equal(b.y, c["b"].expand(20, H))


def test_a_bad_row_stays_alone():
    for H in (96, 1500, 7168):
        for bad in (float("nan"), float("inf"), -float("inf")):
            c = make(30, H)
            clean = check_fwd(c, c["g"], c["b"])
            c["x"][7, H // 3] = bad
            b = ops.alloc_layer_norm(c["n"], dev())
            ops.layer_norm_fwd(c["n"], c["x"], c["g"], c["b"], b)
            rest = torch.arange(30, device=dev()) != 7
            assert bool(b.y[7].isnan().all()) and torch.equal(b.y[rest], clean.y[rest]) and torch.equal(b.stats[rest], clean.stats[rest])


def test_many_rows():
    for rows, H in ((5000, 64), (20000, 200), (4095, 2049), (3000, 7168)):
        c = make(rows, H)
        check_fwd(c, c["g"], c["b"])
        check_bwd(c, c["g"], True)


def test_no_rows():
    n = ops.make_layer_norm_desc(0, 520)
    e = torch.empty((0, 520), dtype=B, device=dev())
    ops.layer_norm_fwd(n, e, None, None, ops.alloc_layer_norm(n, dev()))
    grads = ops.alloc_layer_norm_bwd(n, dev())
    grads.both.fill_(7)
    ops.layer_norm_bwd(n, e, None, None, e, None, grads)
    assert not bool(grads.both.any())


def test_gradient_against_differences():
    c = make(6, 40, F32, F32)
    st = ops.alloc_layer_norm(c["n"], dev())
    ops.layer_norm_fwd(c["n"], c["x"], c["g"], c["b"], st)
    grads = ops.alloc_layer_norm_bwd(c["n"], dev())
    ops.layer_norm_bwd(c["n"], c["x"], c["g"], st.stats, c["dy"], None, grads)

    def value(x, g, b):
        m = x.mean(1, keepdim=True)
        return (((x - m) * torch.rsqrt((x - m).square().mean(1, keepdim=True) + EPS) * g + b) * c["dy"].double()).sum()

    at = [c[k].double() for k in ("x", "g", "b")]
    for i, got in enumerate((grads.dx, grads.dg, grads.db)):
        d = torch.randn_like(at[i])
        lo, hi = ([t + k * 1e-5 * d if j == i else t for j, t in enumerate(at)] for k in (-1, 1))
        want = float(value(*hi) - value(*lo)) / 2e-5
        assert abs(float((got.double() * d).sum()) - want) <= 1e-4 * float((got.double() * d).abs().sum()) + 1e-7


@pytest.mark.parametrize("H", [256, 7168, 12288])
def test_repeats_streams_and_graphs(H):
    c = make(500, H)
    st = check_fwd(c, c["g"], c["b"])
    sets = [(ops.alloc_layer_norm(c["n"], dev()), ops.alloc_layer_norm_bwd(c["n"], dev()), torch.cuda.Stream()) for _ in range(2)]

    def step(b, k, stream=None):
        ops.layer_norm_fwd(c["n"], c["x"], c["g"], c["b"], b, stream)
        ops.layer_norm_bwd(c["n"], c["x"], c["g"], b.stats, c["dy"], c["dres"], k, stream)

    step(*sets[0][:2])
    ref = [t.clone() for t in (sets[0][0].y, sets[0][1].dx, sets[0][1].both)]
    assert torch.equal(ref[0], st.y)
    torch.cuda.synchronize()
    for _ in range(10):
        for b, k, s in sets:
            step(b, k, s)
    torch.cuda.synchronize()
    for b, k, _ in sets:
        assert torch.equal(b.y, ref[0]) and torch.equal(k.dx, ref[1]) and torch.equal(k.both, ref[2])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(*sets[0][:2])
    for r in range(3):
        c["x"].copy_(make(500, H, seed=20 + r)["x"])
        graph.replay()
        step(*sets[1][:2])
        torch.cuda.synchronize()
        assert torch.equal(sets[0][0].y, sets[1][0].y) and torch.equal(sets[0][1].dx, sets[1][1].dx) and torch.equal(sets[0][1].both, sets[1][1].both)


def test_offsets_past_4_gib():
    rows, H, ld = 70, 1000, 1 << 25
    c = make(rows, H)
    x = torch.empty((rows, ld), dtype=B, device=dev())[:, :H]
    x.copy_(c["x"])
    n = ops.make_layer_norm_desc(rows, H, ldx=ld)
    want, got = ops.alloc_layer_norm(c["n"], dev()), ops.alloc_layer_norm(n, dev())
    ops.layer_norm_fwd(c["n"], c["x"], c["g"], c["b"], want)
    ops.layer_norm_fwd(n, x, c["g"], c["b"], got)
    assert torch.equal(want.y, got.y)
    a, b = ops.alloc_layer_norm_bwd(c["n"], dev()), ops.alloc_layer_norm_bwd(n, dev())
    ops.layer_norm_bwd(c["n"], c["x"], c["g"], want.stats, c["dy"], None, a)
    ops.layer_norm_bwd(n, x, c["g"], want.stats, c["dy"], None, b)
    assert torch.equal(a.dx, b.dx) and torch.equal(a.both, b.both)


def test_tensors_that_do_not_fit():
    c = make(8, 64)
    b = ops.alloc_layer_norm(c["n"], dev())
    for kw in (dict(x=c["x"][:7]), dict(x=c["x"].float()), dict(g=c["g"][:60]), dict(g=c["g"].double()), dict(b=c["b"].cpu()), dict(y=b.y.float()),
               dict(stats=b.stats[:4])):
        a = dict(x=c["x"], g=c["g"], b=c["b"], y=b.y, stats=b.stats) | kw
        with pytest.raises((ValueError, TypeError)):
            ops.moe_layer_norm_fwd(c["n"], *a.values())
    with pytest.raises(ops.MoeError):
        k = ops.alloc_layer_norm_bwd(c["n"], dev())
        ops.moe_layer_norm_bwd(c["n"], c["x"], c["g"], b.stats, c["dy"], None, k.dx, k.both[0], None, k.ws)


@pytest.mark.parametrize("H", [9000, 20000, 20001, 32768])
def test_more_rows_than_workgroups(H):
    # two and four chunks a thread, every workgroup with rows after its first
    for tx, ty in ((B, B), (F32, F32)):
        c = make(1200, H, tx, ty)
        check_fwd(c, c["g"], c["b"])
        check_bwd(c, c["g"], True)
