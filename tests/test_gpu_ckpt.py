"""8-bit activation checkpoints: the format bit for bit, the SwiGLU backward on
them against its formulas in 64 bits, and the layer backward that reads them.
"""
import numpy as np
import pytest
import torch

from routing_schedule_expert_amd import inputs, ops
from tests.helpers import dev, rel_l2

pytestmark = pytest.mark.gpu

B = ops.CKPT_BLOCK


def pack_np(x: np.ndarray):
    """The format in numpy's IEEE float32."""
    v = np.ascontiguousarray(x, np.float32).reshape(x.shape[0], -1, B)
    amax = np.abs(v).max(-1, keepdims=True)
    with np.errstate(all="ignore"):
        q = np.rint(v * (np.float32(127) * (np.float32(1) / amax)))
        s = amax / np.float32(127)
    tiny, bad = amax < np.float32(2.0 ** -100), ~np.isfinite(amax)
    q = np.where(tiny | bad, 0, q).astype(np.int8)
    s = np.where(bad, np.float32("nan"), np.where(tiny, np.float32(0), s))
    return q.reshape(x.shape), s[..., 0].astype(np.float32)


def check_pack(x):
    q, s = ops.ckpt_pack(x)
    wq, ws = pack_np(x.float().cpu().numpy())
    assert np.array_equal(q.cpu().numpy(), wq)
    assert np.array_equal(s.cpu().numpy().view(np.uint32) & 0x7FFFFFFF, ws.view(np.uint32) & 0x7FFFFFFF)  # a NaN's sign is free


@pytest.mark.parametrize("rows,cols", [(1, 128), (3, 256), (257, 384), (33, 4096), (2, 65536)])
def test_pack_matches_the_format(rows, cols):
    check_pack(inputs.normal_bf16_device((rows, cols), 1.3, rows, dev()))


def test_pack_edges():
    x = inputs.normal_bf16_device((40, 256), 1.0, 3, dev())
    x[0] = 0
    x[1] = -0.0
    x[2, 5] = float("inf")
    x[3, 200] = float("nan")
    x[4] *= 2.0 ** -105     # below the smallest block
    x[5] = 2.0 ** -100      # at it
    x[6] *= 2.0 ** -130     # subnormal
    x[7] *= 2.0 ** 120
    x[8, 0] = torch.finfo(torch.bfloat16).max
    x[9] = 1.0
    for k in range(10, 40):  # quotients that end on a half: x / amax = m / 254
        x[k] = torch.arange(256, device=dev()).sub(128).float().mul(0.5).to(torch.bfloat16)
        x[k, 7] = x[k, 135] = 63.5 + 0.5 * (k - 10)
    check_pack(x)


def test_pack_every_bf16_value():
    # every bit pattern, in blocks of neighbours
    v = torch.arange(65536, dtype=torch.int32, device=dev()).to(torch.int16).view(torch.bfloat16)
    check_pack(v.reshape(64, 1024))
    check_pack(v.reshape(512, 128).t().contiguous().reshape(128, 512))


@pytest.mark.parametrize("n", [0, 1, 5, 9, 100, -3])
def test_rows_past_the_count_stay(n):
    x = inputs.normal_bf16_device((9, 256), 1.0, 4, dev())
    q, s = torch.full((9, 256), 77, dtype=torch.int8, device=dev()), torch.full((9, 2), 7.0, device=dev())
    cnt = torch.tensor([n], dtype=torch.int32, device=dev())
    ops.moe_ckpt_pack(x, q, s, cnt)
    k = max(0, min(n, 9))
    wq, ws = ops.ckpt_pack(x)
    assert torch.equal(q[:k], wq[:k]) and torch.equal(s[:k], ws[:k])
    assert bool((q[k:] == 77).all()) and bool((s[k:] == 7).all())
    dA = inputs.normal_bf16_device((9, 128), 1.0, 5, dev())
    out = [torch.full((9, m), 7.0, dtype=t, device=dev()) for m, t in ((256, torch.bfloat16), (128, torch.bfloat16), (1, torch.float32))]
    ops.moe_ckpt_swiglu_bwd(wq, ws, dA, None, *out, cnt)
    full = [torch.zeros_like(t) for t in out]
    ops.moe_ckpt_swiglu_bwd(wq, ws, dA, None, *full)
    for a, f in zip(out, full):
        assert torch.equal(a[:k], f[:k]) and bool((a[k:] == 7).all())


def decode(q, s):
    return (q.double().unflatten(-1, (-1, B)) * s.double().unsqueeze(-1)).flatten(-2)


@pytest.mark.parametrize("weighted", [True, False])
@pytest.mark.parametrize("rows,I", [(1, 128), (70, 128), (33, 256), (19, 384), (40, 512), (5, 896), (9, 1024), (65, 2048), (3, 8192)])
def test_swiglu_bwd_matches_formula(rows, I, weighted):
    """bf16 outputs: 2^-8 of the value; the 32-bit chain (decode, exp of |h| <= 10,
    reciprocal, products) stays below 24 steps of 2^-24 of the terms' magnitudes;
    the row's sum adds I / lanes + 6 terms in a row."""
    x = inputs.normal_bf16_device((rows, 2 * I), 1.5, rows + I, dev())
    dA = inputs.normal_bf16_device((rows, I), 0.1, rows, dev())
    w = torch.rand(rows, device=dev()) if weighted else None
    q, s = ops.ckpt_pack(x)
    dHU, A = torch.empty_like(x), torch.empty_like(dA)
    dw = torch.empty(rows, device=dev())
    ops.moe_ckpt_swiglu_bwd(q, s, dA, w, dHU, A, dw)
    v = decode(q, s)
    h, u, d = v[:, :I], v[:, I:], dA.double()
    sg = torch.sigmoid(h)
    a = h * sg * u
    dd = d if w is None else d * w.double().unsqueeze(1)
    F = 24 * 2.0 ** -24
    for name, got, ref, mag in (("A", A, a, a.abs()), ("dh", dHU[:, :I], dd * u * sg * (1 + h * (1 - sg)), (dd * u * sg).abs() * (1 + h.abs())),
                                ("du", dHU[:, I:], dd * h * sg, (dd * h * sg).abs())):
        err, bound = (got.double() - ref).abs(), 2.0 ** -8 * ref.abs() + F * mag + 1e-30
        assert bool((err <= bound).all()), f"{name}: {float((err / bound).max()):.3g} of its bound"
    err, bound = (dw.double() - (d * a).sum(1)).abs(), (F + (I / 8 + 8) * 2.0 ** -24) * (d * a).abs().sum(1) + 1e-30
    assert bool((err <= bound).all())
    # the optional outputs left out: the same gradient
    again = torch.zeros_like(dHU)
    ops.moe_ckpt_swiglu_bwd(q, s, dA, w, again, None, None)
    assert torch.equal(again, dHU)


def test_swiglu_bwd_against_differences():
    I, h = 256, 1e-6
    x = inputs.normal_bf16_device((4, 2 * I), 1.0, 8, dev())
    dA = inputs.normal_bf16_device((4, I), 0.5, 9, dev())
    w = torch.rand(4, device=dev())
    q, s = ops.ckpt_pack(x)
    dHU, A, dw = torch.empty_like(x), torch.empty_like(dA), torch.empty(4, device=dev())
    ops.moe_ckpt_swiglu_bwd(q, s, dA, w, dHU, A, dw)
    v, dd = decode(q, s), dA.double() * w.double().unsqueeze(1)
    act = lambda t: t[:, :I] * torch.sigmoid(t[:, :I]) * t[:, I:]  # noqa: E731
    dirn = torch.randn_like(v)
    num = float(((act(v + h * dirn) - act(v - h * dirn)) * dd).sum() / (2 * h))
    tol = float((dirn.abs() * dHU.double().abs()).sum()) * 2.0 ** -8 * 1.01 + 1e-6
    assert abs(num - float((dHU.double() * dirn).sum())) <= tol
    # d/dw of sum w dA a is dw itself
    assert np.allclose(dw.double().cpu().numpy(), (dA.double() * act(v)).sum(1).cpu().numpy(), rtol=0, atol=1e-4)


def layer(P, Np, E, K, L, base, H, I, seed=3, routing="uniform"):
    d_in = inputs.make_layer_inputs_device(seed, P, Np, E, K, L, H, I, dev(), routing=routing, base=base, with_grad=True)
    d = ops.make_desc(P, Np, K, E, L, expert_base=base, H=H, I=I)
    routes = torch.from_numpy(d_in["routes"]).to(dev())
    w = torch.from_numpy(d_in["w"]).to(dev())
    b = ops.alloc_fwd(d, dev())
    ops.layer_fwd(d, routes, w, d_in["X"], d_in["W13"], d_in["W2"], b)
    return d, routes, w, d_in, b


def grads(d):
    f32 = torch.float32
    return (torch.empty((d.P, d.Np, d.H), dtype=torch.bfloat16, device=dev()), torch.empty((d.L, 2 * d.I, d.H), dtype=f32, device=dev()),
            torch.empty((d.L, d.H, d.I), dtype=f32, device=dev()), torch.empty((d.P, d.Np, d.K), dtype=f32, device=dev()))


def pack_layer(d, b):
    cap = ops.capacity_rows(d)
    q = torch.full((cap, 2 * d.I), 99, dtype=torch.int8, device=dev())
    s = torch.full((cap, 2 * d.I // B), float("nan"), device=dev())
    ops.moe_ckpt_pack(b.HU, q, s, b.seg_off[d.L:])
    return q, s


def run_ckpt(d, w, d_in, b, q, s, ws=None):
    g = grads(d)
    if ws is None:
        ws = torch.empty(ops.workspace_bytes(d, ops.MOE_OP_LAYER_BWD_CKPT), dtype=torch.uint8, device=dev())
    ops.moe_layer_bwd_ckpt(d, d_in["dOut"], w, d_in["X"], b.phi, b.route_row, b.seg_off, q, s, d_in["W13"], d_in["W2"], *g, ws)
    return g


LAYERS = [(1, 40, 4, 2, 4, 0, 256, 128), (2, 300, 8, 2, 4, 2, 512, 384), (1, 1, 4, 1, 2, 0, 256, 128), (1, 16, 8, 2, 2, 0, 256, 256)]


@pytest.mark.parametrize("dims", LAYERS)
def test_layer_bwd_on_exact_checkpoints(dims):
    """Where h and u are on a grid that the codes hold exactly (code * 2^k, 127 in
    every block), the checkpointed backward is moe_layer_bwd on them, bit for bit
    in dX, dW13 and dW2; dw takes a before its rounding to bf16, which is off by
    2^-8 of each term at most."""
    d, routes, w, d_in, b = layer(*dims)
    n = int(b.seg_off[d.L])
    hu = torch.randint(-127, 128, (n, 2 * d.I), device=dev()).float()
    hu[:, ::B] = 127
    hu *= torch.exp2(torch.randint(-7, -4, (n, 2 * d.I // B), device=dev()).float()).repeat_interleave(B, 1)
    hu[b.phi[:n, 0] < 0] = 0
    b.HU[:n] = hu.to(torch.bfloat16)
    q, s = pack_layer(d, b)
    assert torch.equal(decode(q[:n], s[:n]), b.HU[:n].double())
    zero = torch.zeros((n, d.I), dtype=torch.bfloat16, device=dev())
    ops.moe_ckpt_swiglu_bwd(q, s, zero, None, torch.empty_like(b.HU[:n]), b.A, None)
    want = grads(d)
    ws = torch.empty(ops.workspace_bytes(d, ops.MOE_OP_LAYER_BWD), dtype=torch.uint8, device=dev())
    ops.moe_layer_bwd(d, d_in["dOut"], routes, w, b.phi, b.route_row, b.seg_off, b.Xd, b.HU, b.A, d_in["W13"], d_in["W2"], *want, ws)
    got = run_ckpt(d, w, d_in, b, q, s)
    for name, x, y in zip(("dX", "dW13", "dW2"), got, want):
        assert torch.equal(x, y), name
    local = b.route_row >= 0
    assert not got[3][~local].any()
    # the terms' magnitudes: dA' = dO W2 and a, in 64 bits
    rows = b.route_row[local].long()
    tok = b.phi[rows].long()
    e = torch.searchsorted(b.seg_off[:d.L + 1].long(), rows, right=True) - 1
    dap = torch.stack([d_in["dOut"][p, t].double() @ d_in["W2"][k].double() for (p, t), k in zip(tok.tolist(), e.tolist())]) if len(rows) else None
    if dap is not None:
        v = decode(q[rows], s[rows])
        a = v[:, :d.I] * torch.sigmoid(v[:, :d.I]) * v[:, d.I:]
        ref, mag = (dap * a).sum(1), (dap * a).abs().sum(1)
        assert bool(((got[3][local].double() - ref).abs() <= 1e-5 * mag + 1e-12).all())
        assert bool(((want[3][local].double() - ref).abs() <= (2.0 ** -8 + 1e-5) * mag + 1e-12).all())


@pytest.mark.parametrize("dims", LAYERS[:2])
def test_layer_bwd_ckpt_near_the_exact_backward(dims):
    """A linear code of a Gaussian block of 128 is off by amax / 127 / sqrt(12), at
    most 1% of the block's rms (amax <= 4 rms); dh = dA u silu'(h) and du = dA
    silu(h) carry u's and h's error with slopes (|silu'| <= 1.1, |silu''| <= 0.5)
    that leave each gradient within 3% of the one without codes."""
    d, routes, w, d_in, b = layer(*dims)
    want = grads(d)
    ws = torch.empty(ops.workspace_bytes(d, ops.MOE_OP_LAYER_BWD), dtype=torch.uint8, device=dev())
    ops.moe_layer_bwd(d, d_in["dOut"], routes, w, b.phi, b.route_row, b.seg_off, b.Xd, b.HU, b.A, d_in["W13"], d_in["W2"], *want, ws)
    q, s = pack_layer(d, b)
    n = int(b.seg_off[d.L])
    assert bool((q[n:] == 99).all()) and bool(s[n:].isnan().all())
    ws = torch.full((ops.workspace_bytes(d, ops.MOE_OP_LAYER_BWD_CKPT),), 0x5A, dtype=torch.uint8, device=dev())
    got = run_ckpt(d, w, d_in, b, q, s, ws)
    for name, x, y in zip(("dX", "dW13", "dW2", "dw"), got, want):
        r = rel_l2(x.float().cpu().numpy(), y.float().cpu().numpy())
        print(f"    {name}: {r:.2e}", flush=True)
        assert r <= 3e-2, name
    again = run_ckpt(d, w, d_in, b, q, s, ws)
    assert all(torch.equal(x, y) for x, y in zip(got, again))


def test_layer_bwd_ckpt_captured_and_replayed():
    d, routes, w, d_in, b = layer(2, 60, 8, 2, 4, 2, 256, 128)
    q, s = pack_layer(d, b)
    ws = torch.empty(ops.workspace_bytes(d, ops.MOE_OP_LAYER_BWD_CKPT), dtype=torch.uint8, device=dev())
    g = grads(d)

    def step():
        ops.moe_ckpt_pack(b.HU, q, s, b.seg_off[d.L:])
        ops.moe_layer_bwd_ckpt(d, d_in["dOut"], w, d_in["X"], b.phi, b.route_row, b.seg_off, q, s, d_in["W13"], d_in["W2"], *g, ws)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in range(4):
        d_in["dOut"].copy_(inputs.normal_bf16_device(d_in["dOut"].shape, 1.0, 70 + seed, dev()))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in g]
        step()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, g))


def test_ckpt_binding_refuses_wrong_buffers():
    x = inputs.normal_bf16_device((4, 256), 1.0, 1, dev())
    q, s = ops.ckpt_pack(x)
    with pytest.raises(ValueError):
        ops.moe_ckpt_pack(x, q[:3].contiguous(), s)
    with pytest.raises(ValueError):
        ops.moe_ckpt_pack(x.float(), q, s)
    with pytest.raises(ops.MoeError):
        ops.moe_ckpt_pack(x[:, :64].contiguous(), q, s)
    with pytest.raises(ValueError):
        ops.moe_ckpt_pack(x, q, s, torch.tensor([3], device=dev()))


def test_pack_allocates_on_the_stream_it_runs_on():
    # memory that the current stream has freed but still writes does not go to a call on another stream
    x = inputs.normal_bf16_device((64, 4096), 1.0, 21, dev())
    want, ws = ops.ckpt_pack(x)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    big = inputs.normal_bf16_device((4096, 8192), 1.0, 22, dev()).float()
    for _ in range(3):
        for t in (torch.empty_like(want), torch.empty_like(ws)):
            for _ in range(4):
                big.add_(1.0)
            t.fill_(3)
            del t
        q, sc = ops.ckpt_pack(x, stream=s)
        torch.cuda.synchronize()
        assert torch.equal(q, want) and torch.equal(sc, ws)


def test_layer_bwd_ckpt_binding_needs_a_workspace():
    d = ops.make_desc(1, 4, 1, 2, 2, H=256, I=128)
    cap, n, bf, i32, f32 = ops.capacity_rows(d), 4, torch.bfloat16, torch.int32, torch.float32

    def z(dtype, *shape):
        return torch.zeros(shape, dtype=dtype, device=dev())

    with pytest.raises(ops.MoeError):
        ops.moe_layer_bwd_ckpt(d, z(bf, n, 256), z(f32, n), z(bf, n, 256), z(i32, cap, 2), z(i32, n), z(i32, 3),
                               z(torch.int8, cap, 256), z(f32, cap, 2), z(bf, 2, 256, 256), z(bf, 2, 256, 128), z(bf, n, 256),
                               z(f32, 2, 256, 256), z(f32, 2, 256, 128), z(f32, n), None)
