"""The operators run together, as a block uses them, and at sizes whose byte
offsets pass 32 bits.

A decode step: pre-norm, the layer for a few tokens, post-norm with gate and
residual and the next pre-norm.  Between the 64-bit chain and the calls stand
four roundings to bf16 (x, the activations, the layer's output, the result), each
off by 2^-8 / sqrt(3) rms at most: together below 1e-2 in rel-L2, the parity bar
of the layer's other float outputs.

A training step: the same block with the layer's forward, its pre-activations
packed to 8 bits, and the backward through all of it.  The codes put up to 3% on
the gradients that pass the SwiGLU (tests/test_gpu_ckpt.py), the roundings 1%.
"""
import pytest
import torch

from routing_schedule_expert_amd import ops
from tests.helpers import dev

pytestmark = pytest.mark.gpu

EPS = 1e-6


def rand(shape, std, seed, dtype=torch.bfloat16):
    g = torch.Generator(device=dev())
    g.manual_seed(seed)
    return (torch.randn(shape, generator=g, device=dev()) * std).to(dtype)


def rms(v):
    return v * torch.rsqrt(v.square().mean(-1, keepdim=True) + EPS)


def block64(r, g1, ids, w, W13, W2, z, g_post, g_pre, alpha, beta, S13=None, S2=None):
    """The block in the type of its arguments: (layer output, r', next x)."""
    x = rms(r) * g1
    out = torch.zeros_like(x)

    def ffn(v, a, b):
        h = v @ a.t()
        n = b.shape[-1]
        return (torch.nn.functional.silu(h[:, :n]) * h[:, n:]) @ b.t()

    for e in range(W13.shape[0]):
        t, j = (ids == e).nonzero(as_tuple=True)
        if len(t):
            out = out.index_add(0, t, w[t, j].unsqueeze(1) * ffn(x[t], W13[e], W2[e]))
    if S13 is not None:
        out = out + ffn(x, S13, S2)
    new = alpha * r + beta * torch.sigmoid(z).unsqueeze(1) * rms(out) * g_post
    return out, new, rms(new) * g_pre


def rel(a, b):
    return float((a.double() - b).norm() / b.norm())


def setup(T, E, K, H, I, Is=0):
    c = dict(ids=torch.rand((T, E), device=dev()).argsort(1)[:, :K], w=torch.rand((T, K), device=dev()),
             r=rand((T, H), 1.0, 1), g1=1 + rand((H,), 0.1, 2, torch.float32), W13=rand((E, 2 * I, H), 1.5 * H ** -0.5, 3),
             W2=rand((E, H, I), I ** -0.5, 4), z=rand((T,), 1.0, 5, torch.float32), g_post=1 + rand((H,), 0.1, 6, torch.float32),
             g_pre=1 + rand((H,), 0.1, 7, torch.float32))
    c["S13"], c["S2"] = (rand((2 * Is, H), 1.5 * H ** -0.5, 8), rand((H, Is), Is ** -0.5, 9)) if Is else (None, None)
    return c


@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("T", [1, 9, 48])
def test_decode_step(T, mx):
    E, K, H, I, Is = 8, 2, 512, 256, 128
    c = setup(T, E, K, H, I, Is)
    d = ops.make_desc(1, T, K, E, E, H=H, I=I)
    routes, w = c["ids"].to(torch.int32).reshape(1, T, K).contiguous(), c["w"].reshape(1, T, K)
    W13, W2 = c["W13"], c["W2"]
    if mx:
        q13, q2 = ops.quantize_mx(W13), ops.quantize_mx(W2)
        W13, W2 = ((q.view(torch.float8_e4m3fn).double().unflatten(-1, (-1, 32)) * torch.exp2(s.double() - 127).unsqueeze(-1)).flatten(-2)
                   for q, s in (q13, q2))
    pre, post = ops.make_norm_desc(T, H, eps=EPS), ops.make_norm_desc(T, H, ops.MOE_GATE_TOKEN, alpha=0.9, beta=0.6, eps=EPS)
    x, xn, new = torch.empty_like(c["r"]), torch.empty_like(c["r"]), torch.empty_like(c["r"])
    stats, few = torch.empty((T, 2), device=dev()), ops.alloc_few(d, dev(), Is)

    def step():
        ops.moe_block_norm_fwd(pre, None, c["r"], None, None, c["g1"], None, x, stats)
        a = (d, routes, w, x.view(1, T, H))
        if mx:
            ops.layer_fwd_few_mx(*a, *q13, *q2, few, c["S13"], c["S2"])
        else:
            ops.layer_fwd_few(*a, c["W13"], c["W2"], few, c["S13"], c["S2"])
        ops.moe_block_norm_fwd(post, few.out.view(T, H), c["r"], c["z"], c["g_post"], c["g_pre"], new, xn, stats)

    def check():
        D = torch.Tensor.double
        out, new64, x64 = block64(D(c["r"]), D(c["g1"]), c["ids"], D(c["w"]), W13.double(), W2.double(), D(c["z"]), D(c["g_post"]),
                                  D(c["g_pre"]), 0.9, 0.6, D(c["S13"]), D(c["S2"]))
        assert rel(few.out.view(T, H), out) <= 1e-2 and rel(new, new64) <= 1e-2 and rel(xn, x64) <= 1e-2

    step()
    check()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for k in range(3):  # a replay on new inputs, eager work on the same buffers in between
        c["r"].copy_(rand((T, H), 1.0, 100 + k))
        graph.replay()
        check()
        replayed = (few.out.clone(), new.clone(), xn.clone())
        step()
        assert all(torch.equal(a, b) for a, b in zip(replayed, (few.out, new, xn)))


def test_training_step():
    T, E, K, H, I = 300, 4, 2, 512, 256
    c = setup(T, E, K, H, I)
    d = ops.make_desc(1, T, K, E, E, H=H, I=I)
    routes, w = c["ids"].to(torch.int32).reshape(1, T, K).contiguous(), c["w"].reshape(1, T, K).contiguous()
    pre, post = ops.make_norm_desc(T, H, eps=EPS), ops.make_norm_desc(T, H, ops.MOE_GATE_TOKEN, alpha=0.9, beta=0.6, eps=EPS)
    gr, gx = rand((T, H), 1.0, 20), rand((T, H), 1.0, 21)
    # forward
    x, xn, new = torch.empty_like(c["r"]), torch.empty_like(c["r"]), torch.empty_like(c["r"])
    st1, st2 = torch.empty((T, 2), device=dev()), torch.empty((T, 2), device=dev())
    ops.moe_block_norm_fwd(pre, None, c["r"], None, None, c["g1"], None, x, st1)
    b = ops.alloc_fwd(d, dev(), save_xd=False)
    ops.layer_fwd(d, routes, w, x.view(1, T, H), c["W13"], c["W2"], b)
    q, s = ops.ckpt_pack(b.HU, b.seg_off[d.L:])
    b.HU.fill_(float("nan"))  # only the codes are kept
    b.A.fill_(float("nan"))
    y = b.out.view(T, H)
    ops.moe_block_norm_fwd(post, y, c["r"], c["z"], c["g_post"], c["g_pre"], new, xn, st2)
    # backward
    g2 = ops.alloc_norm_bwd(post, dev())
    ops.block_norm_bwd(post, y, c["r"], c["z"], c["g_post"], c["g_pre"], st2, gr, gx, g2)
    f32 = torch.float32
    dX, dw = torch.empty((1, T, H), dtype=torch.bfloat16, device=dev()), torch.empty((1, T, K), dtype=f32, device=dev())
    dW13, dW2 = torch.empty((E, 2 * I, H), dtype=f32, device=dev()), torch.empty((E, H, I), dtype=f32, device=dev())
    ws = torch.empty(ops.workspace_bytes(d, ops.MOE_OP_LAYER_BWD_CKPT), dtype=torch.uint8, device=dev())
    ops.moe_layer_bwd_ckpt(d, g2.dy.view(1, T, H), w, x.view(1, T, H), b.phi, b.route_row, b.seg_off, q, s, c["W13"], c["W2"], dX, dW13,
                           dW2, dw, ws)
    g1 = ops.alloc_norm_bwd(pre, dev(), post=False, y=False)
    ops.block_norm_bwd(pre, None, c["r"], None, None, c["g1"], st1, g2.dr, dX.view(T, H), g1)
    # the same in 64 bits
    leaf = {k: c[k].double().requires_grad_(True) for k in ("r", "g1", "w", "W13", "W2", "z", "g_post", "g_pre")}
    _, new64, x64 = block64(leaf["r"], leaf["g1"], c["ids"], leaf["w"], leaf["W13"], leaf["W2"], leaf["z"], leaf["g_post"], leaf["g_pre"],
                            0.9, 0.6)
    ((new64 * gr.double()).sum() + (x64 * gx.double()).sum()).backward()
    for name, got in (("r", g1.dr), ("g1", g1.dg_pre), ("w", dw.view(T, K)), ("W13", dW13), ("W2", dW2), ("z", g2.dz),
                      ("g_post", g2.dg_post), ("g_pre", g2.dg_pre)):
        e = rel(got, leaf[name].grad)
        print(f"    d{name}: {e:.2e}", flush=True)
        assert e <= 4e-2, name


def test_two_streams_at_once():
    # the same calls on two streams with buffers of their own
    T, E, K, H, I = 16, 8, 2, 512, 256
    sets = []
    for k in range(2):
        c = setup(T, E, K, H, I, 128)
        c["d"] = ops.make_desc(1, T, K, E, E, H=H, I=I)
        c["routes"], c["x"] = c["ids"].to(torch.int32).reshape(1, T, K).contiguous(), rand((1, T, H), 1.0, 40 + k)
        c["few"], c["stream"] = ops.alloc_few(c["d"], dev(), 128), torch.cuda.Stream()
        ops.layer_fwd_few(c["d"], c["routes"], c["w"], c["x"], c["W13"], c["W2"], c["few"], c["S13"], c["S2"])
        c["want"] = c["few"].out.clone()
        sets.append(c)
    torch.cuda.synchronize()
    for _ in range(20):
        for c in sets:
            ops.layer_fwd_few(c["d"], c["routes"], c["w"], c["x"], c["W13"], c["W2"], c["few"], c["S13"], c["S2"], c["stream"])
    torch.cuda.synchronize()
    assert all(torch.equal(c["few"].out, c["want"]) for c in sets)


def test_few_weights_past_4_gib():
    # the last of 80 experts: its weights start past 4 GiB (bf16), as the only expert of a call they start at 0
    H, I, L = 7168, 2048, 80
    W13 = torch.zeros((L, 2 * I, H), dtype=torch.bfloat16, device=dev())
    W2 = torch.zeros((L, H, I), dtype=torch.bfloat16, device=dev())
    W13[-1], W2[-1] = rand((2 * I, H), 0.02, 1), rand((H, I), 0.02, 2)
    assert W13[-1].data_ptr() - W13.data_ptr() > 1 << 32
    x, w = rand((1, 3, H), 1.0, 3), torch.rand((1, 3, 1), device=dev())
    out = []
    for n, a, b in ((L, W13, W2), (1, W13[-1:], W2[-1:])):
        d = ops.make_desc(1, 3, 1, 384, n, expert_base=300 - n, H=H, I=I)
        f = ops.alloc_few(d, dev())
        ops.layer_fwd_few(d, torch.full((1, 3, 1), 299, dtype=torch.int32, device=dev()), w, x, a, b, f)
        out.append(f.out)
    assert torch.equal(*out) and bool(out[0].any())


def test_norm_rows_past_4_gib():
    rows, H = 270_000, 8192
    r = torch.empty((rows, H), dtype=torch.bfloat16, device=dev())
    r[-1000:] = rand((1000, H), 1.0, 1)
    r[:-1000] = 0.5
    g = 1 + rand((H,), 0.1, 2, torch.float32)
    xn, st = torch.empty_like(r), torch.empty((rows, 2), device=dev())
    ops.moe_block_norm_fwd(ops.make_norm_desc(rows, H), None, r, None, None, g, None, xn, st)
    few, fst = torch.empty((1000, H), dtype=torch.bfloat16, device=dev()), torch.empty((1000, 2), device=dev())
    ops.moe_block_norm_fwd(ops.make_norm_desc(1000, H), None, r[-1000:], None, None, g, None, few, fst)
    assert torch.equal(xn[-1000:], few) and torch.equal(st[-1000:], fst)
    n = ops.make_norm_desc(rows, H)
    b = ops.alloc_norm_bwd(n, dev(), post=False, y=False)
    ops.block_norm_bwd(n, None, r, None, None, g, st, None, xn, b)
    n2 = ops.make_norm_desc(1000, H)
    b2 = ops.alloc_norm_bwd(n2, dev(), post=False, y=False)
    ops.block_norm_bwd(n2, None, r[-1000:], None, None, g, fst, None, few, b2)
    assert torch.equal(b.dr[-1000:], b2.dr)


def test_ckpt_rows_past_4_gib():
    rows, I = 34_000, 32768
    x = torch.zeros((rows, 2 * I), dtype=torch.bfloat16, device=dev())
    x[-64:] = rand((64, 2 * I), 1.0, 1)
    q, s = ops.ckpt_pack(x)
    q2, s2 = ops.ckpt_pack(x[-64:])
    assert torch.equal(q[-64:], q2) and torch.equal(s[-64:], s2)
    dA = torch.zeros((rows, I), dtype=torch.bfloat16, device=dev())
    dA[-64:] = rand((64, I), 1.0, 2)
    A, dw = torch.empty_like(dA), torch.empty(rows, device=dev())
    ops.moe_ckpt_swiglu_bwd(q, s, dA, None, x, A, dw)
    dhu, a, w = torch.empty((64, 2 * I), dtype=torch.bfloat16, device=dev()), torch.empty((64, I), dtype=torch.bfloat16, device=dev()), torch.empty(64, device=dev())
    ops.moe_ckpt_swiglu_bwd(q2, s2, dA[-64:], None, dhu, a, w)
    assert torch.equal(x[-64:], dhu) and torch.equal(A[-64:], a) and torch.equal(dw[-64:], w)

