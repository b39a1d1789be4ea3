"""The layer forward for a few tokens against its definition in 64 bits.

The kernel's error on an output element has three parts, each a rounding or a
32-bit sum (u = 2^-8 is half a bf16 step relative to the value, e = 2^-24):
  - every activation a is rounded once to bf16: at most u |a| each, so at most
    u * sum_r |w_r| sum_i |a_ri| |W2_hi| on the output;
  - a itself comes from 32-bit sums of H products: an error of at most
    H e sum |x W| in the gate and the up value, times the slope of silu(g) u
    (|silu'| <= 1.1, |silu(g)| <= |g|), and the exponential's few e;
  - the output's own rounding: u |out|.
The 32-bit sums' part is bounded by GEN * (the same sum as the rounding's) with
GEN = 2^-11: their worst case H e = 2^-11 at H = 8192 relative to the sums of
magnitudes is far above what random signs give, and the rounding term above is
the larger by 8.
"""
import numpy as np
import pytest
import torch

from routing_schedule_expert_amd import inputs, ops
from tests.helpers import dev

U, GEN = 2.0 ** -8, 2.0 ** -11

pytestmark = pytest.mark.gpu


def rand(shape, std, seed):
    return inputs.normal_bf16_device(shape, std, seed, dev())


def make(P, Np, K, E, L, base, H, I, Is=0, mx=False, seed=1, ids=None):
    rng = np.random.Generator(np.random.PCG64(seed))
    d = ops.make_desc(P, Np, K, E, L, expert_base=base, H=H, I=I)
    if ids is None:
        ids = np.stack([rng.permutation(E)[:K] for _ in range(P * Np)])
    c = dict(d=d, ids=np.asarray(ids, np.int32).reshape(P * Np, K))
    c["routes"] = torch.from_numpy(c["ids"].reshape(P, Np, K).copy()).to(dev())
    c["w"] = torch.from_numpy(rng.random((P, Np, K), dtype=np.float32)).to(dev())
    c["X"] = rand((P, Np, H), 1.0, seed)
    W13, W2 = rand((L, 2 * I, H), 1.5 * H ** -0.5, seed + 1), rand((L, H, I), I ** -0.5, seed + 2)
    c["mx"] = mx
    if mx:
        c["W13"], c["W2"] = ops.quantize_mx(W13), ops.quantize_mx(W2)
    else:
        c["W13"], c["W2"] = W13, W2
    c["S13"] = rand((2 * Is, H), 1.5 * H ** -0.5, seed + 3) if Is else None
    c["S2"] = rand((H, Is), Is ** -0.5, seed + 4) if Is else None
    c["Is"] = Is
    c["bufs"] = ops.alloc_few(d, dev(), Is)
    return c


def call(c, stream=None):
    a = (c["d"], c["routes"], c["w"], c["X"])
    if c["mx"]:
        ops.layer_fwd_few_mx(*a, *c["W13"], *c["W2"], c["bufs"], c["S13"], c["S2"], stream)
    else:
        ops.layer_fwd_few(*a, c["W13"], c["W2"], c["bufs"], c["S13"], c["S2"], stream)
    return c["bufs"].out


def weights(m, e):
    """Expert e's matrix in 64 bits."""
    if not isinstance(m, tuple):
        return m[e].double()
    q, s = m[0][e].view(torch.float8_e4m3fn).double(), m[1][e].double()
    return (q.unflatten(-1, (-1, 32)) * torch.exp2(s - 127).unsqueeze(-1)).flatten(-2)


def expected(c):
    """(output, bound of its error) [tokens][H], in 64 bits."""
    d = c["d"]
    T, H = d.P * d.Np, d.H
    x, w = c["X"].reshape(T, H).double(), c["w"].reshape(T, d.K).double()
    out, mag = torch.zeros((T, H), dtype=torch.float64, device=dev()), torch.zeros((T, H), dtype=torch.float64, device=dev())

    def add(toks, wt, w13, w2):
        n = w13.shape[0] // 2
        hu = x[toks] @ w13.t()
        g, u = hu[:, :n], hu[:, n:]
        a = g * torch.sigmoid(g) * u
        out.index_add_(0, toks, wt * (a @ w2.t()))
        # |a| and, where the gate or up value is a small rest of large terms, what the sums' error makes of it
        size = x[toks].abs() @ w13.t().abs()
        amag = U * a.abs() + GEN * (1.1 * size[:, :n] * u.abs() + size[:, n:] * g.abs())
        mag.index_add_(0, toks, wt.abs() * (amag @ w2.t().abs() + GEN * (a.abs() @ w2.t().abs())))

    for e in range(d.L):
        at = np.argwhere(c["ids"] == e + d.expert_base)
        if len(at):
            t, j = (torch.from_numpy(v.copy()).to(dev()) for v in at.T)
            add(t, w[t, j].unsqueeze(1), weights(c["W13"], e), weights(c["W2"], e))
    if c["Is"]:
        add(torch.arange(T, device=dev()), torch.ones((T, 1), dtype=torch.float64, device=dev()), c["S13"].double(), c["S2"].double())
    return out, mag + U * out.abs()


def check(c, got):
    ref, bound = expected(c)
    err = (got.reshape(ref.shape).double() - ref).abs()
    assert bool((err <= bound).all()), f"worst error {float((err / bound.clamp_min(1e-300)).max()):.3g} of its bound"
    rel = float((got.reshape(ref.shape).double() - ref).norm() / ref.norm().clamp_min(1e-300))
    print(f"    rel-L2 {rel:.2e}", flush=True)
    assert rel <= 4e-3  # two roundings of rms 2^-8 / sqrt(3) at most


CASES = [
    # P, Np, K, E, L, base, H, I, Is, mx
    (1, 1, 1, 1, 1, 0, 256, 128, 0, False),
    (1, 1, 2, 8, 8, 0, 256, 128, 0, True),
    (1, 3, 2, 8, 8, 0, 256, 4096, 128, False),       # over two units a workgroup, the shared expert's before them
    (1, 20, 2, 4, 4, 0, 256, 640, 256, True),        # some experts with 9 to 16 routes, some with up to 8
    (2, 3, 2, 8, 4, 3, 512, 384, 0, False),
    (2, 3, 2, 8, 4, 3, 512, 384, 128, True),
    (1, 17, 4, 16, 16, 0, 256, 128, 256, False),     # one column past a tile
    (1, 33, 3, 9, 5, 2, 768, 640, 0, True),
    (1, 64, 1, 3, 1, 1, 256, 128, 0, False),         # every fourth tile full
    (1, 128, 8, 8, 8, 0, 256, 256, 384, False),      # every expert has every token: two passes
    (1, 128, 8, 8, 8, 0, 256, 256, 384, True),
    (1, 1024, 1, 4, 2, 0, 256, 128, 128, False),     # the most tokens
    (1, 1, 1024, 4096, 4096, 0, 256, 128, 0, False),  # the most slots of one token, the most experts
    (8, 1, 8, 384, 48, 96, 1792, 512, 0, False),
    (8, 2, 8, 384, 48, 336, 1792, 512, 512, True),
]


@pytest.mark.parametrize("case", CASES)
def test_few_matches_definition(case):
    *dims, Is, mx = case
    c = make(*dims, Is=Is, mx=mx)
    check(c, call(c))
    bad = ops.read_ws_words(c["bufs"].ws, 0)[0]
    assert bad == 0


def test_few_dropped_foreign_and_repeated_ids():
    # negative and out-of-range ids are counted and skipped; a token that names one expert twice gets both
    ids = [[0, 5], [-1, 9], [-2 ** 31, 2 ** 31 - 1], [3, 3], [2, 3], [8, 7]]
    c = make(1, 6, 2, 8, 4, 2, 256, 128, ids=ids)
    out = call(c)
    check(c, out)
    assert ops.read_ws_words(c["bufs"].ws, 0)[0] == 5
    assert not out[0, 1].any() and not out[0, 2].any()
    # all 1,024 slots of a call at one expert
    c = make(1, 128, 8, 8, 4, 2, 256, 128, ids=np.full((128, 8), 3))
    check(c, call(c))


@pytest.mark.parametrize("Is", [0, 128])
def test_few_without_local_routes(Is):
    c = make(1, 5, 2, 8, 4, 0, 256, 128, Is=Is, ids=np.full((5, 2), 6))
    out = call(c)
    if Is:
        check(c, out)
    else:
        assert not out.any()


def test_few_nan_stays_with_its_token():
    c = make(1, 19, 2, 4, 4, 0, 256, 128, Is=128)
    clean = call(c).clone()
    c["X"][0, 4, 7] = float("nan")
    c["X"][0, 11, 3] = float("inf")
    c["w"][0, 6, 1] = float("nan")
    out = call(c)
    keep = [t for t in range(19) if t not in (4, 6, 11)]
    assert torch.equal(out[0, keep], clean[0, keep])
    assert bool(out[0, 4].isnan().all()) and bool(out[0, 6].isnan().all())


def test_few_mx_every_code_and_scale():
    # identity-like products: every E4M3 code under scales from the smallest to the largest that leaves them finite
    H, I = 256, 128
    c = make(1, 1, 1, 1, 1, 0, H, I, mx=True)
    codes = torch.arange(256, dtype=torch.uint8, device=dev()).repeat(2 * I, 1)
    codes[(codes & 0x7F) == 0x7F] = 0  # NaN codes
    scales = (118 + torch.arange(2 * I, device=dev()) % 12).to(torch.uint8).unsqueeze(1).repeat(1, H // 32)
    scales[0], scales[I] = 0, 1  # the smallest scales: products far below bf16's normal range vanish in the sums
    c["W13"] = (codes[None].contiguous(), scales[None].contiguous())
    check(c, call(c))


def test_few_mx_nan_codes_and_scales():
    # a NaN code or scale byte anywhere in an expert's weights reaches that expert's tokens and no others
    ids = [[0, 1], [2, 3], [1, 1], [4, 5], [5, 0], [3, 2]]
    c = make(1, 6, 2, 6, 6, 0, 512, 256, mx=True, ids=ids)
    clean = call(c)[0].clone()
    (q13, s13), (q2, s2) = c["W13"], c["W2"]
    for t, spot, v in ((q13, (1, 300, 77), 0x7F), (q2, (3, 9, 200), 0xFF), (s13, (4, 3, 5), 255), (s2, (4, 100, 1), 255)):
        old = int(t[spot])
        t[spot] = v
        out = call(c)[0]
        hit = [i for i, e in enumerate(ids) if spot[0] in e]
        keep = [i for i in range(6) if i not in hit]
        assert torch.equal(out[keep], clean[keep])
        cols = slice(None) if t is q13 or t is s13 else spot[1]  # a row of W2 is one output element
        assert not bool(out[hit][:, cols].isfinite().any())
        t[spot] = old
    assert torch.equal(call(c)[0], clean)


def test_few_repeats_bitwise_and_on_another_stream():
    c = make(2, 13, 3, 12, 6, 3, 512, 256, Is=128)
    first = call(c).clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        c["bufs"].out.fill_(7)
        c["bufs"].ws.fill_(0x5A)
        s.wait_stream(torch.cuda.current_stream())
        call(c, s)
        torch.cuda.current_stream().wait_stream(s)
        assert torch.equal(c["bufs"].out, first)


def test_few_token_does_not_depend_on_the_others():
    # the same token in the same batch shape with other neighbours gives the same bits
    c = make(1, 9, 2, 6, 6, 0, 512, 256)
    a = call(c)[0, 4].clone()
    c["X"][0, :4] *= -3
    c["X"][0, 5:] += 1
    assert torch.equal(call(c)[0, 4], a)


def test_few_captured_and_replayed():
    c = make(1, 7, 3, 8, 8, 0, 512, 256, Is=128)
    call(c)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(c)
    for seed in range(4):
        c["X"].copy_(rand(c["X"].shape, 1.0, 50 + seed))
        c["routes"].copy_(torch.rand((7, 8), device=dev()).argsort(1)[:, :3].reshape(1, 7, 3).to(torch.int32))
        c["ids"] = c["routes"].cpu().numpy().reshape(7, 3)
        g.replay()
        torch.cuda.synchronize()
        got = c["bufs"].out.clone()
        check(c, got)
        assert torch.equal(call(c), got)


def test_few_agrees_with_the_layer_forward():
    # same inputs through the grouped GEMMs: one more bf16 rounding there (each expert's row)
    c = make(1, 100, 4, 8, 8, 0, 512, 256)
    got = call(c)
    b = ops.alloc_fwd(c["d"], dev(), save_xd=False)
    ops.layer_fwd(c["d"], c["routes"], c["w"], c["X"], c["W13"], c["W2"], b)
    assert float((got.double() - b.out.double()).norm() / b.out.double().norm()) <= 6e-3


def test_few_binding_refuses_wrong_buffers():
    c = make(1, 2, 2, 4, 4, 0, 256, 128)
    b, d = c["bufs"], c["d"]
    with pytest.raises(ValueError):
        ops.moe_layer_fwd_few(d, 0, c["routes"].long(), c["w"], c["X"], c["W13"], c["W2"], None, None, b.out, b.ws)
    with pytest.raises(ValueError):
        ops.moe_layer_fwd_few(d, 0, c["routes"], c["w"], c["X"], c["W13"][:3].contiguous(), c["W2"], None, None, b.out, b.ws)
    with pytest.raises(ops.MoeError):
        ops.moe_layer_fwd_few(d, 0, c["routes"], c["w"], c["X"], c["W13"], c["W2"], None, None, b.out, b.ws[:64])


@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("H", [2048, 7168])
@pytest.mark.parametrize("K,local,Is", [(1, 1, 0), (2, 1, 0), (2, 2, 0), (4, 3, 0), (1, 1, 2048), (4, 4, 2048), (6, 1, 0), (8, 8, 2048)])
def test_few_one_token_in_parts(K, local, Is, H, mx):
    # the smallest calls: few experts, so the waves of a down workgroup take parts of their rows
    ids = [[3 - 2 * j if j < local and j < 2 else 2 + j % 2 if j < local else 9 for j in range(K)]]
    c = make(1, 1, K, 10, 3, 1, H, 2048, Is, mx, ids=ids, seed=K + local)
    check(c, call(c))


def spread(counts, T, K):
    """Routes of T tokens with K slots, counts[e] of them to expert e and the others nowhere, in no order."""
    flat = np.full(T * K, -1, np.int32)
    flat[:sum(counts)] = np.repeat(np.arange(len(counts)), counts)
    return np.random.Generator(np.random.PCG64(sum(counts))).permutation(flat).reshape(T, K)


# T, K, the experts' routes, H, I, Is.  The four waves of a down workgroup of 16 output columns (H >= 4096 on 256 CUs),
# or eight at 8 columns, are parts of an expert's rows times groups of experts; the parts' sums meet in rounds, as many
# places at a time as there is LDS for.  Experts with up to 8, 16, 32, 64 routes and more, alone and together:
DOWN = [
    (7, 2, [7, 4], 4096, 1024, 0),               # four parts of bf16, two of MXFP8
    (12, 2, [12, 9], 4096, 2048, 512),           # four parts of both, two of the shared expert
    (24, 2, [24, 20], 4096, 1024, 0),
    (50, 2, [50, 41], 7168, 2048, 2048),
    (70, 2, [70, 69], 4096, 1024, 512),
    (64, 2, [40, 30, 15, 11, 6, 1], 4096, 1024, 0),
    (20, 8, [24, 20, 20, 20, 20, 17, 9, 3], 4096, 1024, 0),   # two parts
    (12, 16, [12, 12, 12, 20, 1, 8, 9, 7, 16, 17, 2, 3, 33, 4, 5, 6], 4096, 512, 512),  # whole rows
    (100, 2, [100, 90], 4096, 1024, 512),        # two rounds, the second expert in both
    (128, 8, [500, 300, 200, 13, 4], 4096, 1024, 0),          # 49 places a round
    (300, 1, [140, 100, 30, 12, 6], 4096, 1024, 1024),        # three rounds, the shared expert's tokens too
    (300, 1, [140, 100, 30, 12, 6], 512, 4096, 2048),         # eight waves, eight parts, three rounds
    (128, 8, [500, 300, 200, 13, 4], 256, 2048, 2048),
    (33, 3, [33, 9, 17, 1], 512, 4096, 128),
    (1024, 1, [600, 424], 4096, 1024, 2048),     # no room for parts
    (1024, 1, [600, 400], 256, 2048, 2048),      # 20 rounds
]


@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("T,K,counts,H,I,Is", DOWN)
def test_few_down_tiles_parts_and_rounds(T, K, counts, H, I, Is, mx):
    c = make(1, T, K, len(counts), len(counts), 0, H, I, Is, mx, ids=spread(counts, T, K), seed=T)
    out = call(c).clone()
    check(c, out)
    assert torch.equal(call(c), out)
