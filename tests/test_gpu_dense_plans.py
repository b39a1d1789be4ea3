"""The gated feed-forward block at shapes that reach every tile of its products,
whole and cut along K, against the formulas in 64 bits (the bounds are those of
test_gpu_ffn.py).

Behind each shape stands what is chosen for it: the tile (256 x 256, 128 x 128 with
two workgroups a CU, 128 x 128 alone, 64 x 128) and, where a product is cut, the
parts.  Parts take workspace, which the tests compare; of the tiles there is no
outward sign.
"""
import pytest
import torch

from routing_schedule_expert_amd import ops
from tests.helpers import dev
from tests.test_gpu_ffn import ACTS, backward64, forward64, fwd, kept, make, near

pytestmark = pytest.mark.gpu


def parts(splits, M, N):
    return -(-splits * M * N * 4 // 256) * 256 if splits > 1 else 0


# rows, H, I; parts of the gate / up product and of the down product
FORWARD = [
    (65, 392, 8, 1, 1),  # gate / up 64 x 128, down 128 x 128 (two)
    (65, 1288, 8, 6, 1),  # gate / up 128 x 128 (two), down 128 x 128 (two)
    (70, 2048, 8, 8, 1),  # gate / up 128 x 128 (two), down 128 x 128 (two)
    (65, 7176, 8, 15, 1),  # gate / up 64 x 128, down 128 x 128 (two)
    (128, 7168, 2048, 4, 1),  # gate / up 64 x 128, down 64 x 128
    (129, 7168, 2056, 2, 1),  # gate / up 64 x 128, down 64 x 128
    (5000, 7176, 8, 4, 1),  # gate / up 128 x 128 (alone), down 256 x 256
    (1021, 2056, 1032, 1, 1),  # gate / up 128 x 128 (alone), down 128 x 128 (two)
    (8200, 2056, 72, 1, 1),  # gate / up 128 x 128 (alone), down 128 x 128 (two)
    (5000, 8, 776, 1, 1),  # gate / up 256 x 256, down 64 x 128
    (2500, 1032, 5128, 1, 1),  # gate / up 256 x 256, down 128 x 128 (alone)
    (65, 8, 1288, 1, 6),  # gate / up 128 x 128 (two), down 128 x 128 (two)
    (65, 8, 7176, 1, 15),  # gate / up 128 x 128 (two), down 64 x 128
    (256, 4096, 4096, 1, 2),  # gate / up 64 x 128, down 64 x 128
    (5000, 8, 7176, 1, 4),  # gate / up 256 x 256, down 128 x 128 (alone)
    (8200, 136, 2056, 1, 1),  # gate / up 128 x 128 (two), down 128 x 128 (alone)
    (5000, 1544, 8, 1, 1),  # gate / up 64 x 128, down 256 x 256
    (2000, 7176, 2056, 1, 1),  # gate / up 128 x 128 (alone), down 256 x 256
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("rows,H,I,up,down", FORWARD)
def test_forward(rows, H, I, up, down, dtype):
    c = make(rows, H, I, list(ACTS)[(rows + I) % 4], dtype)
    assert ops.gated_ffn_workspace_bytes(c["n"]) == max(parts(up, rows, 2 * I), parts(down, rows, H))
    b = fwd(c)
    (out, hu, a), (eout, ehu, ea) = forward64(c)
    near("HU", b.HU, hu, ehu)
    near("A", b.A, a, ea)
    near("out", b.out, out, eout)
    plain = fwd(c, save=False)
    assert torch.equal(plain.out, b.out) and torch.equal(plain.A, b.A)


@pytest.mark.parametrize("rows,H,I", [(70, 2048, 8), (128, 2056, 72)])
def test_cut_rows_behind_the_last_stay(rows, H, I):
    c = make(rows, H, I, ldx=H + 24, ldo=H + 40)
    assert ops.gated_ffn_workspace_bytes(c["n"]) > 0
    even = dict(c, n=ops.make_ffn_desc(rows, H, I), X=c["X"].contiguous())
    want = fwd(even)
    big = {k: torch.full((rows + 300, w), 5.0, dtype=torch.bfloat16, device=dev()) for k, w in (("out", H + 40), ("HU", 2 * I), ("A", I))}
    ws = torch.empty(ops.gated_ffn_workspace_bytes(c["n"]), dtype=torch.uint8, device=dev())
    ops.moe_gated_ffn_fwd(c["n"], c["X"], c["W13"], c["W2"], big["HU"], big["A"], big["out"][:, :H], ws)
    assert torch.equal(big["out"][:rows, :H], want.out) and bool((big["out"][:, H:] == 5).all())
    assert torch.equal(big["HU"][:rows], want.HU) and torch.equal(big["A"][:rows], want.A)
    for t in big.values():
        assert bool((t[rows:] == 5).all())


# rows, H, I; parts of the activations' product, of the gradients of W13, of W2 and of X
BACKWARD = [
    (1, 392, 8, 1, 1, 1, 1),  # activations 64 x 128, gradients 64 x 128
    (1, 7176, 8, 15, 1, 1, 1),  # activations 64 x 128, gradients 64 x 128
    (65, 1288, 8, 6, 1, 1, 1),  # activations 128 x 128 (two), gradients 64 x 128
    (5000, 7176, 8, 4, 4, 4, 1),  # activations 128 x 128 (alone), gradients 128 x 128 (two)
    (8200, 2056, 136, 1, 1, 1, 1),  # activations 128 x 128 (alone), gradients 128 x 128 (alone)
    (5000, 8, 1544, 1, 1, 1, 1),  # activations 256 x 256, gradients 64 x 128
    (2500, 1032, 5128, 1, 1, 1, 1),  # activations 256 x 256, gradients 128 x 128 (two)
    (1, 1288, 520, 6, 1, 1, 1),  # activations 128 x 128 (two), gradients 64 x 128
    (1, 520, 1288, 1, 1, 1, 11),  # activations 64 x 128, gradients 128 x 128 (alone)
    (1, 776, 1544, 1, 1, 1, 13),  # activations 64 x 128, gradients 128 x 128 (two)
    (2500, 520, 8, 1, 10, 10, 1),  # activations 64 x 128, gradients 128 x 128 (alone)
    (5000, 8, 200, 1, 16, 16, 2),  # activations 128 x 128 (two), gradients 128 x 128 (alone)
    (4096, 520, 8, 1, 16, 16, 1),  # activations 64 x 128, gradients 128 x 128 (two)
    (777, 8, 2056, 1, 4, 4, 13),  # activations 128 x 128 (two), gradients 128 x 128 (two)
    (257, 8, 1544, 1, 2, 2, 13),  # activations 128 x 128 (two), gradients 64 x 128
    (2500, 8, 8, 1, 10, 10, 1),  # activations 128 x 128 (two), gradients 64 x 128
    (128, 7168, 2048, 8, 1, 1, 4),  # activations 64 x 128, gradients 128 x 128 (two)
    (1021, 7176, 2056, 1, 1, 1, 1),  # activations 128 x 128 (alone), gradients 256 x 256
    (2000, 4104, 1288, 1, 1, 1, 1),  # activations 128 x 128 (alone), gradients 256 x 256
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("rows,H,I,act,w13,w2,x", BACKWARD)
def test_backward(rows, H, I, act, w13, w2, x, dtype):
    given = dtype == torch.float16
    c = make(rows, H, I, list(ACTS)[(rows + I) % 4], dtype)
    base = sum(-(-b // 256) * 256 for b in (4 * rows * I, 2 * rows * I))
    assert ops.gated_ffn_workspace_bytes(c["n"], True) == base + max(
        parts(act, rows, I), parts(w13, 2 * I, H) + parts(w2, H, I) + parts(x, rows, H))
    HU, A = kept(c)
    b = ops.alloc_gated_ffn_bwd(c["n"], dev(), dw_dtype=torch.float32 if (rows + given) % 2 else dtype)
    for t in (b.dX, b.dW13, b.dW2):
        t.fill_(7)
    ops.gated_ffn_bwd(c["n"], c["dOut"], c["X"], HU, A if given else None, c["W13"], c["W2"], b)
    for name, got, (ref, err) in zip(("dX", "dW13", "dW2"), (b.dX, b.dW13, b.dW2), backward64(c, HU, A, given)):
        near(name, got, ref, err)


@pytest.mark.parametrize("rows,H,I", [(1021, 7176, 2056), (128, 7168, 2048)])
def test_a_bad_row_stays_alone(rows, H, I):
    # X's gradient in 256 x 256 tiles, and cut
    c = make(rows, H, I)
    HU, A = kept(c)
    g, gb = (ops.alloc_gated_ffn_bwd(c["n"], dev(), dw=False) for _ in range(2))
    ops.gated_ffn_bwd(c["n"], c["dOut"], c["X"], HU, A, c["W13"], c["W2"], g)
    d, r = c["dOut"].clone(), rows - 30
    d[r, 3] = float("nan")
    ops.gated_ffn_bwd(c["n"], d, c["X"], HU, A, c["W13"], c["W2"], gb)
    rest = torch.arange(rows, device=dev()) != r
    assert bool(gb.dX[r].isnan().all()) and torch.equal(gb.dX[rest], g.dX[rest])
