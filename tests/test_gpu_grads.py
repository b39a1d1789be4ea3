"""The norm of many gradients and their clipping against 64 bits.

The squares are summed in 64 bits, so norm and coef are off by half a step of fp32
and what sums of 2^24 terms lose in 64 bits, nothing that shows: 2^-23 in all.  A
scaled gradient takes two more roundings of 32 bits (scale coef, the product) and
one to its type.
"""
import math

import pytest
import torch

from routing_schedule_expert_amd import ops
from tests.helpers import dev

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: U}
KINDS = {"l2": ops.MOE_NORM_L2, "max": ops.MOE_NORM_MAX}
DT = (torch.float32, torch.bfloat16, torch.float16)


def rand(n, dtype, seed, std=0.05):
    g = torch.Generator(device=dev())
    g.manual_seed(seed)
    return (torch.randn(n, generator=g, device=dev()) * std).to(dtype)


def norm64(grads, kind, scale=1.0):
    if kind == "max":
        return abs(scale) * max([float(t.double().abs().max()) for t in grads if t.numel()], default=0.0)
    return abs(scale) * math.sqrt(sum(float(t.double().square().sum()) for t in grads))


def check(grads, kind="l2", max_norm=1.0, scale=1.0, eps=1e-6, out=None):
    before = [t.clone() for t in grads]
    gl = ops.make_grad_list(grads, out, dev())
    want = norm64(before, kind, scale)
    for call in (ops.grad_norm, ops.grad_clip):
        gl.result.fill_(255)
        call(gl, max_norm, KINDS[kind], scale, eps)
        norm, coef = float(gl.norm), float(gl.coef)
        # past fp32's largest number, 3.4e38, its nearest value is infinity; coef, below its normal range, is off by
        # up to a step of 2^-149 there
        assert (abs(norm - want) <= 2 * U * want if want < 3.4e38 else math.isinf(norm)) and abs(float(gl.sum) - (want if kind == "max" else want ** 2)) <= 1e-12 * want ** 2 + 1e-12 * want
        c = min(1.0, max_norm / (want + eps))
        assert abs(coef - c) <= 2 * U * c + 2.0 ** -149
    f = float(torch.tensor(scale, dtype=torch.float32)) * coef
    for b, o in zip(before, gl.out):
        ref = b.double() * f
        assert bool(((o.double() - ref).abs() <= HALF[o.dtype] * ref.abs() * (1 + 4 * U) + 3 * U * ref.abs() + (2.0 ** -25 if o.dtype == torch.float16 else 1e-44)).all())
    if out is not None:
        assert all(torch.equal(a, b) for a, b in zip(grads, before))
    return gl


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("inside", [True, False])
def test_sizes_and_types(kind, inside):
    sizes = [1, 0, 3, 8, 127, 16384, 16385, 5, 100_000, 0, 70_001]
    grads = [rand(n, DT[(i + j) % 3], 10 * i + j) for i, n in enumerate(sizes) for j in range(3)]
    check(grads, kind, 0.3, out=None if inside else [torch.empty_like(t) for t in grads])


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("n", [1, 2, 7, 8, 9, 1000, 16383, 16384, 16391, 40_000])
def test_starts(dtype, n):
    # a tensor that starts and ends inside a 16-byte word, its neighbours left as they were
    for a in (0, 1, 3, 5):
        flat = rand(n + 32, dtype, n + a)
        o = torch.full_like(flat, 9.0)
        for b in (a, (a + 1) % 8):
            o.fill_(9)
            keep = flat.clone()
            check([flat[8 + a:8 + a + n]], max_norm=0.01, out=[o[8 + b:8 + b + n]])
            assert torch.equal(flat, keep) and bool((o[:8 + b] == 9).all()) and bool((o[8 + b + n:] == 9).all())
        keep = flat.clone()
        check([flat[8 + a:8 + a + n]], max_norm=0.01)
        assert torch.equal(flat[:8 + a], keep[:8 + a]) and torch.equal(flat[8 + a + n:], keep[8 + a + n:])


def test_neighbours_in_one_word():
    # tensors that share 16-byte words, clipped where they lie
    flat = rand(1000, torch.bfloat16, 3)
    keep, cuts = flat.clone(), [3, 10, 11, 4, 1, 1, 1, 200, 300, 469]
    gl = check(list(flat.split(cuts)), max_norm=0.5)
    f = torch.tensor(float(gl.coef), device=dev())
    assert torch.equal(flat, (keep.float() * f).bfloat16())


@pytest.mark.parametrize("count", [0, 1, 127, 128, 129, 177, 192, 247, 248, 249, 400, 641])
def test_many_tensors(count):
    grads = [rand(1 + (37 * i) % 3000, DT[i % 3], i) for i in range(count)]
    check(grads, "l2", 0.7)
    check(grads, "max", 0.01)


def test_scale_and_bounds():
    grads = [rand(5000, torch.float32, 1), rand(333, torch.bfloat16, 2)]
    for scale in (1 / 1024, -0.5, 3.0):
        check([t.clone() for t in grads], "l2", 0.1, scale)
        check([t.clone() for t in grads], "max", 0.1, scale)
    check([t.clone() for t in grads], max_norm=0.0)
    check([t.clone() for t in grads], max_norm=float("inf"))
    same = [t.clone() for t in grads]
    gl = check(same, max_norm=1e6)
    assert float(gl.coef) == 1.0 and all(torch.equal(a, b) for a, b in zip(same, grads))
    zeros = [torch.zeros(100, device=dev())]
    assert float(check(zeros).norm) == 0.0
    gl = ops.grad_clip(ops.make_grad_list(zeros), 0.0, eps=0.0)
    assert float(gl.norm) == 0.0 and float(gl.coef) == 1.0 and not bool(zeros[0].any())


def test_values_whose_squares_leave_fp32():
    for v in (1e25, 1e-30, 3e38):
        check([torch.full((3000,), v, device=dev())], "l2", 1.0, eps=0.0)


def test_bad_values():
    base = [rand(50_000, torch.float32, 1), rand(4001, torch.bfloat16, 2)]
    for kind in KINDS:
        for where in (0, 1):
            grads = [t.clone() for t in base]
            grads[where][1234] = float("nan")
            gl = ops.grad_clip(ops.make_grad_list(grads), 1.0, KINDS[kind])
            assert math.isnan(float(gl.norm)) and math.isnan(float(gl.coef)) and all(bool(t.isnan().all()) for t in grads)
            grads = [t.clone() for t in base]
            grads[where][1234] = -float("inf")
            gl = ops.grad_clip(ops.make_grad_list(grads), 1.0, KINDS[kind])
            assert math.isinf(float(gl.norm)) and float(gl.coef) == 0.0
            for i, t in enumerate(grads):
                bad = t.isnan()
                assert bool((t[~bad] == 0).all()) and int(bad.sum()) == (i == where)


def test_ranks_that_hold_shards():
    # two shards' sums added, and the coefficient of all of them
    shards = [[rand(9000, torch.float32, k), rand(801, torch.bfloat16, 5 + k)] for k in range(2)]
    want = norm64(shards[0] + shards[1], "l2")
    lists = [ops.make_grad_list(s, [torch.empty_like(t) for t in s]) for s in shards]
    for gl in lists:
        ops.grad_norm(gl)
    norm = (lists[0].sum + lists[1].sum).sqrt()
    coef = (0.25 / (norm + 1e-6)).clamp(max=1.0).float()
    assert abs(float(norm) - want) <= 1e-12 * want
    for gl, s in zip(lists, shards):
        ops.grad_scale(gl, coef, 2.0)
        for g, o in zip(s, gl.out):
            ref = g.double() * (2.0 * float(coef))
            assert bool(((o.double() - ref).abs() <= HALF[o.dtype] * ref.abs() * 1.0001 + 3 * U * ref.abs()).all())


def test_large_and_past_4_gib():
    n = (1 << 31) + 12345  # bf16: past 4 GiB and past 2^31 elements
    t = torch.zeros(n, dtype=torch.bfloat16, device=dev())
    t[-3:], t[0] = 2.0, 4.0
    gl = ops.grad_clip(ops.make_grad_list([t]), 1.0)
    assert float(gl.norm) == float(torch.tensor(28.0).sqrt())
    f = float(gl.coef)
    assert float(t[-1]) == float(torch.tensor(2.0 * f).bfloat16()) and float(t[0]) == float(torch.tensor(4.0 * f).bfloat16()) and float(t[5]) == 0


def test_repeats_streams_and_graphs():
    grads = [rand(n, DT[i % 3], i) for i, n in enumerate((100_000, 7, 50_001, 3000))]
    lists = [ops.make_grad_list(grads, [torch.empty_like(t) for t in grads]) for _ in range(2)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    ops.grad_clip(lists[0], 0.5)
    ref = [t.clone() for t in lists[0].out + [lists[0].result]]
    torch.cuda.synchronize()
    for _ in range(10):
        for gl, s in zip(lists, streams):
            ops.grad_clip(gl, 0.5, stream=s)
    torch.cuda.synchronize()
    for gl in lists:
        assert all(torch.equal(a, b) for a, b in zip(ref, gl.out + [gl.result]))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ops.grad_clip(lists[0], 0.5)
    for k in range(3):
        for i, t in enumerate(grads):
            t.copy_(rand(t.numel(), t.dtype, 100 * k + i))
        graph.replay()
        ops.grad_clip(lists[1], 0.5)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(lists[0].out + [lists[0].result], lists[1].out + [lists[1].result]))


def test_lists_that_do_not_fit():
    t = rand(100, torch.float32, 1)
    for bad in ([t.cpu()], [t.double()], [t.view(10, 10).t()]):
        with pytest.raises((ValueError, TypeError)):
            ops.make_grad_list(bad)
    for bad in ([t, t], [t, t[50:]], [t[:51], t[50:]]):
        with pytest.raises(ValueError):
            ops.make_grad_list(bad)
    with pytest.raises(ValueError):
        ops.make_grad_list([t[:50], t[50:]], [t[50:], torch.empty_like(t[:50])])
    ops.make_grad_list([t[:50], t[50:50], t[50:]])
    for out in ([], [t[:50]], [t.bfloat16()]):
        with pytest.raises((ValueError, TypeError)):
            ops.make_grad_list([t], out)
    for kw in (dict(max_norm=-1.0), dict(max_norm=float("nan")), dict(max_norm=1.0, eps=-1.0), dict(max_norm=1.0, kind=2), dict(max_norm=1.0, scale=float("nan"))):
        with pytest.raises(ops.MoeError):
            ops.grad_clip(ops.make_grad_list([t]), **kw)


@pytest.mark.parametrize("count", [160, 161, 385])
def test_many_tensors_elsewhere(count):
    grads = [rand(1 + (37 * i) % 3000, DT[i % 3], i) for i in range(count)]
    keep, out = [t.clone() for t in grads], [torch.empty_like(t) for t in grads]
    gl = ops.grad_clip(ops.make_grad_list(grads, out), 0.7)
    f = gl.coef.clone()
    for g, k, o in zip(grads, keep, out):
        assert torch.equal(g, k) and torch.equal(o, (k.float() * f).to(k.dtype))


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("kind", list(KINDS))
def test_the_sum_does_not_depend_on_where_gradients_lie(dtype, kind):
    # the same values at every start of a 16-byte word: one order of additions, so the same bits
    for n in (1, 5, 9, 2047, 2049, 16_384, 70_003, 6_000_011):
        values, want = rand(n, dtype, n, 1.0), None
        for start in range(8):
            flat = torch.empty(n + 8, dtype=dtype, device=dev())
            flat[start:start + n] = values
            got = ops.grad_norm(ops.make_grad_list([flat[start:start + n]]), 1.0, KINDS[kind]).result.clone()
            want = got if want is None else want
            assert torch.equal(got, want), (n, start)


def test_a_new_list_on_another_stream():
    # a list made while its own stream is busy, and a call at once on another
    grads, side = [rand(100_000, torch.float32, 1), rand(333, torch.bfloat16, 2)], torch.cuda.Stream()
    want = norm64(grads, "l2")
    torch.cuda.synchronize()
    torch.cuda._sleep(100_000_000)
    gl = ops.grad_norm(ops.make_grad_list(grads), stream=side)
    torch.cuda.synchronize()
    assert abs(float(gl.norm) - want) <= 2 * U * want


def test_no_gradients_of_the_current_device():
    gl = ops.grad_clip(ops.make_grad_list([], device="cuda"), 1.0)
    assert gl.result.device == torch.device("cuda", torch.cuda.current_device()) and float(gl.norm) == 0.0 and float(gl.coef) == 1.0


def test_an_infinite_gradient_without_a_bound():
    for kind in KINDS:
        t = rand(5000, torch.float32, 1)
        t[77] = float("inf")
        gl = ops.grad_clip(ops.make_grad_list([t]), float("inf"), KINDS[kind])
        assert math.isinf(float(gl.norm)) and float(gl.coef) == 0.0
        assert bool(t[77].isnan()) and not bool(t[:77].any()) and not bool(t[78:].any())


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("inside", [True, False])
def test_more_slots_than_one_launch(kind, inside):
    # 300 tensors of 16 to 20 pieces: two launches of 2048 and hundreds of slots, which a launch of its own adds
    grads = [rand(260_001 + 211 * i, DT[i % 3], i) for i in range(300)]
    check(grads, kind, 0.3, out=None if inside else [torch.empty_like(t) for t in grads])
