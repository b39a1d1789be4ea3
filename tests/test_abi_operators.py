"""Host-side checks of the few-token layer, the block norms and the 8-bit
checkpoints (no GPU needed): sizes, and refusals before anything is launched."""
import ctypes

import pytest

from routing_schedule_expert_amd import ops


def _fake(addr):
    # aligned, non-NULL addresses that no call below dereferences: each fails its host-side checks
    return ctypes.c_void_p(addr)


P = [_fake(0x10000 * (i + 1)) for i in range(20)]
BAD = _fake(0x10008)


def few_desc(**kw):
    v = dict(P=8, Np=16, K=8, E=384, L=48, H=7168, I=2048) | kw
    return ops.make_desc(v.pop("P"), v.pop("Np"), v.pop("K"), v.pop("E"), v.pop("L"), **v)


def test_few_workspace():
    d = few_desc()
    plain, shared = ops.few_workspace_bytes(d), ops.few_workspace_bytes(d, 2048)
    assert 1024 * 2048 * 2 < plain < 1024 * 2048 * 2 + (64 << 10)
    assert shared - plain == 128 * 2048 * 2
    assert ops.few_workspace_bytes(d, 4096) - plain == 1152 * 4096 * 2 - 1024 * 2048 * 2
    for bad in (few_desc(Np=17), few_desc(H=7000), few_desc(I=100), few_desc(num_batches=2), few_desc(Np=0)):
        assert ops.load().moe_few_workspace_bytes(ctypes.byref(bad), 0) == -1
    for Is in (-1, 64, 1 << 30):
        assert ops.load().moe_few_workspace_bytes(ctypes.byref(d), Is) == -1
    with pytest.raises(ops.MoeError):
        ops.few_workspace_bytes(few_desc(Np=1000))


def test_few_refusals():
    lib, d = ops.load(), few_desc()
    ws = ops.few_workspace_bytes(d, 2048)
    ref = ctypes.byref(d)
    fwd, mx = lib.moe_layer_fwd_few, lib.moe_layer_fwd_few_mx
    assert fwd(None, 0, *P[:5], None, None, P[5], P[6], ws, None) == ops.MOE_EINVAL
    for i in (0, 1, 2, 3, 4, 7, 8):  # without a shared expert the two weights of it are NULL
        a = [P[0], P[1], P[2], P[3], P[4], None, None, P[5], P[6]]
        a[i] = None
        assert fwd(ref, 0, *a, ws, None) == ops.MOE_EINVAL
        a[i] = BAD
        assert fwd(ref, 0, *a, ws, None) == ops.MOE_EINVAL
    assert fwd(ref, 0, *P[:5], P[5], P[6], P[7], P[8], ws, None) == ops.MOE_EINVAL
    assert fwd(ref, 2048, *P[:5], P[5], None, P[7], P[8], ws, None) == ops.MOE_EINVAL
    assert fwd(ref, 2048, *P[:5], BAD, P[6], P[7], P[8], ws, None) == ops.MOE_EINVAL
    assert fwd(ref, 2048, *P[:9], ws - 1, None) == ops.MOE_ENOSPC
    assert fwd(ref, 100, *P[:9], ws, None) == ops.MOE_EUNSUPPORTED
    assert fwd(ref, -128, *P[:9], ws, None) == ops.MOE_EINVAL
    many = few_desc(Np=17)  # 1,088 slots
    assert fwd(ctypes.byref(many), 2048, *P[:9], 1 << 40, None) == ops.MOE_EUNSUPPORTED
    odd = few_desc(H=7168 + 64)
    assert fwd(ctypes.byref(odd), 2048, *P[:9], 1 << 40, None) == ops.MOE_EUNSUPPORTED
    for i in (0, 1, 2, 3, 4, 5, 6, 9, 10):
        a = [P[j] for j in range(7)] + [None, None, P[7], P[8]]
        a[i] = None
        assert mx(ref, 0, *a, ws, None) == ops.MOE_EINVAL
    a = [P[0], P[1], P[2], P[3], _fake(0x10002), P[5], P[6], None, None, P[7], P[8]]
    assert mx(ref, 0, *a, ws, None) == ops.MOE_EINVAL  # scale bytes are 4-byte aligned
    assert mx(ref, 2048, *P[:11], ws - 1, None) == ops.MOE_ENOSPC
