"""Host-side checks of the gated feed-forward block, layer norm and the clipping
of gradients (no GPU needed): sizes, and refusals before anything is launched."""
import ctypes

import pytest
import torch

from routing_schedule_expert_amd import ops


def _fake(addr):
    # aligned, non-NULL addresses that no call below dereferences: each fails its host-side checks
    return ctypes.c_void_p(addr)


P = [_fake(0x10000 * (i + 1)) for i in range(20)]
BAD = _fake(0x10008)
ODD = _fake(0x10001)
EINVAL, ENOSPC, EUNSUP = ops.MOE_EINVAL, ops.MOE_ENOSPC, ops.MOE_EUNSUPPORTED


def ffn(**kw):
    v = dict(rows=100, H=264, I=136) | kw
    return ops.make_ffn_desc(v.pop("rows"), v.pop("H"), v.pop("I"), **v)


def test_ffn_sizes():
    lib = ops.load()
    assert ops.gated_ffn_workspace_bytes(ffn(rows=0)) == ops.gated_ffn_workspace_bytes(ffn(rows=0), True) == 0
    assert ops.gated_ffn_workspace_bytes(ffn(rows=16384, H=7168, I=2048)) == 0  # tiles for every CU: no parts
    assert ops.gated_ffn_workspace_bytes(ffn(rows=16384, H=7168, I=2048), True) == 16384 * 6 * 2048
    assert ops.gated_ffn_workspace_bytes(ffn(rows=100), True) >= 100 * 6 * 136
    bad = [ffn(rows=-1), ffn(H=0), ffn(I=0), ffn(act=4), ffn(act=-1), ffn(H=260), ffn(I=132), ffn(H=65544), ffn(I=65544), ffn(ldx=256), ffn(ldo=8),
           ffn(ldx=268), ffn(ldo=-8), ffn(ldx=(1 << 20) + 8), ffn(H=32768, I=32768), ffn(rows=1 << 30), ffn(rows=1 << 25, H=2048), ffn(rows=1 << 25, I=1024),
           ffn(dtype=torch.float32)]
    for n in bad:
        assert lib.moe_gated_ffn_workspace_bytes(ctypes.byref(n), 0) == lib.moe_gated_ffn_workspace_bytes(ctypes.byref(n), 1) == -1
    assert lib.moe_gated_ffn_workspace_bytes(ctypes.byref(ffn()), 2) == -1
    assert lib.moe_gated_ffn_workspace_bytes(None, 0) == -1
    with pytest.raises(ops.MoeError):
        ops.gated_ffn_workspace_bytes(ffn(H=260))
    with pytest.raises(ValueError):
        ffn(dtype=torch.float64)


def test_ffn_refusals():
    lib = ops.load()
    names = ("X", "W13", "W2", "HU", "A", "out", "ws")

    def fwd(n, ws_bytes=1 << 40, **kw):
        a = dict(zip(names, P)) | kw
        return lib.moe_gated_ffn_fwd(ctypes.byref(n), *(a[k] for k in names), ws_bytes, None)

    assert lib.moe_gated_ffn_fwd(None, *P[:7], 1 << 40, None) == EINVAL
    assert lib.moe_gated_ffn_fwd(ctypes.byref(ffn(rows=0)), *([None] * 7), 0, None) == ops.MOE_OK
    for k in ("X", "W13", "W2", "A", "out"):
        assert fwd(ffn(), **{k: None}) == EINVAL, k
    for k in names:
        assert fwd(ffn(), **{k: BAD}) == EINVAL, k
    small = ffn(rows=70, H=2048, I=8)  # few tiles: cut along K
    need = ops.gated_ffn_workspace_bytes(small)
    assert need > 0 and fwd(small, need - 1) == ENOSPC and fwd(small, ws=None) == EINVAL
    for n, code in ((ffn(H=260), EUNSUP), (ffn(I=12), EUNSUP), (ffn(act=9), EINVAL), (ffn(ldx=12), EINVAL), (ffn(ldx=268), EUNSUP),
                    (ffn(rows=1 << 31), EUNSUP), (ffn(dtype=torch.float32), EINVAL)):
        assert fwd(n) == code

    names2 = ("dOut", "X", "HU", "A", "W13", "W2", "dX", "dW13", "dW2")

    def bwd(n, dw=ops.MOE_TYPE_FP32, add=0, ws=P[10], ws_bytes=1 << 40, **kw):
        a = dict(zip(names2, P)) | kw
        return lib.moe_gated_ffn_bwd(ctypes.byref(n), *(a[k] for k in names2), dw, add, ws, ws_bytes, None)

    for k in ("dOut", "X", "HU", "W13", "W2"):
        assert bwd(ffn(), **{k: None}) == EINVAL, k
    for k in names2:
        assert bwd(ffn(), **{k: BAD}) == EINVAL, k
    assert bwd(ffn(), ws=None) == bwd(ffn(), ws=BAD) == EINVAL
    assert bwd(ffn(), ws_bytes=ops.gated_ffn_workspace_bytes(ffn(), True) - 1) == ENOSPC
    assert bwd(ffn(), dX=None, dW13=None, dW2=None) == EINVAL
    assert bwd(ffn(), dX=P[0]) == bwd(ffn(), dX=P[1]) == EINVAL  # the place of dOut, of X
    assert bwd(ffn(), dw=ops.MOE_TYPE_FP16) == bwd(ffn(), dw=3) == bwd(ffn(), add=2) == EINVAL
    assert bwd(ffn(), dw=ops.MOE_TYPE_BF16, add=1) == EUNSUP
    assert lib.moe_gated_ffn_bwd(ctypes.byref(ffn(rows=0)), *([None] * 9), 2, 1, None, 0, None) == ops.MOE_OK
    assert lib.moe_gated_ffn_bwd(ctypes.byref(ffn(rows=0)), *([None] * 9), 2, 0, None, 0, None) == ops.MOE_OK


def ln(**kw):
    v = dict(rows=100, H=520) | kw
    return ops.make_layer_norm_desc(v.pop("rows"), v.pop("H"), **v)


def test_ln_sizes_and_refusals():
    lib = ops.load()
    assert ops.layer_norm_workspace_bytes(ln(rows=0)) == 0
    assert ops.layer_norm_workspace_bytes(ln(rows=1)) == -(-2 * 520 * 4 // 256) * 256
    assert ops.layer_norm_workspace_bytes(ln(rows=1 << 20, H=7168)) == 256 * 2 * 7168 * 4
    F32, B, H16 = torch.float32, torch.bfloat16, torch.float16
    for n, code in ((ln(rows=-1), EINVAL), (ln(H=0), EINVAL), (ln(H=32769), EUNSUP), (ln(ldx=519), EINVAL), (ln(ldy=-1), EINVAL), (ln(eps=-1.0), EINVAL),
                    (ln(eps=float("nan")), EINVAL), (ln(x_dtype=B, y_dtype=F32), EUNSUP), (ln(x_dtype=B, y_dtype=H16), EUNSUP),
                    (ln(x_dtype=H16, y_dtype=B), EUNSUP), (ln(ldx=(1 << 40) + 1), EUNSUP), (ln(rows=(1 << 40) + 1), EUNSUP)):
        assert lib.moe_layer_norm_workspace_bytes(ctypes.byref(n)) == -1
        assert lib.moe_layer_norm_fwd(ctypes.byref(n), *P[:5], None) == code
        assert lib.moe_layer_norm_bwd(ctypes.byref(n), *P[:9], 1 << 40, None) == code
    odd = ln()
    odd.x_type = 3
    assert lib.moe_layer_norm_fwd(ctypes.byref(odd), *P[:5], None) == EINVAL
    assert lib.moe_layer_norm_fwd(None, *P[:5], None) == EINVAL
    for n in (ln(x_dtype=F32, y_dtype=B), ln(ldy=528)):  # rows that do not fit into x's place, dx's into dy's
        assert lib.moe_layer_norm_fwd(ctypes.byref(n), P[0], P[1], P[2], P[0], P[4], None) == EINVAL
        assert lib.moe_layer_norm_bwd(ctypes.byref(n), *P[:5], P[3], *P[6:9], 1 << 40, None) == EINVAL
    assert lib.moe_layer_norm_fwd(ctypes.byref(ln(rows=0)), *([None] * 5), None) == ops.MOE_OK
    names = ("x", "g", "b", "y", "stats")

    def fwd(n, **kw):
        a = dict(zip(names, P)) | kw
        return lib.moe_layer_norm_fwd(ctypes.byref(n), *(a[k] for k in names), None)

    for kw in (dict(x=None), dict(y=None), dict(x=ODD), dict(y=ODD), dict(g=ODD), dict(b=ODD), dict(stats=_fake(0x10004))):
        assert fwd(ln(), **kw) == EINVAL, kw
    assert fwd(ln(x_dtype=F32), x=_fake(0x10002)) == EINVAL
    names2 = ("x", "g", "stats", "dy", "dres", "dx", "dg", "db", "ws")

    def bwd(n, ws_bytes=1 << 40, **kw):
        a = dict(zip(names2, P)) | kw
        return lib.moe_layer_norm_bwd(ctypes.byref(n), *(a[k] for k in names2), ws_bytes, None)

    for kw in (dict(x=None), dict(stats=None), dict(dy=None), dict(dx=None), dict(dg=None), dict(db=None), dict(ws=None), dict(ws=BAD), dict(dres=ODD),
               dict(dx=ODD), dict(dy=ODD), dict(dg=ODD), dict(stats=_fake(0x10004))):
        assert bwd(ln(), **kw) == EINVAL, kw
    assert bwd(ln(), ops.layer_norm_workspace_bytes(ln()) - 1) == ENOSPC
    assert lib.moe_layer_norm_bwd(ctypes.byref(ln(rows=0)), *([None] * 9), 0, None) == ops.MOE_OK


def test_grad_refusals():
    lib = ops.load()
    assert lib.moe_grad_workspace_bytes(-1) == -1 and lib.moe_grad_workspace_bytes(0) > 0

    def table(*rows):
        t = (ops.moe_grad * max(1, len(rows)))()
        for i, r in enumerate(rows):
            t[i] = ops.moe_grad(*r)
        return t

    good = (0x10000, 0x20000, 100, ops.MOE_TYPE_FP32, 0)

    def calls(t, n, kind=0, scale=1.0, max_norm=1.0, eps=0.0, result=P[0], ws=P[1], ws_bytes=1 << 30):
        return [f(t, n, kind, scale, max_norm, eps, result, ws, ws_bytes, None) for f in (lib.moe_grad_norm, lib.moe_grad_clip)]

    nan = float("nan")
    for kw in (dict(kind=2), dict(kind=-1), dict(scale=nan), dict(max_norm=-1.0), dict(max_norm=nan), dict(eps=-1.0), dict(eps=nan), dict(result=None),
               dict(ws=None), dict(result=_fake(0x10004)), dict(ws=_fake(0x10004))):
        assert calls(table(good), 1, **kw) == [EINVAL] * 2, kw
    assert calls(table(good), 1, ws_bytes=lib.moe_grad_workspace_bytes(1) - 1) == [ENOSPC] * 2
    assert calls(table(good), -1) == calls(None, 1) == [EINVAL] * 2
    for bad, code in (((None, 0x20000, 100, 2, 0), EINVAL), ((0x10002, 0x20000, 100, 2, 0), EINVAL), ((0x10001, 0x20000, 100, 0, 0), EINVAL),
                      ((0x10000, 0x20000, -1, 2, 0), EINVAL), ((0x10000, 0x20000, 100, 3, 0), EINVAL), ((0x10000, 0x20000, 100, 2, 1), EINVAL),
                      ((0x10000, 0x20000, 1 << 44, 2, 0), EUNSUP), ((1 << 48, 0x20000, 100, 2, 0), EUNSUP)):
        assert calls(table(good, bad), 2) == [code] * 2, bad
        assert lib.moe_grad_scale(table(good, bad), 2, P[0], 1.0, None) == code
    half = (1 << 43)
    assert calls(table(good, (0x10000, 0x20000, half, 2, 0), (0x10000, 0x20000, half, 2, 0)), 3) == [EUNSUP] * 2
    for bad in ((0x10000, None, 100, 2, 0), (0x10000, 0x20002, 100, 2, 0)):
        assert lib.moe_grad_clip(table(bad), 1, 0, 1.0, 1.0, 0.0, P[0], P[1], 1 << 30, None) == EINVAL
    assert lib.moe_grad_scale(table(good), 1, None, 1.0, None) == lib.moe_grad_scale(table(good), 1, ODD, 1.0, None) == EINVAL
    assert lib.moe_grad_scale(table(good), 1, P[0], nan, None) == EINVAL
    assert lib.moe_grad_scale(None, 0, P[0], 1.0, None) == ops.MOE_OK
    with pytest.raises(TypeError):
        ops.make_grad_list([torch.zeros(4)])
    with pytest.raises(TypeError):
        ops.make_grad_list([], device="cpu")


def test_tensors_on_the_host():
    n = ops.make_ffn_desc(4, 64, 64)
    x, w13, w2 = (torch.zeros(s, dtype=torch.bfloat16) for s in ((4, 64), (128, 64), (64, 64)))
    with pytest.raises(TypeError):
        ops.moe_gated_ffn_fwd(n, x, w13, w2, None, x, x, None)
    with pytest.raises(TypeError):
        ops.moe_layer_norm_fwd(ops.make_layer_norm_desc(4, 64), x, None, None, x, None)


def test_ffn_outputs_in_the_place_of_what_is_read():
    # what a launch still reads beside the output, or writes besides: refused where both start alike
    lib = ops.load()
    names = ("X", "W13", "W2", "HU", "A", "out", "ws")

    def fwd(n, **kw):
        a = dict(zip(names, P)) | kw
        return lib.moe_gated_ffn_fwd(ctypes.byref(n), *(a[k] for k in names), 1 << 40, None)

    at = dict(zip(names, P))
    for o, i in (("A", "X"), ("HU", "X"), ("A", "W13"), ("HU", "W13"), ("A", "W2"), ("HU", "W2"), ("HU", "A"), ("out", "A"), ("out", "W2"), ("out", "W13"),
                 ("out", "HU")):
        assert fwd(ffn(), **{o: at[i]}) == EINVAL, (o, i)
    cut = ffn(rows=70, H=2048, I=8)  # parts in the workspace
    for i in names[:-1]:
        assert fwd(cut, ws=at[i]) == EINVAL, i
    names2 = ("dOut", "X", "HU", "A", "W13", "W2", "dX", "dW13", "dW2", "ws")

    def bwd(n, **kw):
        a = dict(zip(names2, P)) | kw
        return lib.moe_gated_ffn_bwd(ctypes.byref(n), *(a[k] for k in names2[:-1]), ops.MOE_TYPE_BF16, 0, a["ws"], 1 << 40, None)

    at = dict(zip(names2, P))
    for o in names2[6:]:
        for i in names2:
            if i != o:
                assert bwd(ffn(), **{o: at[i]}) == EINVAL, (o, i)


def test_a_failed_build_leaves_no_compiler_behind(tmp_path, monkeypatch):
    from routing_schedule_expert_amd import build

    # a compiler that refuses the first source at once and takes a while over the other
    done, hipcc = tmp_path / "done", tmp_path / "hipcc"
    hipcc.write_text(f"#!/bin/sh\ncase \"$*\" in *{build.SRCS[0]}*) echo refused >&2; exit 1;; esac\nsleep 1\necho done > {done}\n")
    hipcc.chmod(0o755)
    monkeypatch.setenv("HIPCC", str(hipcc))
    monkeypatch.setattr(build, "OUT", str(tmp_path / "libmoe.so"))
    with pytest.raises(RuntimeError, match="refused"):
        build.build()
    assert done.exists()
    assert not (tmp_path / "libmoe.so").exists()
