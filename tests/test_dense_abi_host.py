"""The dense operators' calls on the host: sizes, refusals and empty batches that need no GPU
(CPU only; the fake pointers are never dereferenced)."""
import ctypes

import pytest
import torch

from routing_dispatch_expert_logits_amd import binding as B

L = B.lib
BIG = 1 << 40


def at(i):
    """Fake aligned buffers, far apart."""
    return (i + 1) << 44


def gated(s, ws=at(20), ws_bytes=BIG, **over):
    a = dict(x=at(0), w1=at(1), w3=at(2), h=at(3), g=None, u=None)
    a.update(over)
    return L.moe_gated_forward(a["x"], a["w1"], a["w3"], a["h"], a["g"], a["u"],
                               ctypes.byref(s) if s is not None else None, ws, ws_bytes, None)


def gated_b(s, ws=at(20), ws_bytes=BIG, **over):
    a = dict(dh=at(0), x=at(1), w1=at(2), w3=at(3), g=at(4), u=at(5), dx=at(6), dw1=at(7), dw3=at(8))
    a.update(over)
    return L.moe_gated_backward(*[a[n] for n in ("dh", "x", "w1", "w3", "g", "u", "dx", "dw1", "dw3")],
                                ctypes.byref(s), ws, ws_bytes, None)


def linear(s, ws=at(20), ws_bytes=BIG, **over):
    a = dict(x=at(0), w=at(1), bias=at(2), residual=at(3), y=at(4), z=None)
    a.update(over)
    return L.moe_linear_forward(*[a[n] for n in ("x", "w", "bias", "residual", "y", "z")], ctypes.byref(s), ws,
                                ws_bytes, None)


def linear_b(s, ws=at(20), ws_bytes=BIG, **over):
    a = dict(dy=at(0), x=at(1), w=at(2), z=at(3), dx=at(4), dw=at(5), dbias=at(6))
    a.update(over)
    return L.moe_linear_backward(*[a[n] for n in ("dy", "x", "w", "z", "dx", "dw", "dbias")], ctypes.byref(s), ws,
                                 ws_bytes, None)


def norm(s, **over):
    a = dict(x=at(0), w=at(1), b=at(2), y=at(3), mean=None, rstd=None)
    a.update(over)
    return L.moe_layer_norm_forward(*[a[n] for n in ("x", "w", "b", "y", "mean", "rstd")], ctypes.byref(s), None)


def norm_b(s, ws=at(20), ws_bytes=BIG, **over):
    a = dict(dy=at(0), x=at(1), w=at(2), mean=at(3), rstd=at(4), dx=at(5), dw=at(6), db=at(7))
    a.update(over)
    return L.moe_layer_norm_backward(*[a[n] for n in ("dy", "x", "w", "mean", "rstd", "dx", "dw", "db")],
                                     ctypes.byref(s), ws, ws_bytes, None)


def with_(s, **kw):
    for k, v in kw.items():
        setattr(s, k, v)
    return s


DENSE_CALLS = [gated, gated_b, linear, linear_b]


@pytest.mark.parametrize("call", DENSE_CALLS, ids=lambda f: f.__name__)
def test_dense_shapes_are_checked(call):
    ok = dict(T=33, K=96, N=80, act="silu")
    bad = [with_(B.dense_shape(**ok), **kw) for kw in (
        dict(T=-1), dict(K=0), dict(N=0), dict(N=-8), dict(dtype=2), dict(act=5), dict(act=-1),
        dict(grad_dtype=7), dict(reserved=1))]
    bad.append(B.dense_shape(33, 96, 80, dtype="f32", act="silu", grad_dtype="bf16"))  # narrower than the layer
    for s in bad:
        assert call(s) == B.MOE_ERR_INVALID_ARG
        assert all(B.dense_workspace_bytes(s, c) == 0 for c in range(4))
    for kw in (dict(T=(1 << 28) + 1), dict(K=(1 << 21) + 1), dict(N=(1 << 21) + 1),
               dict(T=1 << 28, K=64), dict(T=1 << 28, N=33, K=8), dict(K=1 << 21, N=1 << 13)):
        assert call(with_(B.dense_shape(**ok), **kw)) == B.MOE_ERR_UNSUPPORTED


def test_dense_pointers_are_checked():
    s = B.dense_shape(33, 96, 80, act="silu")
    assert L.moe_gated_forward(at(0), at(1), at(2), at(3), None, None, None, None, 0, None) == B.MOE_ERR_INVALID_ARG
    for n in ("x", "w1", "w3", "h"):
        assert gated(s, **{n: None}) == B.MOE_ERR_INVALID_ARG
        assert gated(s, **{n: at(9) + 2}) == B.MOE_ERR_INVALID_ARG        # not 16-byte aligned
    assert gated(s, g=at(5)) == B.MOE_ERR_INVALID_ARG                     # g and u: both or neither
    assert gated(s, u=at(5)) == B.MOE_ERR_INVALID_ARG
    for n in ("dh", "x", "w1", "w3", "g", "u"):
        assert gated_b(s, **{n: None}) == B.MOE_ERR_INVALID_ARG
    assert gated_b(s, dw1=None) == B.MOE_ERR_INVALID_ARG                  # dw1 and dw3: both or neither
    assert gated_b(s, dx=None, dw1=None, dw3=None) == B.MOE_ERR_INVALID_ARG
    for n in ("x", "w", "y"):
        assert linear(s, **{n: None}) == B.MOE_ERR_INVALID_ARG
    for n in ("bias", "residual", "z"):
        assert linear(s, **{n: at(9) + 8}) == B.MOE_ERR_INVALID_ARG
    for n in ("dy", "x", "w", "z"):
        assert linear_b(s, **{n: None}) == B.MOE_ERR_INVALID_ARG
    assert linear_b(s, dx=None, dw=None, dbias=None) == B.MOE_ERR_INVALID_ARG
    none = B.dense_shape(33, 96, 80)
    assert linear_b(none) == B.MOE_ERR_INVALID_ARG                        # z without an activation


def test_outputs_may_not_overlap():
    s = B.dense_shape(33, 96, 80, act="silu")
    assert gated(s, h=at(0)) == B.MOE_ERR_INVALID_ARG
    assert gated(s, h=at(1) + 80 * 96 * 2 - 16) == B.MOE_ERR_INVALID_ARG  # the last bytes of w1
    assert gated(s, g=at(5), u=at(5) + 16) == B.MOE_ERR_INVALID_ARG
    assert gated_b(s, dx=at(1)) == B.MOE_ERR_INVALID_ARG
    assert gated_b(s, ws=at(6)) == B.MOE_ERR_INVALID_ARG                  # the workspace over dx
    assert linear(s, y=at(3) + 16) == B.MOE_ERR_INVALID_ARG               # shifted against its residual
    assert linear(s, y=at(3), residual=at(3), z=at(3)) == B.MOE_ERR_INVALID_ARG
    assert linear_b(s, dx=at(0)) == B.MOE_ERR_INVALID_ARG
    n = B.norm_shape(33, 96)
    assert norm(n, y=at(0)) == B.MOE_ERR_INVALID_ARG
    assert norm(n, mean=at(5), rstd=at(5)) == B.MOE_ERR_INVALID_ARG
    assert norm_b(n, dx=at(0)) == B.MOE_ERR_INVALID_ARG
    assert norm_b(n, dw=at(7)) == B.MOE_ERR_INVALID_ARG


def test_workspaces_are_checked():
    s = B.dense_shape(33, 96, 80, act="silu")
    for call, which in ((gated_b, B.MOE_CALL_GATED_BACKWARD), (linear_b, B.MOE_CALL_LINEAR_BACKWARD)):
        need = B.dense_workspace_bytes(s, which)
        assert need > 0
        assert call(s, ws_bytes=need - 1) == B.MOE_ERR_WORKSPACE
        assert call(s, ws=None) == B.MOE_ERR_WORKSPACE
        assert call(s, ws=at(20) + 8) == B.MOE_ERR_INVALID_ARG
    # fp32 weight gradients of a bf16 layer keep three terms
    f = B.dense_shape(33, 96, 80, act="silu", grad_dtype="f32")
    assert B.dense_workspace_bytes(f, B.MOE_CALL_GATED_BACKWARD) > B.dense_workspace_bytes(s, B.MOE_CALL_GATED_BACKWARD)
    n = B.norm_shape(33, 96)
    need = B.norm_workspace_bytes(n)
    assert need >= 2 * 96 * 4
    assert norm_b(n, ws_bytes=need - 1) == B.MOE_ERR_WORKSPACE
    assert B.dense_workspace_bytes(s, 9) == 0


def test_norm_is_checked():
    ok = dict(T=5, H=40)
    for kw in (dict(T=-1), dict(H=0), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")),
               dict(dtype=3), dict(grad_dtype=4), dict(reserved=2)):
        s = with_(B.norm_shape(**ok), **kw)
        assert norm(s) == B.MOE_ERR_INVALID_ARG and norm_b(s) == B.MOE_ERR_INVALID_ARG
        assert B.norm_workspace_bytes(s) == 0
    for kw in (dict(T=(1 << 28) + 1), dict(H=(1 << 21) + 1), dict(T=1 << 28, H=64)):
        assert norm(with_(B.norm_shape(**ok), **kw)) == B.MOE_ERR_UNSUPPORTED
    s = B.norm_shape(**ok)
    for n in ("x", "w", "y"):
        assert norm(s, **{n: None}) == B.MOE_ERR_INVALID_ARG
    for n in ("dy", "x", "w", "mean", "rstd"):
        assert norm_b(s, **{n: None}) == B.MOE_ERR_INVALID_ARG
    assert norm_b(s, dx=None, dw=None, db=None) == B.MOE_ERR_INVALID_ARG


def test_forward_of_no_rows_does_nothing():
    """T = 0 needs no rows and launches nothing."""
    s = B.dense_shape(0, 96, 80, act="silu")
    assert gated(s, x=None, h=None) == B.MOE_OK
    assert linear(s, x=None, y=None, residual=None) == B.MOE_OK
    assert norm(B.norm_shape(0, 96), x=None, y=None) == B.MOE_OK
    assert gated(s, x=None, h=None, w1=None) == B.MOE_ERR_INVALID_ARG


def test_binding_refuses_other_tensors():
    """What a pointer cannot carry: sizes, types, strides, the device."""
    s = B.dense_shape(4, 16, 8)
    x, w, y = torch.zeros(4, 16), torch.zeros(8, 16), torch.zeros(4, 8)
    f = B.dense_shape(4, 16, 8, dtype="f32")
    for shape, args, why in ((s, (x, w, None, None, y), "type"), (f, (x[:3], w, None, None, y), "shape"),
                             (f, (x, w, None, None, y), "not on a GPU")):
        with pytest.raises(B.MoeError, match=why) as e:
            B.linear_forward(*args, shape, None)
        assert e.value.status == B.MOE_ERR_INVALID_ARG
    with pytest.raises(KeyError):
        B.dense_shape(4, 16, 8, act="swish2")


def test_binding_refuses_workspaces_for_what_they_are():
    """A workspace may be of any type: what is wrong with it is not its type."""
    s = B.dense_shape(33, 96, 80)
    for dtype in (torch.float32, torch.uint8):
        with pytest.raises(B.MoeError, match=r"ws: not on a GPU") as e:
            B.linear_forward(at(0), at(1), None, None, at(4), s, torch.zeros(64, dtype=dtype))
        assert e.value.status == B.MOE_ERR_INVALID_ARG
