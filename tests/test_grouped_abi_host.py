"""The grouped, integer and combine-gradient calls on the host: sizes, refusals and empty batches that
need no GPU (CPU only; the fake pointers are never dereferenced)."""
import ctypes

import pytest
import torch

from routing_dispatch_expert_logits_amd import binding as B

L = B.lib
BIG = 1 << 42


def at(i):
    """Fake aligned buffers, far apart."""
    return (i + 1) << 44


def caller(fn, names, required, outputs, has_ws=True):
    def call(s, ws=at(30), ws_bytes=BIG, **over):
        a = {n: at(i) for i, n in enumerate(names)}
        a.update(over)
        args = [a[n] for n in names] + [ctypes.byref(s) if s is not None else None]
        return getattr(L, fn)(*args, *((ws, ws_bytes) if has_ws else ()), None)
    call.__name__ = fn
    call.names, call.required, call.outputs = names, required, outputs
    return call


LF = caller("moe_grouped_linear_forward", ("x", "offsets", "w", "y"), ("x", "offsets", "w", "y"), ("y",))
LB = caller("moe_grouped_linear_backward", ("dy", "x", "offsets", "w", "dx", "dw"), ("dy", "x", "offsets", "w"), ("dx", "dw"))
GF = caller("moe_grouped_gated_forward", ("x", "offsets", "w1", "w3", "h", "g", "u"), ("x", "offsets", "w1", "w3", "h"), ("h", "g", "u"))
GB = caller("moe_grouped_gated_backward", ("dh", "x", "offsets", "w1", "w3", "g", "u", "dx", "dw1", "dw3"),
            ("dh", "x", "offsets", "w1", "w3", "g", "u"), ("dx", "dw1", "dw3"))
LI = caller("moe_grouped_linear_int8_forward", ("x", "x_scale", "offsets", "w", "w_scale", "y"),
            ("x", "x_scale", "offsets", "w", "w_scale", "y"), ("y",))
GI = caller("moe_grouped_gated_int8_forward", ("x", "x_scale", "offsets", "w1", "w1_scale", "w3", "w3_scale", "h"),
            ("x", "x_scale", "offsets", "w1", "w1_scale", "w3", "w3_scale", "h"), ("h",))
DL = caller("moe_linear_int8_forward", ("x", "x_scale", "w", "w_scale", "bias", "residual", "y"),
            ("x", "x_scale", "w", "w_scale", "y"), ("y",), False)
DG = caller("moe_gated_int8_forward", ("x", "x_scale", "w1", "w1_scale", "w3", "w3_scale", "h"),
            ("x", "x_scale", "w1", "w1_scale", "w3", "w3_scale", "h"), ("h",), False)
GROUPED = [LF, LB, GF, GB, LI, GI]
GATED = (GF, GB, GI)
CALL = {f: i for i, f in enumerate(GROUPED)}


def shape(call, **kw):
    a = dict(R=333, K=96, N=80, E=5, act="silu" if call in GATED else "none")
    a.update(kw)
    return B.grouped_shape(**a)


def with_(s, **kw):
    for k, v in kw.items():
        setattr(s, k, v)
    return s


@pytest.mark.parametrize("call", GROUPED, ids=lambda f: f.__name__)
def test_shapes_are_checked(call):
    bad = [with_(shape(call), **kw) for kw in (
        dict(R=-1), dict(K=0), dict(N=0), dict(E=0), dict(E=-3), dict(dtype=2), dict(act=5), dict(act=-1), dict(grad_dtype=7),
        dict(reserved=1))]
    bad.append(shape(call, dtype="f32", grad_dtype="bf16"))      # narrower than the layer
    if call not in GATED:
        bad.append(shape(call, act="relu"))                      # a linear product has no activation
    for s in bad:
        assert call(s) == B.MOE_ERR_INVALID_ARG
        assert B.grouped_workspace_bytes(s, CALL[call]) == 0
    for kw in (dict(R=(1 << 28) + 1), dict(K=(1 << 21) + 1), dict(N=(1 << 21) + 1), dict(E=1025), dict(R=1 << 28, K=64),
               dict(R=1 << 28, N=33, K=8), dict(K=1 << 20, N=1 << 12), dict(E=1024, N=1 << 18, K=8), dict(E=1024, K=1 << 18, N=8)):
        s = with_(shape(call), **kw)
        assert call(s) == B.MOE_ERR_UNSUPPORTED
        assert B.grouped_workspace_bytes(s, CALL[call]) == 0
    assert call(None) == B.MOE_ERR_INVALID_ARG
    assert B.grouped_workspace_bytes(shape(call), 6) == 0 and B.grouped_workspace_bytes(shape(call), -1) == 0


@pytest.mark.parametrize("call", GROUPED + [DL, DG], ids=lambda f: f.__name__)
def test_pointers_are_checked(call):
    s = shape(call) if call in GROUPED else B.dense_shape(33, 96, 80)
    for n in call.required:
        assert call(s, **{n: None}) == B.MOE_ERR_INVALID_ARG, n
    for i, n in enumerate(call.names):
        assert call(s, **{n: at(i) + 4}) == B.MOE_ERR_INVALID_ARG, n      # not 16-byte aligned
    for o in call.outputs:                                                # no output over another buffer
        for i, n in enumerate(call.names):
            if n != o and not (call is DL and n == "residual"):
                assert call(s, **{o: at(i)}) == B.MOE_ERR_INVALID_ARG, (o, n)
    if call in GROUPED:
        i = call.names.index(call.outputs[0])
        assert call(s, ws=at(i)) == B.MOE_ERR_INVALID_ARG                 # nor the workspace over one


def test_gradients_asked_for_in_part():
    s = shape(GB)
    assert GB(s, dw1=None) == B.MOE_ERR_INVALID_ARG                       # dw1 and dw3: both or neither
    assert GB(s, dx=None, dw1=None, dw3=None) == B.MOE_ERR_INVALID_ARG
    assert GF(shape(GF), g=None) == B.MOE_ERR_INVALID_ARG                 # g and u: both or neither
    assert LB(shape(LB), dx=None, dw=None) == B.MOE_ERR_INVALID_ARG
    # operands that only the other gradient needs may be left out: the workspace is what is missing here
    assert GB(s, ws=None, x=None, dw1=None, dw3=None) == B.MOE_ERR_WORKSPACE
    assert GB(s, ws=None, w1=None, w3=None, dx=None) == B.MOE_ERR_WORKSPACE
    assert LB(shape(LB), ws=None, x=None, dw=None) == B.MOE_ERR_WORKSPACE
    assert LB(shape(LB), ws=None, w=None, dx=None) == B.MOE_ERR_WORKSPACE


@pytest.mark.parametrize("call", GROUPED, ids=lambda f: f.__name__)
def test_workspaces_are_checked(call):
    for s in (shape(call), shape(call, K=97, N=83), shape(call, R=4000)):
        need = B.grouped_workspace_bytes(s, CALL[call])
        assert need > 0
        assert call(s, ws_bytes=need - 1) == B.MOE_ERR_WORKSPACE
        assert call(s, ws=None) == B.MOE_ERR_WORKSPACE
        assert call(s, ws=at(30) + 8) == B.MOE_ERR_INVALID_ARG


def test_few_rows_forward_need_no_workspace():
    """Decoding steps read weights of any width in place and make no table."""
    for call in (LF, GF, LI, GI):
        for s in (shape(call, R=16), shape(call, R=1, K=97, N=83)):
            assert B.grouped_workspace_bytes(s, CALL[call]) == 0


def test_fp32_weight_gradients_keep_terms():
    s, f = shape(GB), shape(GB, grad_dtype="f32")
    assert B.grouped_workspace_bytes(f, CALL[GB]) > B.grouped_workspace_bytes(s, CALL[GB])


def test_no_rows_launch_nothing_forward():
    for call in (LF, GF, LI, GI):
        s = shape(call, R=0)
        rows = {n: None for n in call.names if n in ("x", "x_scale", "y", "h", "g", "u")}
        assert call(s, ws=None, ws_bytes=0, **rows) == (B.MOE_OK if B.grouped_workspace_bytes(s, CALL[call]) == 0 else
                                                        B.MOE_ERR_WORKSPACE)
    for call in (DL, DG):
        s = B.dense_shape(0, 96, 80)
        assert call(s, x=None, x_scale=None, **({"y": None, "residual": None} if call is DL else {"h": None})) == B.MOE_OK


def test_int8_sizes():
    for f in (B.int8_row_bytes, L.moe_int8_row_bytes):
        assert [f(n) for n in (1, 16, 17, 1 << 21)] == [16, 16, 32, 1 << 21]
        assert [f(n) for n in (0, -5, (1 << 21) + 1)] == [0, 0, 0]
    # the sums of longer contractions would not fit 32 bits
    assert DL(B.dense_shape(2, (1 << 17) + 1, 8)) == B.MOE_ERR_UNSUPPORTED
    assert LI(shape(LI, K=(1 << 17) + 1, N=8)) == B.MOE_ERR_UNSUPPORTED
    assert B.grouped_workspace_bytes(shape(LI, K=(1 << 17) + 1, N=8), CALL[LI]) == 0
    for kw in (dict(T=-1), dict(K=0), dict(dtype=4), dict(act=9), dict(reserved=3)):
        assert DL(with_(B.dense_shape(3, 32, 8), **kw)) == B.MOE_ERR_INVALID_ARG
        assert DG(with_(B.dense_shape(3, 32, 8), **kw)) == B.MOE_ERR_INVALID_ARG
    assert DL(None) == B.MOE_ERR_INVALID_ARG


def test_quantize_is_checked():
    def q(src=at(0), dt=B.MOE_BF16, rows=4, cols=40, codes=at(1), scale=at(2)):
        return L.moe_quantize_int8(src, dt, rows, cols, codes, scale, None)
    assert q(rows=0, src=None, codes=None, scale=None) == B.MOE_OK
    for kw in (dict(src=None), dict(codes=None), dict(scale=None), dict(src=at(0) + 2), dict(codes=at(1) + 8), dict(dt=3),
               dict(rows=-1), dict(cols=0), dict(codes=at(0)), dict(scale=at(1) + 16)):
        assert q(**kw) == B.MOE_ERR_INVALID_ARG, kw
    for kw in (dict(cols=(1 << 21) + 1), dict(rows=1 << 30, cols=16), dict(rows=(1 << 63) - 1, cols=2)):
        assert q(**kw) == B.MOE_ERR_UNSUPPORTED, kw


def test_combine_backward_is_checked():
    def call(s, dout=at(0), y=at(1), rows=at(2), w=at(3), dy=at(4), dw=at(5), code=B.MOE_BF16):
        return L.moe_combine_backward(dout, y, rows, w, dy, dw, code, ctypes.byref(s) if s else None, None)
    s = B.shape(10, 128, 8, 2, 64)
    for kw in (dict(dout=None), dict(y=None), dict(rows=None), dict(w=None), dict(dy=None, dw=None), dict(code=2),
               dict(dout=at(0) + 8), dict(dy=at(1)), dict(dw=at(3)), dict(dw=at(4) + 16)):
        assert call(s, **kw) == B.MOE_ERR_INVALID_ARG, kw
    assert call(B.shape(10, 130, 8, 2, 64)) == B.MOE_ERR_UNSUPPORTED      # as the layer's other calls
    assert call(B.shape(10, 128, 8, 9, 64)) == B.MOE_ERR_INVALID_ARG
    assert call(None) == B.MOE_ERR_INVALID_ARG


def test_binding_refuses_other_tensors():
    """What a pointer cannot carry: sizes, types, the device."""
    s = B.grouped_shape(4, 16, 8, 2, dtype="f32")
    x, w, y, off = torch.zeros(4, 16), torch.zeros(2, 8, 16), torch.zeros(4, 8), torch.zeros(3, dtype=torch.int32)
    for args, why in (((x, off.long(), w, y), "not on a GPU|type"), ((x[:3], off, w, y), "shape"), ((x, off, w, y), "not on a GPU")):
        with pytest.raises(B.MoeError, match=why) as e:
            B.grouped_linear_forward(*args, s, None)
        assert e.value.status == B.MOE_ERR_INVALID_ARG
    with pytest.raises(B.MoeError, match="not on a GPU"):
        B.quantize_int8(x, torch.zeros(4, 16, dtype=torch.int8), torch.zeros(4))
    with pytest.raises(B.MoeError, match="not on a GPU"):
        B.combine_backward(x, x, off, x, x, x, B.MOE_F32, B.shape(4, 16, 2, 1, 64, dtype="f32"))


@pytest.mark.parametrize("dtype", ("bf16", "f32"))
def test_cut_contractions_have_room_for_their_sums(dtype):
    """Few tiles with a long contraction: the sums of two slices at least, besides the tiles' table; none
    where the contraction is short, or in integers."""
    for call, R, K, N, planes, width in ((LF, 238, 6960, 512, 1, 512), (GF, 238, 4096, 64, 2, 64), (LB, 40, 128, 4096, 1, 128),
                                         (GB, 40, 128, 4096, 1, 128)):
        s = shape(call, R=R, K=K, N=N, E=2, dtype=dtype)
        assert B.grouped_workspace_bytes(s, CALL[call]) > 2 * planes * R * width * 4
    for call, K in ((LF, 64), (LI, 6960)):
        assert B.grouped_workspace_bytes(shape(call, R=238, K=K, N=512, E=2, dtype=dtype), CALL[call]) <= 1024


def test_row_lengths_of_codes_are_the_library_s(monkeypatch):
    """The binding has no rule of its own for them."""
    B._row_bytes.cache_clear()
    monkeypatch.setattr(L, "moe_int8_row_bytes", lambda cols: 4 * cols)
    assert B.int8_row_bytes(5) == 20
    monkeypatch.undo()
    B._row_bytes.cache_clear()
    n = torch.tensor(5)                         # any whole number, by its value
    assert B.int8_row_bytes(5) == B.int8_row_bytes(n) == 16
    assert B.int8_row_bytes(n.fill_(40)) == 48
