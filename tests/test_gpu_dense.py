"""Dense operators on the GPU against their definitions in 64 bits.

Tolerances count roundings: u = 2^-8 (bf16) or 2^-24 (fp32) relative for each value rounded
to the layer's type, n 2^-24 sum |a b| for an fp32 sum of n products in any order, and the
activations' own error: the bf16 kernels form them from the hardware's exp2 and reciprocal
(about 2^-23 of the result each, exp2's argument rounded at 2^-24 |a|) and a 1.5e-7 error
function, together below F = 2^-20 (1 + |a|) of |a|, and four times that for a slope.
"""
import math
import random

import pytest
import torch

from routing_dispatch_expert_logits_amd import binding as B
from tests import gpu_util as gu

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
U32 = 2.0 ** -24
ACTS = ("none", "relu", "silu", "gelu", "gelu_tanh")
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
U = {"bf16": 2.0 ** -8, "f32": U32}
SLOPE = 1.13   # largest |act'| of the five


def act64(a, act):
    """act(a) and act'(a) in 64 bits."""
    if act == "none":
        return a, torch.ones_like(a)
    if act == "relu":
        return a.clamp(min=0), (a > 0).double()
    if act == "silu":
        s = torch.sigmoid(a)
        return a * s, s * (1 + a * (1 - s))
    if act == "gelu":
        p = torch.special.ndtr(a)
        return a * p, p + a * torch.exp(-a * a / 2) / math.sqrt(2 * math.pi)
    c = math.sqrt(2 / math.pi)
    t = torch.tanh(c * (a + 0.044715 * a ** 3))
    return a * (1 + t) / 2, (1 + t) / 2 + a * (1 - t * t) / 2 * c * (1 + 3 * 0.044715 * a * a)


def framed(t):
    """A GPU copy of t with NaN right before and behind it: a read past an edge that enters a
    result shows."""
    pad = 2048
    buf = torch.full((t.numel() + 2 * pad,), float("nan"), dtype=t.dtype, device=DEV)
    view = buf[pad:pad + t.numel()].view(t.shape)
    view.copy_(t)
    return view


def rand(gen, *shape, dtype="bf16", std=1.0):
    return torch.empty(shape, dtype=torch.float32).normal_(0, std, generator=gen).to(TYPES[dtype])


def out(shape, dtype):
    """A guarded output buffer (raw bits for bf16), and how to read it in 64 bits."""
    return gu.empty(shape, dtype)


def f64(t, dtype):
    if dtype == "bf16":
        t = t.view(torch.bfloat16)
    return t.cpu().double()


def ws_for(s, call=None):
    """Exactly the bytes asked for, between guard bands, NaN where they are read unwritten."""
    n = B.norm_workspace_bytes(s) if call is None else B.dense_workspace_bytes(s, call)
    return gu.empty((n,), "u8").fill_(0xFF) if n else None


def check(name, got, ref, tol):
    assert torch.isfinite(got).all(), name
    over = (got - ref).abs() - tol
    assert bool((over <= 0).all()), f"{name}: {float((got - ref).abs().max()):.3e} off, {float(over.max()):.3e} over"


def fsum(a, b, n):
    """Bound of the fp32 sums in a @ b^T (n products each, and a few terms beside)."""
    return (n + 8) * U32 * (a.abs() @ b.abs().T)


# T, K, N: single rows, whole tiles, sizes that end inside tiles, chunks and pairs
SIZES = [(1, 64, 64), (1, 257, 131), (2, 8, 8), (3, 1, 1), (7, 1024, 96), (16, 136, 200), (17, 72, 56),
         (33, 333, 77), (64, 64, 64), (65, 128, 129), (130, 515, 260), (256, 256, 256), (257, 200, 264),
         (300, 64, 1000), (1000, 1032, 72)]


def small(i):
    return "x".join(map(str, i)) if isinstance(i, tuple) else None


@pytest.mark.parametrize("dtype", ("bf16", "f32"))
@pytest.mark.parametrize("size", SIZES, ids=small)
def test_gated_forward(size, dtype):
    T, K, N = size
    gen = torch.Generator().manual_seed(sum(size))
    act = ACTS[sum(size) % 5]
    x, w1, w3 = rand(gen, T, K, dtype=dtype), rand(gen, N, K, dtype=dtype, std=K ** -0.5), rand(gen, N, K, dtype=dtype, std=0.1)
    s = B.dense_shape(T, K, N, dtype=dtype, act=act)
    h, g, u, h2 = (out((T, N), dtype) for _ in range(4))
    ws = ws_for(s, B.MOE_CALL_GATED_FORWARD)
    dx, dw1, dw3 = framed(x), framed(w1), framed(w3)
    B.gated_forward(dx, dw1, dw3, h, s, ws, g=g, u=u)
    B.gated_forward(dx, dw1, dw3, h2, s, ws)                   # without the projections kept
    x, w1, w3 = x.double(), w1.double(), w3.double()
    rg, ru = x @ w1.T, x @ w3.T
    a, _ = act64(rg, act)
    eg, eu = fsum(x, w1, K), fsum(x, w3, K)
    check("g", f64(g, dtype), rg, U[dtype] * rg.abs() + 2 * eg)
    check("u", f64(u, dtype), ru, U[dtype] * ru.abs() + 2 * eu)
    tol = U[dtype] * (a * ru).abs() + 2 * (SLOPE * eg * ru.abs() + a.abs() * eu + SLOPE * eg * eu) \
        + 2.0 ** -20 * (1 + rg.abs()) * rg.abs() * ru.abs()
    check("h", f64(h, dtype), a * ru, tol)
    assert torch.equal(h, h2)


@pytest.mark.parametrize("dtype,grad", (("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")))
@pytest.mark.parametrize("size", SIZES, ids=small)
def test_gated_backward(size, dtype, grad):
    T, K, N = size
    gen = torch.Generator().manual_seed(sum(size) + 1)
    act = ACTS[(sum(size) + 2) % 5]
    x, dh = rand(gen, T, K, dtype=dtype), rand(gen, T, N, dtype=dtype)
    w1, w3 = rand(gen, N, K, dtype=dtype, std=0.1), rand(gen, N, K, dtype=dtype, std=0.1)
    g, u = rand(gen, T, N, dtype=dtype, std=1.7), rand(gen, T, N, dtype=dtype, std=1.7)
    s = B.dense_shape(T, K, N, dtype=dtype, act=act, grad_dtype=grad)
    dx, dw1, dw3 = out((T, K), dtype), out((N, K), grad), out((N, K), grad)
    ws = ws_for(s, B.MOE_CALL_GATED_BACKWARD)
    args = [framed(t) for t in (dh, x, w1, w3, g, u)]
    B.gated_backward(*args, dx, dw1, dw3, s, ws)
    x, dh, w1, w3, g, u = (t.double() for t in (x, dh, w1, w3, g, u))
    a, slope = act64(g, act)
    dg, du = dh * u * slope, dh * a
    fe = 2.0 ** -18 * (1 + g.abs())
    eg, eu = fe * (dh * u).abs(), fe * (dh * g).abs()
    r = U[dtype]
    # each gradient asked for alone too
    dx2, p, q = out((T, K), dtype), out((N, K), grad), out((N, K), grad)
    B.gated_backward(*args, dx2, None, None, s, ws)
    B.gated_backward(*args, None, p, q, s, ws)
    for got in (dx, dx2):
        check("dx", f64(got, dtype), dg @ w1 + du @ w3,
              r * (dg @ w1 + du @ w3).abs() + (r * dg.abs() + eg) @ w1.abs() + (r * du.abs() + eu) @ w3.abs()
              + 2 * (fsum(dg, w1.T, 2 * N) + fsum(du, w3.T, 2 * N)))
    rw = U[grad]                # three bf16 terms hold an fp32 value
    for name, got, d, e in (("dw1", dw1, dg, eg), ("dw3", dw3, du, eu), ("dw1", p, dg, eg), ("dw3", q, du, eu)):
        check(name, f64(got, grad), d.T @ x,
              U[grad] * (d.T @ x).abs() + (rw * d.abs() + e).T @ x.abs() + 2 * fsum(d.T, x.T, 3 * T))


@pytest.mark.parametrize("dtype", ("bf16", "f32"))
@pytest.mark.parametrize("size", SIZES, ids=small)
def test_linear_forward(size, dtype):
    T, K, N = size
    gen = torch.Generator().manual_seed(sum(size) + 2)
    x, w = rand(gen, T, K, dtype=dtype), rand(gen, N, K, dtype=dtype, std=K ** -0.5)
    bias, res = rand(gen, N, dtype=dtype), rand(gen, T, N, dtype=dtype)
    x64, w64 = x.double(), w.double()
    dev = [framed(t) for t in (x, w, bias, res)]
    for act, b, r, keep in (("none", 0, 0, 0), (ACTS[sum(size) % 5], 1, 1, 1), ("gelu", 1, 0, 0), ("silu", 0, 1, 1)):
        s = B.dense_shape(T, K, N, dtype=dtype, act=act)
        ws = ws_for(s, B.MOE_CALL_LINEAR_FORWARD)
        y, z = out((T, N), dtype), out((T, N), dtype)
        B.linear_forward(dev[0], dev[1], dev[2] if b else None, dev[3] if r else None, y, s, ws, z=z if keep else None)
        rz = x64 @ w64.T + (bias.double() if b else 0.0)
        a, _ = act64(rz, act)
        ry = a + (res.double() if r else 0.0)
        ez = 2 * fsum(x64, w64, K) + U32 * rz.abs()
        if keep:
            check("z", f64(z, dtype), rz, U[dtype] * rz.abs() + 2 * ez)
        check("y", f64(y, dtype), ry, U[dtype] * ry.abs() + SLOPE * ez + 2.0 ** -20 * (1 + rz.abs()) * rz.abs()
              + 2 * U32 * ry.abs())
    # in place of the residual: the same bits
    y2 = out((T, N), dtype)
    y2.copy_(dev[3].view(y2.dtype))
    B.linear_forward(dev[0], dev[1], None, y2, y2, s, ws)
    assert torch.equal(y, y2)


@pytest.mark.parametrize("dtype,grad", (("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")))
@pytest.mark.parametrize("size", SIZES, ids=small)
def test_linear_backward(size, dtype, grad):
    T, K, N = size
    gen = torch.Generator().manual_seed(sum(size) + 3)
    x, dy = rand(gen, T, K, dtype=dtype), rand(gen, T, N, dtype=dtype)
    w, z = rand(gen, N, K, dtype=dtype, std=0.1), rand(gen, T, N, dtype=dtype, std=1.7)
    dev = [framed(t) for t in (dy, x, w, z)]
    x, dy, w, z = (t.double() for t in (x, dy, w, z))
    for act in ("none", ACTS[1 + sum(size) % 4]):
        s = B.dense_shape(T, K, N, dtype=dtype, act=act, grad_dtype=grad)
        dx, dw, db = out((T, K), dtype), out((N, K), grad), out((N,), grad)
        ws = ws_for(s, B.MOE_CALL_LINEAR_BACKWARD)
        dz_in = dev[3] if act != "none" else None
        B.linear_backward(dev[0], dev[1], dev[2], dz_in, dx, dw, db, s, ws)
        dz = dy * act64(z, act)[1]
        r = U[dtype] if act != "none" else 0.0
        e = 2.0 ** -18 * (1 + z.abs()) * dy.abs() if act != "none" else 0.0 * dy
        rw = U[grad]                # three bf16 terms hold an fp32 value
        ref = ((dz @ w, U[dtype] * (dz @ w).abs() + (r * dz.abs() + e) @ w.abs() + 2 * fsum(dz, w.T, N)),
               (dz.T @ x, U[grad] * (dz.T @ x).abs() + (min(r, rw) * dz.abs() + e).T @ x.abs()
                + 2 * fsum(dz.T, x.T, 3 * T)),
               (dz.sum(0), U[grad] * dz.sum(0).abs() + e.sum(0) + (T + 8) * U32 * dz.abs().sum(0)))
        kinds = (dtype, grad, grad)
        for name, got, kind, (want, tol) in zip(("dx", "dw", "dbias"), (dx, dw, db), kinds, ref):
            check(name, f64(got, kind), want, tol)
        for keep in range(3):                    # each gradient alone
            o = [out((T, K), dtype), out((N, K), grad), out((N,), grad)]
            o = [t if i == keep else None for i, t in enumerate(o)]
            B.linear_backward(dev[0], dev[1] if keep == 1 else None, dev[2] if keep == 0 else None, dz_in, *o, s, ws)
            check("alone", f64(o[keep], kinds[keep]), *ref[keep])


@pytest.mark.parametrize("act", ("none", "relu"))
@pytest.mark.parametrize("size", ((1, 64, 64), (130, 515, 260), (700, 72, 129)), ids=small)
def test_f32_gradients_of_a_slope_of_one(size, act):
    """With slopes of 0 and 1 the gradient before the activation is one bf16 number or a product
    of two, which the operands of the products hold exactly: only the fp32 sums are off."""
    T, K, N = size
    gen = torch.Generator().manual_seed(sum(size) + 4)
    dy, x, g, u = rand(gen, T, N), rand(gen, T, K), rand(gen, T, N), rand(gen, T, N)
    s = B.dense_shape(T, K, N, act=act, grad_dtype="f32")
    dev = [framed(t) for t in (dy, x, g, u)]
    w = framed(rand(gen, N, K))
    dw, dw1, dw3 = (out((N, K), "f32") for _ in range(3))
    B.linear_backward(dev[0], dev[1], None, dev[2] if act != "none" else None, None, dw, None, s,
                      ws_for(s, B.MOE_CALL_LINEAR_BACKWARD))
    B.gated_backward(dev[0], dev[1], w, w, dev[2], dev[3], None, dw1, dw3, s, ws_for(s, B.MOE_CALL_GATED_BACKWARD))
    dy, x, g, u = (t.double() for t in (dy, x, g, u))
    a, slope = act64(g, act)
    for name, got, d in (("dw", dw, dy * slope), ("dw1", dw1, dy * u * slope), ("dw3", dw3, dy * a)):
        check(name, f64(got, "f32"), d.T @ x, U32 * (d.T @ x).abs() + 2 * fsum(d.T, x.T, 2 * T))


@pytest.mark.parametrize("act", ACTS)
def test_infinite_gradients_stay_infinite(act):
    """An infinite gradient row gives infinite weight gradients of its own row and no others, in
    fp32 as in bf16: the terms of an fp32 gradient do not make it NaN."""
    T, K, N = 3, 40, 24
    gen = torch.Generator().manual_seed(7)
    dy, x, g, u = rand(gen, T, N), rand(gen, T, K).abs() + 0.5, rand(gen, T, N).abs() + 0.5, rand(gen, T, N).abs() + 0.5
    w = rand(gen, N, K).to(DEV)
    dy[1, 5] = float("inf")
    for grad in ("bf16", "f32"):
        s = B.dense_shape(T, K, N, act=act, grad_dtype=grad)
        dev = [t.to(DEV) for t in (dy, x, g, u)]
        dw, dw1, dw3, db = (out(sh, grad) for sh in ((N, K), (N, K), (N, K), (N,)))
        B.linear_backward(dev[0], dev[1], None, dev[2] if act != "none" else None, None, dw, db, s,
                          ws_for(s, B.MOE_CALL_LINEAR_BACKWARD))
        B.gated_backward(dev[0], dev[1], w, w, dev[2], dev[3], None, dw1, dw3, s, ws_for(s, B.MOE_CALL_GATED_BACKWARD))
        for name, got in (("dw", dw), ("dbias", db), ("dw1", dw1), ("dw3", dw3)):
            got = f64(got, grad)
            assert bool((got[5] == float("inf")).all()), name
            assert bool(torch.isfinite(torch.cat((got[:5], got[6:]))).all()), name


@pytest.mark.parametrize("dtype", ("bf16", "f32"))
@pytest.mark.parametrize("act", ACTS)
def test_activations_of_the_largest_values(act, dtype):
    """act and act' of finite pre-activations up to the type's largest: themselves and 1, or 0."""
    z = torch.tensor([20.0, 1e5, 1e13, 1e20, 3e38], dtype=TYPES[dtype])
    z = torch.cat((z, -z, -z[:2])).view(1, -1)
    N = z.numel()
    s = B.dense_shape(1, N, N, dtype=dtype, act=act)
    eye = torch.eye(N, dtype=TYPES[dtype]).to(DEV)
    y, db = out((1, N), dtype), out((N,), dtype)
    B.linear_forward(z.to(DEV), eye, None, None, y, s, ws_for(s, B.MOE_CALL_LINEAR_FORWARD))
    B.linear_backward(torch.full_like(z, 2.0).to(DEV), None, None, z.to(DEV) if act != "none" else None, None, None, db, s,
                      ws_for(s, B.MOE_CALL_LINEAR_BACKWARD))
    up = (z.double() > 0) | (act == "none")
    # |act(-20)| and |act'(-20)| are below 20 e^(-20), and so far are act(20) and act'(20) from 20
    # and 1; e^(-20), the sum, the reciprocal and the product round in fp32 (2^-18 for all of them)
    far = 20 * math.exp(-20.0) * (1 + 2.0 ** -18)
    want = torch.where(up, z.double(), 0.0)
    check("y", f64(y, dtype), want, 2 * U32 * want.abs() + far)
    check("dbias", f64(db, dtype), torch.where(up, 2.0, 0.0).double()[0], 2 * far + 2 * U32)


# Sizes that end inside the largest tiles and fill the device, together with those above on every
# tile shape and with the contraction cut into slices; the 64-bit products run on the GPU.
LARGE = [(3800, 4072, 4000), (8200, 520, 4100), (4104, 1096, 4112), (1030, 2056, 2100), (520, 4096, 520), (100, 7168, 1000),
         (5000, 300, 2200)]


def random_sizes(n):
    """Sizes spread over their logarithms, whole tiles, whole chunks and odd ones."""
    r = random.Random(20)
    spread = lambda lo, hi: int(math.exp(r.uniform(math.log(lo), math.log(hi))))  # noqa: E731
    return [(spread(1, 4000),) + tuple(max(1, spread(8, 5000) // s * s) for s in r.choices((64, 8, 1), k=2)) for _ in range(n)]


LARGE += random_sizes(28)


def close(name, got, dtype, ref, tol):
    got = (got.view(torch.bfloat16) if dtype == "bf16" else got).double()
    over = (got - ref).abs() - tol
    assert bool(torch.isfinite(got).all()) and bool((over <= 0).all()), \
        f"{name}: {float((got - ref).abs().max()):.3e} off, {float(over.max()):.3e} over"


@pytest.mark.parametrize("dtype", ("bf16", "f32"))
@pytest.mark.parametrize("size", LARGE, ids=small)
def test_large_gated(size, dtype):
    T, K, N = size
    gen = torch.Generator().manual_seed(T)
    x, w1, w3 = (rand(gen, *s, dtype=dtype, std=v).to(DEV) for s, v in (((T, K), 1), ((N, K), 0.05), ((N, K), 0.05)))
    s = B.dense_shape(T, K, N, dtype=dtype, act="silu")
    h, g, u = (out((T, N), dtype) for _ in range(3))
    B.gated_forward(x, w1, w3, h, s, ws_for(s, B.MOE_CALL_GATED_FORWARD), g=g, u=u)
    x, w1, w3 = x.double(), w1.double(), w3.double()
    rg, ru = x @ w1.T, x @ w3.T
    eg, eu = 2 * fsum(x, w1, K), 2 * fsum(x, w3, K)
    a, _ = act64(rg, "silu")
    r = U[dtype]
    close("g", g, dtype, rg, r * rg.abs() + eg)
    close("u", u, dtype, ru, r * ru.abs() + eu)
    close("h", h, dtype, a * ru, r * (a * ru).abs() + SLOPE * eg * ru.abs() + a.abs() * eu + SLOPE * eg * eu
          + 2.0 ** -20 * (1 + rg.abs()) * rg.abs() * ru.abs())


@pytest.mark.parametrize("dtype,grad", (("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")))
@pytest.mark.parametrize("size", LARGE, ids=small)
def test_large_gated_backward(size, dtype, grad):
    T, K, N = size
    gen = torch.Generator().manual_seed(T + 1)
    x, dh, w1, w3, g, u = (rand(gen, *s, dtype=dtype, std=v).to(DEV) for s, v in (
        ((T, K), 1), ((T, N), 1), ((N, K), 0.05), ((N, K), 0.05), ((T, N), 1.7), ((T, N), 1.7)))
    s = B.dense_shape(T, K, N, dtype=dtype, act="gelu", grad_dtype=grad)
    dx, dw1, dw3 = out((T, K), dtype), out((N, K), grad), out((N, K), grad)
    B.gated_backward(dh, x, w1, w3, g, u, dx, dw1, dw3, s, ws_for(s, B.MOE_CALL_GATED_BACKWARD))
    x, dh, w1, w3, g, u = (t.double() for t in (x, dh, w1, w3, g, u))
    a, slope = act64(g, "gelu")
    dg, du = dh * u * slope, dh * a
    fe = 2.0 ** -18 * (1 + g.abs())
    eg, eu = fe * (dh * u).abs(), fe * (dh * g).abs()
    r, rw = U[dtype], U[grad]
    ref = dg @ w1 + du @ w3
    close("dx", dx, dtype, ref, r * ref.abs() + (r * dg.abs() + eg) @ w1.abs() + (r * du.abs() + eu) @ w3.abs()
          + 2 * (fsum(dg, w1.T, 2 * N) + fsum(du, w3.T, 2 * N)))
    for name, got, d, e in (("dw1", dw1, dg, eg), ("dw3", dw3, du, eu)):
        ref = d.T @ x
        close(name, got, grad, ref, rw * ref.abs() + (rw * d.abs() + e).T @ x.abs() + 2 * fsum(d.T, x.T, 3 * T))


@pytest.mark.parametrize("dtype", ("bf16", "f32"))
@pytest.mark.parametrize("size", LARGE, ids=small)
def test_large_linear(size, dtype):
    T, K, N = size
    gen = torch.Generator().manual_seed(T + 2)
    x, w, bias, res, dy = (rand(gen, *s, dtype=dtype, std=v).to(DEV) for s, v in (
        ((T, K), 1), ((N, K), 0.05), ((N,), 1), ((T, N), 1), ((T, N), 1)))
    s = B.dense_shape(T, K, N, dtype=dtype, act="gelu_tanh")
    y, z = out((T, N), dtype), out((T, N), dtype)
    B.linear_forward(x, w, bias, res, y, s, ws_for(s, B.MOE_CALL_LINEAR_FORWARD), z=z)
    dx, dw, db = out((T, K), dtype), out((N, K), dtype), out((N,), dtype)
    n = B.dense_shape(T, K, N, dtype=dtype)
    B.linear_backward(dy, x, w, None, dx, dw, db, n, ws_for(n, B.MOE_CALL_LINEAR_BACKWARD))
    x, w, bias, res, dy = (t.double() for t in (x, w, bias, res, dy))
    rz = x @ w.T + bias
    ez = 2 * fsum(x, w, K) + U32 * rz.abs()
    a, _ = act64(rz, "gelu_tanh")
    r = U[dtype]
    close("z", z, dtype, rz, r * rz.abs() + 2 * ez)
    close("y", y, dtype, a + res, r * (a + res).abs() + SLOPE * ez + 2.0 ** -20 * (1 + rz.abs()) * rz.abs()
          + 2 * U32 * (a + res).abs())
    close("dx", dx, dtype, dy @ w, r * (dy @ w).abs() + 2 * fsum(dy, w.T, N))
    close("dw", dw, dtype, dy.T @ x, r * (dy.T @ x).abs() + 2 * fsum(dy.T, x.T, T))
    close("dbias", db, dtype, dy.sum(0), r * dy.sum(0).abs() + (T + 8) * U32 * dy.abs().sum(0))


NORM_SIZES = [(1, 1), (1, 8), (2, 7), (3, 64), (5, 1021), (64, 512), (33, 2048), (31, 2056), (300, 1000), (9, 4096),
              (70, 7168), (5, 8200), (3, 20001), (2, 40000), (4100, 129)]


def norm_inputs(T, H, dtype, seed):
    gen = torch.Generator().manual_seed(seed)
    rows = torch.empty(T, 2).normal_(generator=gen)
    x = (torch.empty(T, H).normal_(generator=gen) * torch.exp2(rows[:, :1]) + rows[:, 1:]).to(TYPES[dtype])
    return x, (1 + rand(gen, H, dtype="f32", std=0.1)).to(TYPES[dtype]), rand(gen, H, dtype=dtype, std=0.1), \
        rand(gen, T, H, dtype=dtype)


@pytest.mark.parametrize("dtype", ("bf16", "f32"))
@pytest.mark.parametrize("size", NORM_SIZES, ids=small)
def test_norm_forward(size, dtype):
    T, H = size
    x, w, b, _ = norm_inputs(T, H, dtype, sum(size))
    s = B.norm_shape(T, H, eps=1e-3, dtype=dtype)
    for bias in (True, False):
        y, mean, rstd = out((T, H), dtype), out((T,), "f32"), out((T,), "f32")
        B.layer_norm_forward(framed(x), framed(w), framed(b) if bias else None, y, s, mean=mean, rstd=rstd)
        x64 = x.double()
        m = x64.mean(1, keepdim=True)
        d = x64 - m
        r = 1 / torch.sqrt((d * d).mean(1, keepdim=True) + 1e-3)
        # the mean of H terms in fp32, at most 8 + H / 64 additions deep on any lane's path; the
        # centred row carries that error, one rounding and the variance's relative error
        depth = 16 + H // 64
        em = depth * U32 * x64.abs().mean(1, keepdim=True)
        check("mean", f64(mean, "f32"), m[:, 0], 2 * em[:, 0])
        ed = em + U32 * (x64.abs() + m.abs())
        er = r * (depth * U32 + r * r * ((ed * d.abs()).mean(1, keepdim=True) + ed.square().mean(1, keepdim=True)))
        check("rstd", f64(rstd, "f32"), r[:, 0], 2 * er[:, 0])
        ref = d * r * w.double() + (b.double() if bias else 0)
        tol = U[dtype] * ref.abs() + 2 * ((ed * r + d.abs() * er) * w.double().abs()
                                          + 4 * U32 * ((d * r * w.double()).abs() + b.double().abs()))
        check("y", f64(y, dtype), ref, tol)
        y2 = out((T, H), dtype)
        B.layer_norm_forward(framed(x), framed(w), framed(b) if bias else None, y2, s)
        assert torch.equal(y, y2)


@pytest.mark.parametrize("dtype,grad", (("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")))
@pytest.mark.parametrize("size", NORM_SIZES, ids=small)
def test_norm_backward(size, dtype, grad):
    T, H = size
    x, w, b, dy = norm_inputs(T, H, dtype, sum(size) + 7)
    mean = x.double().mean(1).float()
    rstd = (1 / torch.sqrt((x.double() - mean.double()[:, None]).square().mean(1) + 1e-3)).float()
    s = B.norm_shape(T, H, eps=1e-3, dtype=dtype, grad_dtype=grad)
    dx, dw, db = out((T, H), dtype), out((H,), grad), out((H,), grad)
    ws = ws_for(s)
    dev = [framed(t) for t in (dy, x, w, mean, rstd)]
    B.layer_norm_backward(*dev, dx, dw, db, s, ws)
    x, w, dy, m, r = x.double(), w.double(), dy.double(), mean.double()[:, None], rstd.double()[:, None]
    n = (x - m) * r
    en = 2 * U32 * n.abs() + U32 * r * (x - m).abs()          # x - m and its product with rstd
    e = dy * w
    c1, c2 = e.mean(1, keepdim=True), (e * n).mean(1, keepdim=True)
    ref = r * (e - c1 - n * c2)
    depth = 16 + H // 64
    e1 = depth * U32 * e.abs().mean(1, keepdim=True)
    e2 = depth * U32 * (e * n).abs().mean(1, keepdim=True) + (e.abs() * en).mean(1, keepdim=True)
    tol = U[dtype] * ref.abs() + 2 * r * (e1 + n.abs() * e2 + en * c2.abs()
                                          + 6 * U32 * (e.abs() + c1.abs() + (n * c2).abs()))
    check("dx", f64(dx, dtype), ref, tol)
    check("dw", f64(dw, grad), (dy * n).sum(0), U[grad] * (dy * n).sum(0).abs() + (dy.abs() * en).sum(0)
          + (T + 8) * U32 * (dy * n).abs().sum(0))
    check("db", f64(db, grad), dy.sum(0), U[grad] * dy.sum(0).abs() + (T + 8) * U32 * dy.abs().sum(0))
    for keep in range(3):
        o = [out((T, H), dtype), out((H,), grad), out((H,), grad)]
        o = [t if i == keep else None for i, t in enumerate(o)]
        B.layer_norm_backward(*dev, *o, s, ws)
        assert torch.equal(o[keep], (dx, dw, db)[keep])


def test_norm_rows_that_cancel():
    """Rows that are constant (variance 0, one of them far from 0) and rows whose mean is large
    against their spread: the centred row decides, not a difference of squares."""
    H = 1000
    x = torch.full((4, H), 3.0)
    x[1] = 4096.0
    x[2] = 4096.0 + torch.arange(H) % 2               # spread 0.5 about 4096.5
    x[3] = 0.0
    y, mean, rstd = out((4, H), "f32"), out((4,), "f32"), out((4,), "f32")
    one = torch.ones(H, device=DEV)
    B.layer_norm_forward(x.to(DEV), one, None, y, B.norm_shape(4, H, eps=1e-5, dtype="f32"), mean=mean, rstd=rstd)
    assert y.cpu()[[0, 1, 3]].abs().max() == 0 and torch.isfinite(y).all()
    # the sum of 1000 integers up to 4097 is exact in fp32 (below 2^24), so is its quotient 4096.5
    assert mean.cpu().tolist() == [3.0, 4096.0, 4096.5, 0.0]
    torch.testing.assert_close(y.cpu()[2].abs().double(), torch.full((H,), 0.5 / math.sqrt(0.25 + 1e-5),
                               dtype=torch.float64), rtol=8 * U32, atol=0)


@pytest.mark.parametrize("dtype", ("bf16", "f32"))
def test_bad_values_stay_in_their_rows(dtype):
    """NaN and infinities of one token reach that token's outputs and no other's."""
    T, K, N, H = 70, 136, 72, 136
    gen = torch.Generator().manual_seed(5)
    x, w, w3 = rand(gen, T, K, dtype=dtype), rand(gen, N, K, dtype=dtype), rand(gen, N, K, dtype=dtype)
    bad = x.clone()
    bad[3, 5], bad[69, 135], bad[64, 0] = float("nan"), float("inf"), float("-inf")
    rows = [r for r in range(T) if r not in (3, 64, 69)]
    s = B.dense_shape(T, K, N, dtype=dtype, act="silu")
    res = []
    for v in (x, bad):
        h, y = out((T, N), dtype), out((T, N), dtype)
        n = out((T, H), dtype)
        B.gated_forward(framed(v), framed(w), framed(w3), h, s, ws_for(s, B.MOE_CALL_GATED_FORWARD))
        B.linear_forward(framed(v), framed(w), None, None, y, s, ws_for(s, B.MOE_CALL_LINEAR_FORWARD))
        B.layer_norm_forward(framed(v), framed(torch.ones(H, dtype=TYPES[dtype])), None, n,
                             B.norm_shape(T, H, dtype=dtype))
        res.append([f64(t, dtype) for t in (h, y, n)])
    for a, b in zip(*res):
        assert torch.equal(a[rows], b[rows])
        assert not torch.isfinite(b[3]).any()
        assert not torch.isfinite(b[[64, 69]]).all()


def test_no_rows():
    """T = 0: forward passes write nothing, backward passes write zero weight gradients."""
    for dtype in ("bf16", "f32"):
        s = B.dense_shape(0, 40, 24, dtype=dtype, act="silu")
        e = torch.empty(0, 24, dtype=TYPES[dtype], device=DEV)
        x = torch.empty(0, 40, dtype=TYPES[dtype], device=DEV)
        w = torch.zeros(24, 40, dtype=TYPES[dtype], device=DEV)
        dw1, dw3, db = out((24, 40), dtype), out((24, 40), dtype), out((24,), dtype)
        B.gated_backward(e, x, w, w, e, e, torch.empty_like(x), dw1, dw3, s, ws_for(s, B.MOE_CALL_GATED_BACKWARD))
        assert f64(dw1, dtype).eq(0).all() and f64(dw3, dtype).eq(0).all()
        B.linear_backward(e, x, w, e, torch.empty_like(x), dw1, db, s, ws_for(s, B.MOE_CALL_LINEAR_BACKWARD))
        assert f64(dw1, dtype).eq(0).all() and f64(db, dtype).eq(0).all()
        n = B.norm_shape(0, 24, dtype=dtype)
        m = torch.empty(0, device=DEV)
        dw = out((24,), dtype)
        B.layer_norm_backward(e, e, db.view(TYPES[dtype]), m, m, None, dw, None, n, ws_for(n))
        assert f64(dw, dtype).eq(0).all()


# ---- the operators together: y = x + linear(gated(norm(x)))

class Block:
    """One pre-norm dense block through the calls, its buffers kept."""

    def __init__(self, T, H, I, dtype, seed, act="silu"):
        gen = torch.Generator().manual_seed(seed)
        self.T, self.H, self.I, self.dtype, self.act = T, H, I, dtype, act
        t = TYPES[dtype]
        self.p = dict(nw=(1 + rand(gen, H, dtype="f32", std=0.1)).to(t), nb=rand(gen, H, dtype=dtype, std=0.1),
                      w1=rand(gen, I, H, dtype=dtype, std=H ** -0.5), w3=rand(gen, I, H, dtype=dtype, std=H ** -0.5),
                      w2=rand(gen, H, I, dtype=dtype, std=I ** -0.5), b2=rand(gen, H, dtype=dtype, std=0.1))
        self.x, self.dy = rand(gen, T, H, dtype=dtype), rand(gen, T, H, dtype=dtype)
        self.d = {k: v.to(DEV) for k, v in dict(self.p, x=self.x, dy=self.dy).items()}
        self.sn = B.norm_shape(T, H, dtype=dtype)
        self.sg = B.dense_shape(T, H, I, dtype=dtype, act=act)
        self.sl = B.dense_shape(T, I, H, dtype=dtype)
        n = max(B.norm_workspace_bytes(self.sn), *(B.dense_workspace_bytes(s, c) for s, c in (
            (self.sg, B.MOE_CALL_GATED_FORWARD), (self.sg, B.MOE_CALL_GATED_BACKWARD),
            (self.sl, B.MOE_CALL_LINEAR_FORWARD), (self.sl, B.MOE_CALL_LINEAR_BACKWARD))))
        self.ws = torch.empty(max(n, 16), dtype=torch.uint8, device=DEV)
        e = lambda *shape, dt=t: torch.empty(shape, dtype=dt, device=DEV)  # noqa: E731
        self.o = dict(n=e(T, H), mean=e(T, dt=torch.float32), rstd=e(T, dt=torch.float32), h=e(T, I), g=e(T, I),
                      u=e(T, I), y=e(T, H), dh=e(T, I), dn=e(T, H), dx=e(T, H), dnw=e(H), dnb=e(H), dw1=e(I, H),
                      dw3=e(I, H), dw2=e(H, I), db2=e(H))

    def run(self, stream=None):
        d, o, ws = self.d, self.o, self.ws
        B.layer_norm_forward(d["x"], d["nw"], d["nb"], o["n"], self.sn, o["mean"], o["rstd"], stream=stream)
        B.gated_forward(o["n"], d["w1"], d["w3"], o["h"], self.sg, ws, g=o["g"], u=o["u"], stream=stream)
        B.linear_forward(o["h"], d["w2"], d["b2"], d["x"], o["y"], self.sl, ws, stream=stream)
        B.linear_backward(d["dy"], o["h"], d["w2"], None, o["dh"], o["dw2"], o["db2"], self.sl, ws, stream=stream)
        B.gated_backward(o["dh"], o["n"], d["w1"], d["w3"], o["g"], o["u"], o["dn"], o["dw1"], o["dw3"], self.sg, ws,
                         stream=stream)
        B.layer_norm_backward(o["dn"], d["x"], d["nw"], o["mean"], o["rstd"], o["dx"], o["dnw"], o["dnb"], self.sn,
                              ws, stream=stream)

    def forward64(self, x, **over):
        p = {k: v.double() for k, v in self.p.items()}
        p.update(over)
        m = x.mean(1, keepdim=True)
        n = (x - m) / torch.sqrt((x - m).square().mean(1, keepdim=True) + 1e-5) * p["nw"] + p["nb"]
        a, _ = act64(n @ p["w1"].T, self.act)
        return x + (a * (n @ p["w3"].T)) @ p["w2"].T + p["b2"]


@pytest.mark.parametrize("dtype", ("bf16", "f32"))
@pytest.mark.parametrize("size", [(1, 64, 128), (37, 136, 200), (300, 256, 520)], ids=small)
def test_block_against_64_bits(size, dtype):
    """The run of all six calls against autograd in 64 bits.  Up to six values rounded to the
    layer's type lie between an input and a gradient (n, g and u, h, dh, dn, the gradient), each
    entering through factors whose effect on the gradient's norm is about that of the value
    itself: 8 u of the norm bounds them for the quantities' 2-norms.  In fp32 the sums of up
    to 520 products take the place of the roundings: 64 u."""
    T, H, I = size
    b = Block(T, H, I, dtype, 40 + T)
    b.run()
    leaves = {k: v.double().requires_grad_() for k, v in b.p.items()}
    x = b.x.double().requires_grad_()
    y = b.forward64(x, **leaves)
    y.backward(b.dy.double())
    bound = 8 * U["bf16"] if dtype == "bf16" else 64 * U32
    ref = dict(y=y.detach(), dnw=leaves["nw"].grad, dnb=leaves["nb"].grad, dw1=leaves["w1"].grad,
               dw3=leaves["w3"].grad, dw2=leaves["w2"].grad, db2=leaves["b2"].grad,
               dx=x.grad - b.dy.double())          # the residual's share is dy itself
    for k, r in ref.items():
        err = float((b.o[k].cpu().double() - r).norm() / r.norm())
        assert err <= bound, (k, err)


def test_block_gradients_against_differences():
    """<gradient, v> against the central difference of the 64-bit block along v (step 1e-4: its
    own error is of the order 1e-8); the fp32 gradients are within 64 u of the 64-bit ones."""
    b = Block(19, 72, 104, "f32", 91, act="gelu_tanh")
    b.run()
    gen = torch.Generator().manual_seed(3)
    dy = b.dy.double()

    def loss(x=None, **over):
        return float((b.forward64(b.x.double() if x is None else x, **over) * dy).sum())

    for leaf, grad in (("nw", "dnw"), ("nb", "dnb"), ("w1", "dw1"), ("w3", "dw3"), ("w2", "dw2"), ("b2", "db2"), ("x", "dx")):
        p = (b.x if leaf == "x" else b.p[leaf]).double()
        v = torch.empty(p.shape, dtype=torch.float64).normal_(generator=gen)
        h = 1e-4
        diff = (loss(**{leaf: p + h * v}) - loss(**{leaf: p - h * v})) / (2 * h)
        got = b.o[grad].cpu().double() + (dy if leaf == "x" else 0)
        assert abs(float((got * v).sum()) - diff) <= 64 * U32 * float(got.norm() * v.norm()) + 1e-6 * abs(diff), leaf


def test_block_in_a_graph_replays_like_eager():
    """Captured once, replayed with new inputs and with eager work between: every replay gives
    the eager calls' bits."""
    b = Block(130, 136, 264, "bf16", 17)
    b.run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b.run()
    for k in range(4):
        gen = torch.Generator().manual_seed(100 + k)
        b.d["x"].copy_(rand(gen, 130, 136))
        b.d["dy"].copy_(rand(gen, 130, 136))
        b.run()
        want = {n: t.clone() for n, t in b.o.items()}
        for t in b.o.values():
            t.fill_(float("nan"))
        b.ws.fill_(0xFF)
        graph.replay()
        torch.cuda.synchronize()
        for n, t in b.o.items():
            assert torch.equal(t, want[n]), (k, n)


def test_two_streams_at_once():
    """Two blocks on two streams, each with its workspace, at the same time: the bits each has alone."""
    one, two = Block(200, 264, 328, "bf16", 5), Block(90, 128, 1000, "bf16", 6)
    want = []
    for b in (one, two):
        b.run()
        torch.cuda.synchronize()
        want.append({n: t.clone() for n, t in b.o.items()})
        for t in b.o.values():
            t.zero_()
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(5):
        one.run(stream=s1)
        two.run(stream=s2)
    torch.cuda.synchronize()
    for b, w in zip((one, two), want):
        for n, t in b.o.items():
            assert torch.equal(t, w[n]), n


def test_binding_refuses_strided_tensors():
    s = B.dense_shape(4, 16, 8, dtype="f32")
    x, w = torch.zeros(4, 32, device=DEV)[:, ::2], torch.zeros(8, 16, device=DEV)
    with pytest.raises(B.MoeError, match="dense row-major"):
        B.linear_forward(x, w, None, None, torch.zeros(4, 8, device=DEV), s, None)
    with pytest.raises(B.MoeError, match="dense row-major"):
        B.linear_forward(w.T.contiguous().T[:4], w, None, None, torch.zeros(4, 8, device=DEV), s, None)


def test_rows_past_32_bit_offsets():
    """A tensor of more than 2^31 elements: the last rows are computed like the first."""
    T, H = 300001, 8192
    x = torch.empty(T, H, dtype=torch.bfloat16, device=DEV)
    x[:] = torch.linspace(-2, 3, H, device=DEV).bfloat16()
    x[-1] = torch.linspace(1, -5, H, device=DEV).bfloat16()
    w = torch.full((H,), 0.5, dtype=torch.bfloat16, device=DEV)
    y = torch.empty_like(x)
    B.layer_norm_forward(x, w, None, y, B.norm_shape(T, H))
    few = torch.cat([x[:1], x[-1:]])
    want = torch.empty_like(few)
    B.layer_norm_forward(few, w, None, want, B.norm_shape(2, H))
    assert torch.equal(y[0], want[0]) and torch.equal(y[-1], want[1]) and torch.equal(y[T // 2], want[0])
