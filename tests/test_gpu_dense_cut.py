"""Dense products whose output columns are cut into two launches, and tensors of more than 2^31
elements, against 64 bits.  Tolerances as in tests/test_gpu_dense.py; the large tensors hold small
whole numbers, whose products and sums are exact in every order.
"""
import pytest
import torch

from routing_dispatch_expert_logits_amd import binding as B
from tests import test_gpu_dense as test_dense
from tests.dense_sizes import CUT_BACKWARD, CUT_FORWARD
from tests.test_gpu_dense import ACTS, DEV, SLOPE, TYPES, U, U32, act64, close, framed, fsum, out, rand, small, ws_for

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("act,grad", (("none", "bf16"), ("none", "f32"), ("silu", "bf16"), ("gelu_tanh", "f32")))
@pytest.mark.parametrize("size", CUT_BACKWARD, ids=small)
def test_cut_linear_backward(size, act, grad):
    T, K, N = size
    gen = torch.Generator().manual_seed(K)
    x, w, dy, z = (framed(rand(gen, *s, std=v)) for s, v in (((T, K), 1), ((N, K), 0.05), ((T, N), 1), ((T, N), 1.7)))
    s = B.dense_shape(T, K, N, act=act, grad_dtype=grad)
    dx, dw, db = out((T, K), "bf16"), out((N, K), grad), out((N,), grad)
    B.linear_backward(dy, x, w, z if act != "none" else None, dx, dw, db, s, ws_for(s, B.MOE_CALL_LINEAR_BACKWARD))
    x, w, dy, z = (t.double() for t in (x, w, dy, z))
    dz = dy * act64(z, act)[1]
    r = U["bf16"] if act != "none" else 0.0
    e = 2.0 ** -18 * (1 + z.abs()) * dy.abs() if act != "none" else 0.0 * dy
    ref = dz @ w
    close("dx", dx, "bf16", ref, U["bf16"] * ref.abs() + (r * dz.abs() + e) @ w.abs() + 2 * fsum(dz, w.T, N))
    ref = dz.T @ x
    close("dw", dw, grad, ref, U[grad] * ref.abs() + (min(r, U[grad]) * dz.abs() + e).T @ x.abs() + 2 * fsum(dz.T, x.T, 3 * T))
    ref = dz.sum(0)
    close("dbias", db, grad, ref, U[grad] * ref.abs() + e.sum(0) + (T + 8) * U32 * dz.abs().sum(0))


@pytest.mark.parametrize("act,grad", (("silu", "bf16"), ("relu", "f32"), ("gelu", "f32")))
@pytest.mark.parametrize("size", CUT_BACKWARD, ids=small)
def test_cut_gated_backward(size, act, grad):
    T, K, N = size
    gen = torch.Generator().manual_seed(K + 1)
    x, dh, w1, w3, g, u = (framed(rand(gen, *s, std=v)) for s, v in (
        ((T, K), 1), ((T, N), 1), ((N, K), 0.05), ((N, K), 0.05), ((T, N), 1.7), ((T, N), 1.7)))
    s = B.dense_shape(T, K, N, act=act, grad_dtype=grad)
    dx, dw1, dw3 = out((T, K), "bf16"), out((N, K), grad), out((N, K), grad)
    B.gated_backward(dh, x, w1, w3, g, u, dx, dw1, dw3, s, ws_for(s, B.MOE_CALL_GATED_BACKWARD))
    x, dh, w1, w3, g, u = (t.double() for t in (x, dh, w1, w3, g, u))
    a, slope = act64(g, act)
    dg, du = dh * u * slope, dh * a
    fe = 2.0 ** -18 * (1 + g.abs())
    eg, eu = fe * (dh * u).abs(), fe * (dh * g).abs()
    r, rw = U["bf16"], U[grad]
    ref = dg @ w1 + du @ w3
    close("dx", dx, "bf16", ref, r * ref.abs() + (r * dg.abs() + eg) @ w1.abs() + (r * du.abs() + eu) @ w3.abs()
          + 2 * (fsum(dg, w1.T, 2 * N) + fsum(du, w3.T, 2 * N)))
    for name, got, d, e in (("dw1", dw1, dg, eg), ("dw3", dw3, du, eu)):
        ref = d.T @ x
        close(name, got, grad, ref, rw * ref.abs() + (rw * d.abs() + e).T @ x.abs() + 2 * fsum(d.T, x.T, 3 * T))


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("size", CUT_FORWARD, ids=small)
def test_cut_linear_forward_in_place(size, act):
    """Both launches of a cut product with all that their epilogues read and write; y in place of
    its residual has the same bits."""
    T, K, N = size
    gen = torch.Generator().manual_seed(N)
    x, w, bias, res = (framed(rand(gen, *s, std=v)) for s, v in (((T, K), 1), ((N, K), 0.05), ((N,), 1), ((T, N), 1)))
    s = B.dense_shape(T, K, N, act=act)
    ws = ws_for(s, B.MOE_CALL_LINEAR_FORWARD)
    y, z, y2, z2 = (out((T, N), "bf16") for _ in range(4))
    B.linear_forward(x, w, bias, res, y, s, ws, z=z)
    y2.copy_(res.view(y2.dtype))
    B.linear_forward(x, w, bias, y2, y2, s, ws, z=z2)
    assert torch.equal(y, y2) and torch.equal(z, z2)
    x, w, bias, res = (t.double() for t in (x, w, bias, res))
    rz = x @ w.T + bias
    ez = 2 * fsum(x, w, K) + U32 * rz.abs()
    a, _ = act64(rz, act)
    r = U["bf16"]
    close("z", z, "bf16", rz, r * rz.abs() + 2 * ez)
    close("y", y, "bf16", a + res, r * (a + res).abs() + SLOPE * ez + 2.0 ** -20 * (1 + rz.abs()) * rz.abs()
          + 2 * U32 * (a + res).abs())


# more than 2^31 elements in [T x N]
FAR = (1048579, 8, 2056)


def ones(gen, *shape, dtype="bf16"):
    """-1, 0 and 1."""
    return torch.randint(-1, 2, shape, generator=gen, device=DEV, dtype=torch.int8).to(TYPES[dtype])


def rows(T, step=1 << 16):
    return [slice(t, min(T, t + step)) for t in range(0, T, step)]


@pytest.mark.parametrize("dtype", ("bf16", "f32"))
def test_linear_past_32_bit_offsets(dtype):
    T, K, N = FAR
    gen = torch.Generator(device=DEV).manual_seed(1)
    x, w, res = ones(gen, T, K, dtype=dtype), ones(gen, N, K, dtype=dtype), ones(gen, T, N, dtype=dtype)
    s = B.dense_shape(T, K, N, dtype=dtype, act="relu", grad_dtype="f32")
    y, z = torch.empty_like(res), torch.empty_like(res)
    B.linear_forward(x, w, None, res, y, s, None, z=z)
    for t in rows(T):
        want = x[t].float() @ w.float().T
        assert torch.equal(z[t].float(), want), t
        assert torch.equal(y[t].float(), want.clamp(min=0) + res[t].float()), t
    del y
    # res as the gradient of y
    dx, dw, db = torch.empty_like(x), torch.empty(N, K, device=DEV), torch.empty(N, device=DEV)
    ws = torch.empty(B.dense_workspace_bytes(s, B.MOE_CALL_LINEAR_BACKWARD), dtype=torch.uint8, device=DEV)
    B.linear_backward(res, x, w, z, dx, dw, db, s, ws)
    sw, sb = torch.zeros(N, K, device=DEV), torch.zeros(N, device=DEV)
    for t in rows(T):
        dz = torch.where(z[t] > 0, res[t].float(), 0.0)
        assert torch.equal(dx[t], (dz @ w.float()).to(dx.dtype)), t
        sw += dz.T @ x[t].float()
        sb += dz.sum(0)
    assert torch.equal(dw, sw) and torch.equal(db, sb)


def test_gated_past_32_bit_offsets():
    """In bf16 with fp32 gradients: two terms of two gradients, each past 2^31 elements."""
    T, K, N = FAR
    gen = torch.Generator(device=DEV).manual_seed(2)
    x, w1, w3, dh = ones(gen, T, K), ones(gen, N, K), ones(gen, N, K), ones(gen, T, N)
    s = B.dense_shape(T, K, N, act="relu", grad_dtype="f32")
    h, g, u = (torch.empty_like(dh) for _ in range(3))
    B.gated_forward(x, w1, w3, h, s, None, g=g, u=u)
    for t in rows(T):
        rg, ru = x[t].float() @ w1.float().T, x[t].float() @ w3.float().T
        assert torch.equal(g[t].float(), rg) and torch.equal(u[t].float(), ru), t
        assert torch.equal(h[t].float(), rg.clamp(min=0) * ru), t
    del h
    dx, dw1, dw3 = torch.empty_like(x), torch.empty(N, K, device=DEV), torch.empty(N, K, device=DEV)
    ws = torch.empty(B.dense_workspace_bytes(s, B.MOE_CALL_GATED_BACKWARD), dtype=torch.uint8, device=DEV)
    B.gated_backward(dh, x, w1, w3, g, u, dx, dw1, dw3, s, ws)
    s1, s3 = torch.zeros(N, K, device=DEV), torch.zeros(N, K, device=DEV)
    for t in rows(T):
        dg = torch.where(g[t] > 0, dh[t].float() * u[t].float(), 0.0)
        du = dh[t].float() * g[t].float().clamp(min=0)
        assert torch.equal(dx[t], (dg @ w1.float() + du @ w3.float()).to(dx.dtype)), t
        s1 += dg.T @ x[t].float()
        s3 += du.T @ x[t].float()
    assert torch.equal(dw1, s1) and torch.equal(dw3, s3)


# the largest row count, the largest widths, and decoding rows of them
@pytest.mark.parametrize("size", [(1 << 28, 1, 8), (40, 1 << 21, 24), (40, 24, 1 << 21), (4, 1 << 21, 24), (4, 24, 1 << 21)],
                         ids=small)
def test_largest_sizes(size):
    T, K, N = size
    gen = torch.Generator(device=DEV).manual_seed(3)
    x, w, dy = ones(gen, T, K), ones(gen, N, K), ones(gen, T, N)
    s = B.dense_shape(T, K, N, act="none", grad_dtype="f32")
    y, dx = torch.empty_like(dy), torch.empty_like(x)
    dw, db = torch.empty(N, K, device=DEV), torch.empty(N, device=DEV)
    ws = torch.empty(max(B.dense_workspace_bytes(s, c) for c in (B.MOE_CALL_LINEAR_FORWARD, B.MOE_CALL_LINEAR_BACKWARD)),
                     dtype=torch.uint8, device=DEV)
    B.linear_forward(x, w, None, None, y, s, ws)
    B.linear_backward(dy, x, w, None, dx, dw, db, s, ws)
    sw, sb = torch.zeros(N, K, device=DEV), torch.zeros(N, device=DEV)
    for t in rows(T, 1 << 24):
        assert torch.equal(y[t], (x[t].float() @ w.float().T).to(y.dtype)), t
        assert torch.equal(dx[t], (dy[t].float() @ w.float()).to(dx.dtype)), t
        sw += dy[t].float().T @ x[t].float()
        sb += dy[t].float().sum(0)
    assert torch.equal(dw, sw) and torch.equal(db, sb)


@pytest.mark.parametrize("dtype", ("bf16", "f32"))
def test_widest_norm(dtype):
    test_dense.test_norm_forward((3, 1 << 21), dtype)
    test_dense.test_norm_backward((3, 1 << 21), dtype, "f32")


@pytest.mark.parametrize("dtype,H", (("bf16", 8192), ("bf16", 20000), ("f32", 8200)))
def test_norm_gradient_past_32_bit_offsets(dtype, H):
    """dy is zero but in the first and the last row, which then give the column sums of a call on the
    two alone, and have its dx; the rows between have none.  dw is a sum of two products of dy and
    n = (x - mean) rstd: at most five roundings at 2^-24 each (x - mean, n, the product, which a fused
    multiply-add in a block of both rows leaves out, and the sum), of the terms' magnitudes."""
    T = (1 << 31) // H + 37
    gen = torch.Generator().manual_seed(H)
    few = [rand(gen, 2, H, dtype=dtype).to(DEV) for _ in range(2)]
    w = rand(gen, H, dtype=dtype).to(DEV)
    dy, x = (torch.zeros(T, H, dtype=TYPES[dtype], device=DEV) for _ in range(2))
    for big, two in zip((dy, x), few):
        big[0], big[-1] = two[0], two[1]
    grads = []
    for d, v in ((dy, x), few):
        rows_ = d.shape[0]
        s = B.norm_shape(rows_, H, dtype=dtype, grad_dtype="f32")
        mean, rstd = torch.zeros(rows_, device=DEV), torch.ones(rows_, device=DEV)
        mean[-1], rstd[0] = 0.25, 2.0
        o = [torch.empty_like(d), torch.empty(H, device=DEV), torch.empty(H, device=DEV)]
        ws = torch.empty(B.norm_workspace_bytes(s), dtype=torch.uint8, device=DEV)
        B.layer_norm_backward(d, v, w, mean, rstd, *o, s, ws)
        grads.append(o)
    (dx, dw, db), (dx2, dw2, db2) = grads
    assert torch.equal(dx[0], dx2[0]) and torch.equal(dx[-1], dx2[1])
    assert not any(bool(dx[1:-1][t].any()) for t in rows(T - 2))
    d, n = few[0].double(), (few[1].double() - mean.double()[:, None]) * rstd.double()[:, None]
    for got in (dw, dw2):
        assert bool(((got.double() - (d * n).sum(0)).abs() <= 5 * U32 * (d * n).abs().sum(0)).all())
    assert torch.equal(db, db2)
