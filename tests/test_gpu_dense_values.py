"""Dense operators at values where a rounding, a term or a padding column could show, against 64 bits."""
import math

import pytest
import torch

from routing_dispatch_expert_logits_amd import binding as B
from tests.test_gpu_dense import DEV, U, act64, f64, out, rand, ws_for

pytestmark = pytest.mark.gpu


def every_bf16(lo, hi):
    """Every bf16 number of [lo, hi] and its negative."""
    bits = torch.arange(0, 0x7f80, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    bits = bits[(bits.double() >= lo) & (bits.double() <= hi)]
    return torch.cat((bits, -bits))


def through_act(z, act):
    """act(z) and act'(z) as a [T x 1] layer with weight 1 gives them, its one product being exact."""
    T = z.numel()
    z = z.view(T, 1).to(DEV)
    s = B.dense_shape(T, 1, 1, dtype="bf16", act=act)
    one = torch.ones(1, 1, dtype=torch.bfloat16, device=DEV)
    y, dx = out((T, 1), "bf16"), out((T, 1), "bf16")
    B.linear_forward(z, one, None, None, y, s, ws_for(s, B.MOE_CALL_LINEAR_FORWARD))
    B.linear_backward(torch.ones_like(z), None, one, z, dx, None, None, s, ws_for(s, B.MOE_CALL_LINEAR_BACKWARD))
    return f64(y, "bf16")[:, 0], f64(dx, "bf16")[:, 0]


@pytest.mark.parametrize("rows", (16, 1 << 20))
def test_gelu_tail(rows):
    """GELU and its slope are within their rounding down to where they leave bf16's normal range
    (a = -13.1), not only against |a|: the normal mass is within 2^-13 of itself; e^(-a^2 / 2) within
    2^-16 (its exponent, at most 124, rounded three times at 2^-24) and the reciprocal, the sums and
    products of up to 10 terms within 2^-20.  The slope's two parts, of opposite signs, count apart."""
    z = every_bf16(2.0 ** -20, 13.0)[::1 if rows > 16 else 2]
    y, dx = map(torch.cat, zip(*(through_act(v, "gelu") for v in z.split(rows))))
    z = z.double()
    rel = 2.0 ** -13 + 2.0 ** -16 + 2.0 ** -20
    # by erfc: torch's ndtr is (1 + erf) / 2, whose rounding at 2^-53 is all that is left of the tail
    # from a = -8.3 on
    mass, bell = torch.erfc(-z * math.sqrt(0.5)) / 2, z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    small = torch.erfc(z.abs() * math.sqrt(0.5)) / 2   # a positive argument's mass is 1 less that of its negative
    a, slope = z * mass, mass + bell
    over = (y - a).abs() - (U["bf16"] * a.abs() + z.abs() * (rel * small + 2.0 ** -23))
    neg = z < 0
    over[neg] = ((y - a).abs() - (U["bf16"] + rel) * a.abs())[neg]
    assert bool((over <= 0).all()), (float(over.max()), z[over.argmax()])
    tol = U["bf16"] * slope.abs() + rel * (small + bell.abs()) + torch.where(neg, 0.0, 2.0 ** -23)
    over = (dx - slope).abs() - 2 * tol        # rounded twice: before the product with w, and after
    assert bool((over <= 0).all()), (float(over.max()), z[over.argmax()])


def same_kind(name, got, ref):
    """NaN, infinities of either sign and finite numbers where ref has them."""
    assert torch.equal(got.isnan(), ref.isnan()), f"{name}: NaN in {int(got.isnan().sum())} of {got.numel()}, expected {int(ref.isnan().sum())}"
    inf = ref.isinf()
    assert torch.equal(got.isinf(), inf) and torch.equal(got[inf], ref[inf]), name


@pytest.mark.parametrize("dtype,grad", (("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")))
@pytest.mark.parametrize("act", ("silu", "gelu", "gelu_tanh", "relu", "none"))
@pytest.mark.parametrize("size", ((3, 40, 24), (70, 41, 130), (300, 1000, 264)), ids=lambda s: "x".join(map(str, s)))
def test_infinite_inputs_give_infinite_weight_gradients(size, act, dtype, grad):
    """dw = sum_t dz x is infinite where one x of the column is, and NaN where x is or where infinities
    of both signs meet; the terms that hold a dz in fp32 have other signs and zeros among them."""
    T, K, N = size
    gen = torch.Generator().manual_seed(T + K)
    dy, x, g, u, w = (rand(gen, *s, dtype=dtype) for s in ((T, N), (T, K), (T, N), (T, N), (N, K)))
    g = g.abs() + 0.25                                  # no slope and no value is 0
    x[1, 3], x[2, 5], x[0, 7], x[2, 7], x[1, 9] = (float(v) for v in ("inf", "-inf", "inf", "inf", "nan"))
    s = B.dense_shape(T, K, N, dtype=dtype, act=act, grad_dtype=grad)
    dev = [t.to(DEV) for t in (dy, x, g, u, w)]
    dw, dw1, dw3 = (out((N, K), grad) for _ in range(3))
    B.linear_backward(dev[0], dev[1], None, dev[2] if act != "none" else None, None, dw, None, s,
                      ws_for(s, B.MOE_CALL_LINEAR_BACKWARD))
    dx = out((T, K), dtype)
    B.gated_backward(dev[0], dev[1], dev[4], dev[4], dev[2], dev[3], dx, dw1, dw3, s, ws_for(s, B.MOE_CALL_GATED_BACKWARD))
    dy, x, g, u, w = (t.double() for t in (dy, x, g, u, w))
    a, slope = act64(g, act)
    for name, got, d in (("dw", dw, dy * slope), ("dw1", dw1, dy * u * slope), ("dw3", dw3, dy * a)):
        assert not d[:3].eq(0).any()
        same_kind(name, f64(got, grad), d.T @ x)
    assert torch.isfinite(f64(dx, dtype)).all()         # dx does not read x


def test_terms_of_the_largest_gradients():
    """A gradient before the activation between the largest bf16 number and the largest fp32 one is
    finite: 129/128 times 254/128 2^127 is 1.99988 2^127, which rounds to infinity in bf16 (from
    1.99609 2^127 on).  With x = 2^-10 its weight gradient is exact in fp32, like dh act(g)'s."""
    dh, g, u, x = 129 / 128, 1.0, 254 / 128 * 2.0 ** 127, 2.0 ** -10
    s = B.dense_shape(1, 1, 1, act="none", grad_dtype="f32")
    dev = [torch.full((1, 1), v, dtype=torch.bfloat16, device=DEV) for v in (dh, x, 1.0, 1.0, g, u)]
    for sign in (1, -1):
        dw1, dw3 = out((1, 1), "f32"), out((1, 1), "f32")
        B.gated_backward(dev[0] * sign, *dev[1:], None, dw1, dw3, s, ws_for(s, B.MOE_CALL_GATED_BACKWARD))
        assert f64(dw1, "f32").item() == sign * dh * u * x and f64(dw3, "f32").item() == sign * dh * x
    inf = torch.full((1, 1), float("inf"), dtype=torch.bfloat16, device=DEV)
    B.gated_backward(inf, *dev[1:], None, dw1, dw3, s, ws_for(s, B.MOE_CALL_GATED_BACKWARD))
    assert f64(dw1, "f32").item() == f64(dw3, "f32").item() == float("inf")


def test_binding_refuses_strided_workspaces():
    s = B.dense_shape(4, 16, 8, act="silu")
    x, w, y = (torch.zeros(sh, dtype=torch.bfloat16, device=DEV) for sh in ((4, 16), (8, 16), (4, 8)))
    for dtype in (torch.float32, torch.uint8):
        with pytest.raises(B.MoeError, match="ws: not dense row-major"):
            B.linear_backward(y, x, w, y, torch.empty_like(x), None, None, s,
                              torch.zeros(1 << 20, dtype=dtype, device=DEV)[::2])


@pytest.mark.parametrize("dtype", ("bf16", "f32"))
@pytest.mark.parametrize("H", (100, 500, 1021, 8200, 20001))
def test_norm_gradient_of_a_far_constant_row(H, dtype):
    """A constant row has n = 0 and dx = rstd (e - mean(e)), however far it lies: mean times rstd
    overflows here, and the columns that fill a row up to whole chunks and waves have no part in it."""
    far = 2.0 ** 126 / 2 ** math.ceil(math.log2(H))     # the row's sum is below 2^127
    eps = 2.0 ** -50                                    # rstd 2^25
    gen = torch.Generator().manual_seed(H)
    x, w, dy = rand(gen, 3, H, dtype=dtype), rand(gen, H, dtype=dtype), rand(gen, 3, H, dtype=dtype)
    x[1] = far
    s = B.norm_shape(3, H, eps=eps, dtype=dtype)
    y, dx, dw, db = out((3, H), dtype), out((3, H), dtype), out((H,), dtype), out((H,), dtype)
    mean, rstd = out((3,), "f32"), out((3,), "f32")
    dev = [t.to(DEV) for t in (x, w, dy)]
    B.layer_norm_forward(dev[0], dev[1], None, y, s, mean=mean, rstd=rstd)
    assert mean[1].item() == far and rstd[1].item() == 2.0 ** 25 and f64(y, dtype)[1].eq(0).all()
    B.layer_norm_backward(dev[2], dev[0], dev[1], mean, rstd, dx, dw, db, s, ws_for(s))
    e = (dy.double() * w.double())[1]
    ref = 2.0 ** 25 * (e - e.mean())
    # e, its mean of H terms (at most 16 + H / 64 additions deep), their difference and its product
    tol = U[dtype] * ref.abs() + 2.0 ** 25 * 2.0 ** -24 * (4 * e.abs() + (20 + H // 64) * e.abs().mean())
    got = f64(dx, dtype)
    assert bool(((got[1] - ref).abs() <= tol).all()) and torch.isfinite(got).all(), float((got[1] - ref).abs().max())
    assert torch.isfinite(f64(dw, dtype)).all()
