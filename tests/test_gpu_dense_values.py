"""Dense operators at values where a rounding, a term or a padding column could show, against 64 bits."""
import math

import pytest
import torch

from routing_dispatch_expert_logits_amd import binding as B
from tests.test_gpu_dense import DEV, U, f64, out, ws_for

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
