"""Expert and integer products at values where a factor, a term or a rounding could show, against 64 bits."""
import pytest
import torch

from routing_dispatch_expert_logits_amd import binding as B
from tests.test_gpu_dense import TYPES, U, U32, out, rand
from tests.test_gpu_grouped import DEV, groups, offsets_of, random_codes, rows_left, skewed, ws_for

pytestmark = pytest.mark.gpu


def scales(gen, lo, hi, *shape):
    """fp32 numbers between 2^lo and 2^(hi + 1), spread over the exponents."""
    e = torch.randint(lo, hi + 1, shape, generator=gen).double()
    return (torch.exp2(e) * (1 + torch.rand(shape, generator=gen).double())).float()


def ranged(name, got, dtype, ref, tol):
    """Within tol and half a step of the smallest numbers where the definition is well inside the type's range, an
    infinity of its sign where it is beyond, and never NaN."""
    got = (got.view(torch.bfloat16) if dtype == "bf16" else got).double()
    assert not got.isnan().any(), f"{name}: NaN in {int(got.isnan().sum())} of {got.numel()}"
    inf, fin = ref.abs() > 2.0 ** 129, ref.abs() < 2.0 ** 127
    assert torch.equal(got[inf], ref[inf].sign() * float("inf")), name
    over = ((got - ref).abs() - tol - 2.0 ** -149 - (2.0 ** -134 if dtype == "bf16" else 0.0))[fin]
    assert bool((over <= 0).all()), f"{name}: {int((over > 0).sum())} of {int(fin.sum())}, {float(over.max()):.3e} over"


def coded(gen, *shape):
    return random_codes(gen, *shape)[0].to(DEV)


# decoding steps, and tiles of 64, 256 x 128 (the gated product: 256 x 256), 256 x 256, and those with columns left for smaller ones
@pytest.mark.parametrize("dtype", ("bf16", "f32"))
@pytest.mark.parametrize("size", ((12, 200, 77), (40, 200, 77), (2000, 300, 3000), (4096, 200, 4000), (8000, 200, 2100)), ids=str)
def test_int8_scales_of_any_size(size, dtype):
    """row_scale col_scale sum(q q) is its value, whichever of the scales is large or small: rows whose scale times
    the sum is beyond fp32's largest number (scales are up to 2^121) have a finite product with a small column
    scale.  Three factors: two roundings, a third for the sum."""
    T, K, N = size
    gen = torch.Generator().manual_seed(sum(size))
    x, w, w3 = coded(gen, T, K), coded(gen, N, K), coded(gen, N, K)
    x[3] = 0
    sx, sw = scales(gen, -149, 120, T).to(DEV), scales(gen, -149, 120, N).to(DEV)
    sx[::7] = 2.0 ** 121 * 127 / 128
    sx[5], x[5] = float("nan"), 0
    sound = torch.arange(T, device=DEV) != 5
    bias, res = (rand(gen, *s, dtype=dtype).to(DEV) for s in ((N,), (T, N)))
    z = (x.double() @ w.double().T) * sx.double()[:, None] * sw.double()
    s = B.dense_shape(T, K, N, dtype=dtype)
    y = out((T, N), dtype)
    B.linear_int8_forward(x, sx, w, sw, None, None, y, s)
    ranged("y", y[sound], dtype, z[sound], ((U[dtype] + 4 * U32) * z.abs())[sound])
    assert TYPES[dtype] == torch.float32 or y.view(torch.bfloat16)[5].isnan().all()
    B.linear_int8_forward(x, sx, w, sw, bias, res, y, s)
    ref = z + bias.double() + res.double()
    parts = z.abs() + bias.double().abs() + res.double().abs()
    ranged("y with bias and residual", y[sound], dtype, ref[sound], (U[dtype] * ref.abs() + 8 * U32 * parts)[sound])
    # both projections of rows of large scales: 2^97 .. 2^121 by 2^-118 .. 2^-109
    sx, s1, s3 = scales(gen, 97, 120, T).to(DEV), scales(gen, -118, -110, N).to(DEV), scales(gen, -118, -110, N).to(DEV)
    h = out((T, N), dtype)
    B.gated_int8_forward(x, sx, w, s1, w3, s3, h, s)
    g, u = ((x.double() @ a.double().T) * sx.double()[:, None] * b.double() for a, b in ((w, s1), (w3, s3)))
    ranged("h", h, dtype, g * u, (U[dtype] + 8 * U32) * (g * u).abs())


# decoding steps, tiles of 64, of 64 x 128 (many experts), of 128 and of 320 rows
@pytest.mark.parametrize("dtype", ("bf16", "f32"))
@pytest.mark.parametrize("case", (([3, 0, 8, 2], 1, 2, 200, 77), ([64, 1, 0, 130, 63], 0, 5, 128, 96), (skewed(52, 800, 1), 0, 0, 333, 2477),
                                  (skewed(32, 4100, 2), 0, 0, 260, 1030), ([3000, 0, 2900, 3100], 0, 0, 2049, 2056)),
                         ids=lambda c: f"{len(c[0])}experts-{sum(c[0])}rows-{c[3]}x{c[4]}")
def test_grouped_int8_scales_of_any_size(case, dtype):
    counts, before, behind, K, N = case
    off = offsets_of(counts, before)
    R, E = int(off[-1]) + behind, len(counts)
    gen = torch.Generator().manual_seed(R + K)
    x, w, w3 = coded(gen, R, K), coded(gen, E, N, K), coded(gen, E, N, K)
    sx, sw = scales(gen, -149, 120, R).to(DEV), scales(gen, -149, 120, E, N).to(DEV)
    sx[::7] = 2.0 ** 121 * 127 / 128
    sg, s1, s3 = scales(gen, 97, 120, R).to(DEV), scales(gen, -118, -110, E, N).to(DEV), scales(gen, -118, -110, E, N).to(DEV)
    y, h, doff, s = out((R, N), dtype), out((R, N), dtype), off.to(DEV), B.grouped_shape(R, K, N, E, dtype=dtype)
    B.grouped_linear_int8_forward(x, sx, doff, w, sw, y, s, ws_for(s, B.MOE_CALL_GROUPED_LINEAR_INT8))
    B.grouped_gated_int8_forward(x, sg, doff, w, s1, w3, s3, h, s, ws_for(s, B.MOE_CALL_GROUPED_GATED_INT8))
    rows_left(y, off, "y")
    rows_left(h, off, "h")
    for e, r in groups(off):
        X = x[r].double()
        z = (X @ w[e].double().T) * sx[r].double()[:, None] * sw[e].double()
        ranged("y", y[r], dtype, z, (U[dtype] + 4 * U32) * z.abs())
        g, u = ((X @ a[e].double().T) * sg[r].double()[:, None] * b[e].double() for a, b in ((w, s1), (w3, s3)))
        ranged("h", h[r], dtype, g * u, (U[dtype] + 8 * U32) * (g * u).abs())
