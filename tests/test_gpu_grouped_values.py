"""Expert and integer products at values where a factor, a term or a rounding could show, against 64 bits."""
import pytest
import torch

from routing_dispatch_expert_logits_amd import binding as B
from tests.test_gpu_dense import TYPES, U, U32, act64, fsum, out, rand
from tests.test_gpu_dense_values import same_kind
from tests.test_gpu_grouped import DEV, bad_rows, close, groups, offsets_of, random_codes, rows_left, skewed, ws_for

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


def name_of(case):
    return f"{len(case[0])}experts-{sum(case[0])}rows-{case[3]}x{case[4]}" if isinstance(case, tuple) else None


def gated_backward(case, act, grad):
    """Inputs (x, dh, g, u, w1, w3) on the GPU, the offsets, and dx, dw1, dw3 of a bf16 layer."""
    counts, before, behind, K, N = case
    off = offsets_of(counts, before)
    R, E = int(off[-1]) + behind, len(counts)
    gen = torch.Generator().manual_seed(R + N)
    x, dh, g, u = (bad_rows(rand(gen, R, n), off).to(DEV) for n in (K, N, N, N))
    w1, w3 = (rand(gen, E, N, K, std=0.05).to(DEV) for _ in range(2))
    s = B.grouped_shape(R, K, N, E, act=act, grad_dtype=grad)
    dx, dw1, dw3 = out((R, K), "bf16"), out((E, N, K), grad), out((E, N, K), grad)
    B.grouped_gated_backward(dh, x, off.to(DEV), w1, w3, g, u, dx, dw1, dw3, s, ws_for(s, B.MOE_CALL_GROUPED_GATED_BACKWARD))
    rows_left(dx, off, "dx")
    return (x, dh, g, u, w1, w3), off, (dx, dw1, dw3)


# both products in one launch, a cut contraction, and the tiles of 128, 256 and 320 rows
@pytest.mark.parametrize("act", ("relu", "none"))
@pytest.mark.parametrize("case", (([5, 0, 3], 2, 4, 72, 40), ([64, 1, 0, 130, 63], 0, 0, 129, 97), ([40, 1, 0, 70], 0, 5, 100, 2048),
                                  (skewed(32, 8200, 3), 0, 0, 1024, 768), ([1900, 0, 300, 1950], 0, 3, 1104, 1544)), ids=name_of)
def test_gated_gradients_round_their_operands_once(case, act):
    """dg and du as bf16 operands of the products, and nothing else between the definition and the gradients but fp32
    sums and the last rounding.  With slopes of 0 and 1 dg is a product of two bf16 numbers, exact in fp32, so its
    rounding is known."""
    (x, dh, g, u, w1, w3), off, (dx, dw1, dw3) = gated_backward(case, act, "bf16")
    on = (g > 0).float() if act == "relu" else 1.0
    dg = (dh.float() * u.float() * on).bfloat16().double()
    du = (dh.float() * (g.float().clamp(min=0) if act == "relu" else g.float())).bfloat16().double()
    N, r = case[4], U["bf16"]
    for e, k in groups(off):
        X, A, C, W1, W3 = x[k].double(), dg[k], du[k], w1[e].double(), w3[e].double()
        ref = A @ W1 + C @ W3
        close("dx", dx[k], "bf16", ref, r * ref.abs() + 2 * (fsum(A, W1.T, 2 * N) + fsum(C, W3.T, 2 * N)))
        for name, got, d in (("dw1", dw1, A), ("dw3", dw3, C)):
            ref = d.T @ X
            close(name, got[e], "bf16", ref, r * ref.abs() + 2 * fsum(d.T, X.T, k.stop - k.start))


# weight gradients on tiles of 256 x 256 (the last: 128 x 256) with three terms to each operand, widths that end inside tiles
# and chunks
@pytest.mark.parametrize("case", (([1900, 0, 300, 1950], 3, 5, 4101, 1543), (skewed(31, 8200, 8) + [0], 0, 0, 1021, 771),
                                  ([2100, 0, 4000, 300], 0, 9, 520, 1096)), ids=name_of)
def test_fp32_gradients_of_large_bf16_layers(case):
    """Three bf16 terms hold dg and du: fp32 weight gradients are within fp32's roundings of the definition, and an expert
    without rows has zeros."""
    (x, dh, g, u, w1, w3), off, (dx, dw1, dw3) = gated_backward(case, "silu", "f32")
    r, N, rows = U32, case[4], dict(groups(off))
    for e in range(len(case[0])):
        if e not in rows:
            assert dw1[e].eq(0).all() and dw3[e].eq(0).all()
            continue
        k = rows[e]
        X, D, G, V, W1, W3 = (t.double() for t in (x[k], dh[k], g[k], u[k], w1[e], w3[e]))
        a, slope = act64(G, "silu")
        dg, du, fe = D * V * slope, D * a, 2.0 ** -18 * (1 + G.abs())
        eg, eu, b = fe * (D * V).abs(), fe * (D * G).abs(), U["bf16"]
        for name, got, d, err in (("dw1", dw1, dg, eg), ("dw3", dw3, du, eu)):
            ref = d.T @ X
            close(name, got[e], "f32", ref, r * ref.abs() + (r * d.abs() + err).T @ X.abs() + 2 * fsum(d.T, X.T, 3 * (k.stop - k.start)))
        ref = dg @ W1 + du @ W3
        close("dx", dx[k], "bf16", ref, b * ref.abs() + (b * dg.abs() + eg) @ W1.abs() + (b * du.abs() + eu) @ W3.abs()
              + 2 * (fsum(dg, W1.T, 2 * N) + fsum(du, W3.T, 2 * N)))


@pytest.mark.parametrize("grad", ("bf16", "f32"))
@pytest.mark.parametrize("act", ("silu", "relu"))
@pytest.mark.parametrize("case", (([70, 0, 30], 1, 2, 41, 130), ([1900, 0, 300, 1950], 0, 3, 1100, 1544)), ids=name_of)
def test_infinite_inputs_stay_with_their_expert(case, act, grad):
    """dw[e] = sum dz x over the rows of e is infinite where one x of the column is, NaN where x is or where infinities of
    both signs meet, and finite for the other experts; the terms that hold dz in fp32 have other signs and zeros among them."""
    counts, before, behind, K, N = case
    off = offsets_of(counts, before)
    R, E = int(off[-1]) + behind, len(counts)
    gen = torch.Generator().manual_seed(R + K)
    x, dh, g, u = (rand(gen, R, n) for n in (K, N, N, N))
    g = g.abs() + 0.25                                  # no slope and no value is 0
    r = int(off[2])                                     # the third expert's first rows
    x[r + 1, 3], x[r + 2, 5], x[r, 7], x[r + 2, 7], x[r + 1, 9] = (float(v) for v in ("inf", "-inf", "inf", "inf", "nan"))
    x, dh, g, u = (bad_rows(t, off).to(DEV) for t in (x, dh, g, u))
    w = rand(gen, E, N, K).to(DEV)
    s = B.grouped_shape(R, K, N, E, act=act, grad_dtype=grad)
    dx, dw1, dw3 = out((R, K), "bf16"), out((E, N, K), grad), out((E, N, K), grad)
    B.grouped_gated_backward(dh, x, off.to(DEV), w, w, g, u, dx, dw1, dw3, s, ws_for(s, B.MOE_CALL_GROUPED_GATED_BACKWARD))
    for name, got, first in (("dw1", dw1, True), ("dw3", dw3, False)):
        got = got.view(torch.bfloat16) if grad == "bf16" else got
        assert torch.isfinite(got[[e for e in range(E) if e != 2]]).all(), name
        k = slice(r, int(off[3]))
        a, slope = act64(g[k].double(), act)
        d = dh[k].double() * (u[k].double() * slope if first else a)
        assert not d[:3].eq(0).any()
        same_kind(name, got[2].cpu().double(), (d.T @ x[k].double()).cpu())
    v = slice(int(off[0]), int(off[-1]))                # dx does not read x
    assert torch.isfinite(dx.view(torch.bfloat16)[v]).all()
