"""Expert and integer products called as a serving loop calls them: in graphs replayed with other row counts, on streams at
once, and with as many experts as there may be."""
import pytest
import torch

from routing_dispatch_expert_logits_amd import binding as B
from tests import gpu_util as gu
from tests.test_gpu_dense import TYPES, U, act64, fsum, out, rand
from tests.test_gpu_grouped import DEV, close, groups, offsets_of, rows_left, ws_for

pytestmark = pytest.mark.gpu


class Served:
    """quantise, gated product, quantise, linear product of one expert layer, weights quantised once."""

    def __init__(self, R, E, H, I, dtype, seed):
        gen = torch.Generator().manual_seed(seed)
        self.R, self.E, self.H, self.dtype = R, E, H, dtype
        self.x, self.offsets = rand(gen, R, H, dtype=dtype).to(DEV), offsets_of([R // E] * E).to(DEV)

        def codes(*shape):
            t = rand(gen, *shape, dtype=dtype, std=shape[-1] ** -0.5).to(DEV)
            q = torch.empty(*shape[:-1], B.int8_row_bytes(shape[-1]), dtype=torch.int8, device=DEV)
            s = torch.empty(shape[:-1], device=DEV)
            B.quantize_int8(t, q, s)
            return q, s

        self.w1, self.w3, self.w2 = codes(E, I, H), codes(E, I, H), codes(E, H, I)
        self.sg, self.sl = B.grouped_shape(R, H, I, E, dtype=dtype, act="silu"), B.grouped_shape(R, I, H, E, dtype=dtype)
        n = max(B.grouped_workspace_bytes(self.sg, B.MOE_CALL_GROUPED_GATED_INT8),
                B.grouped_workspace_bytes(self.sl, B.MOE_CALL_GROUPED_LINEAR_INT8))
        self.ws = torch.empty(max(n, 16), dtype=torch.uint8, device=DEV)
        t = TYPES[dtype]
        self.o = dict(qx=torch.zeros(R, B.int8_row_bytes(H), dtype=torch.int8, device=DEV), sx=torch.zeros(R, device=DEV),
                      h=torch.zeros(R, I, dtype=t, device=DEV), qh=torch.zeros(R, B.int8_row_bytes(I), dtype=torch.int8, device=DEV),
                      sh=torch.zeros(R, device=DEV), y=torch.zeros(R, H, dtype=t, device=DEV))

    def run(self, stream=None):
        o, off, ws = self.o, self.offsets, self.ws
        B.quantize_int8(self.x, o["qx"], o["sx"], stream=stream)
        B.grouped_gated_int8_forward(o["qx"], o["sx"], off, *self.w1, *self.w3, o["h"], self.sg, ws, stream=stream)
        B.quantize_int8(o["h"], o["qh"], o["sh"], stream=stream)
        B.grouped_linear_int8_forward(o["qh"], o["sh"], off, *self.w2, o["y"], self.sl, ws, stream=stream)

    def clear(self):
        for t in self.o.values():
            t.zero_()
        self.ws.fill_(0xFF)


# decoding steps, small tiles without a table, streamed ones, and tiles of 128 or 320 rows with one
@pytest.mark.parametrize("dtype", ("bf16", "f32"))
@pytest.mark.parametrize("size", ((8, 20, 200, 136), (130, 5, 264, 136), (300, 60, 1000, 1096), (5000, 20, 520, 1032)), ids=str)
def test_integer_products_in_a_graph_replay_like_eager(size, dtype):
    """Captured once, replayed with other rows and row counts (empty experts, one expert of all, rows of no expert) and eager
    work between: every replay gives the eager calls' bits, on rows of no expert too."""
    R, E, H, I = size
    b = Served(R, E, H, I, dtype, sum(size))
    b.run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b.run()
    one = [0] * E
    one[E // 2] = R
    few = [0] * E
    few[-1], few[0] = R // 3, R // 2
    for i, (counts, first) in enumerate(((one, 0), (few, R - sum(few)), ([0] * E, 3), ([R // E] * (E - 1) + [0], 1))):
        gen = torch.Generator().manual_seed(i)
        b.x.copy_(rand(gen, R, H, dtype=dtype))
        b.offsets.copy_(offsets_of(counts, first))
        b.clear()
        b.run()
        want = {n: t.clone() for n, t in b.o.items()}
        b.clear()
        graph.replay()
        torch.cuda.synchronize()
        for n, t in b.o.items():
            assert torch.equal(t, want[n]), (i, n)
        assert not b.o["y"][first + sum(counts):].any() and not b.o["y"][:first].any()


def test_integer_products_on_two_streams_at_once():
    served = [Served(300, 60, 1000, 1096, "bf16", 1), Served(8, 20, 200, 136, "f32", 2), Served(2000, 6, 520, 264, "bf16", 3)]
    want = []
    for b in served:
        b.clear()
        b.run()
        torch.cuda.synchronize()
        want.append({n: t.clone() for n, t in b.o.items()})
        b.clear()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in served]
    for _ in range(5):
        for b, s in zip(served, streams):
            b.run(stream=s)
    torch.cuda.synchronize()
    for b, w in zip(served, want):
        for n, t in b.o.items():
            assert torch.equal(t, w[n]), n


@pytest.mark.parametrize("dtype,grad", (("bf16", "f32"), ("f32", "f32")))
@pytest.mark.parametrize("size", ((60, 4, 72, 2048), (700, 5, 264, 136), (4000, 3, 1032, 520)), ids=str)
def test_backward_in_a_graph_replays_like_eager(size, dtype, grad):
    """Both products in one launch, a cut contraction and large tiles, replayed with other row counts."""
    R, E, K, N = size
    gen = torch.Generator().manual_seed(sum(size))
    x, dh, g, u = (rand(gen, R, n, dtype=dtype).to(DEV) for n in (K, N, N, N))
    w1, w3 = (rand(gen, E, N, K, dtype=dtype, std=0.1).to(DEV) for _ in range(2))
    off, s = offsets_of([R // E] * E).to(DEV), B.grouped_shape(R, K, N, E, dtype=dtype, act="gelu", grad_dtype=grad)
    ws = ws_for(s, B.MOE_CALL_GROUPED_GATED_BACKWARD)
    o = out((R, K), dtype), out((E, N, K), grad), out((E, N, K), grad)

    def run():
        B.grouped_gated_backward(dh, x, off, w1, w3, g, u, *o, s, ws)

    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for counts, first in (([R] + [0] * (E - 1), 0), ([0] * (E - 1) + [R // 2], R // 3), ([0] * E, 2), ([R // E - 1] * E, 1)):
        off.copy_(offsets_of(counts, first))
        got = []
        for f in (run, graph.replay):
            for t in o:
                t.view(torch.uint8).fill_(gu.POISON)
            ws.fill_(0xFF)
            f()
            torch.cuda.synchronize()
            got.append([t.clone() for t in o])
        for a, b in zip(*got):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
        rows_left(o[0], offsets_of(counts, first), "dx")
        for e, n in enumerate(counts):
            assert n or not (o[1][e].any() or o[2][e].any())


# decoding steps, streamed and small tiles, with and without a table
@pytest.mark.parametrize("dtype", ("bf16", "f32"))
@pytest.mark.parametrize("R", (16, 40, 1500, 20000))
def test_as_many_experts_as_there_may_be(R, dtype):
    K, N, E = 72, 40, 1024
    gen = torch.Generator().manual_seed(R)
    p = torch.rand(E, generator=gen).double() ** 4
    off = offsets_of(torch.bincount(torch.multinomial(p, R - 2, replacement=True, generator=gen), minlength=E).tolist(), 1)
    x, dy, w = rand(gen, R, K, dtype=dtype).to(DEV), rand(gen, R, N, dtype=dtype).to(DEV), rand(gen, E, N, K, dtype=dtype).to(DEV)
    doff, s = off.to(DEV), B.grouped_shape(R, K, N, E, dtype=dtype)
    sg = B.grouped_shape(R, K, N, E, dtype=dtype, act="silu")
    y, h, dx, dw = out((R, N), dtype), out((R, N), dtype), out((R, K), dtype), out((E, N, K), dtype)
    B.grouped_linear_forward(x, doff, w, y, s, ws_for(s, B.MOE_CALL_GROUPED_LINEAR_FORWARD))
    B.grouped_gated_forward(x, doff, w, w, h, sg, ws_for(sg, B.MOE_CALL_GROUPED_GATED_FORWARD))
    B.grouped_linear_backward(dy, x, doff, w, dx, dw, s, ws_for(s, B.MOE_CALL_GROUPED_LINEAR_BACKWARD))
    for n, t in (("y", y), ("h", h), ("dx", dx)):
        rows_left(t, off, n)
    ref = {n: torch.zeros(t.shape, dtype=torch.float64, device=DEV) for n, t in (("y", y), ("h", h), ("dx", dx), ("dw", dw))}
    tol = {n: torch.zeros_like(t) for n, t in ref.items()}
    for e, r in groups(off):
        X, D, W = x[r].double(), dy[r].double(), w[e].double()
        z, t = X @ W.T, 2 * fsum(X, W, K)
        a, _ = act64(z, "silu")
        ref["y"][r], tol["y"][r] = z, t
        ref["h"][r] = a * z
        tol["h"][r] = 1.13 * t * z.abs() + a.abs() * t + 1.13 * t * t + 2.0 ** -20 * (1 + z.abs()) * z * z
        ref["dx"][r], tol["dx"][r] = D @ W, 2 * fsum(D, W.T, N)
        ref["dw"][e], tol["dw"][e] = D.T @ X, 2 * fsum(D.T, X.T, r.stop - r.start)
    for n, t in (("y", y), ("h", h), ("dx", dx), ("dw", dw)):
        v = slice(1, int(off[-1])) if n != "dw" else slice(None)
        close(n, t[v], dtype, ref[n][v], U[dtype] * ref[n][v].abs() + tol[n][v])
