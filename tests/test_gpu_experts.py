"""GPU tests of the FP8 experts as they are used together: tokens sorted by expert as e4m3 codes,
gate and up product, silu(g) u in e4m3, down product, weighted sum per token; a training step of
one product with its gradients; the same captured in a HIP graph, on another stream."""
import math

import pytest
import torch

from tests.helpers import require_gpu
from tests.test_gpu_fp8 import blocks_of, gen_of, row_ref, rows_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lib():
    require_gpu()
    import int4_group_quantized_g128_amd as lib
    return lib


class Block:
    """Experts [first, first + held) of `e` with their weights, and a batch."""

    def __init__(self, lib, t, h, i, k, e, first, held, dt, seed=1):
        g = gen_of(seed)
        self.lib, self.k, self.first, self.held, self.dt, self.i = lib, k, first, held, dt, i
        self.x = torch.randn(t, h, generator=g, device="cuda").to(dt)
        score = torch.randn(t, e, generator=g, device="cuda")
        top, ids = score.topk(k, dim=1)
        self.ids, self.w = ids.int().contiguous(), torch.softmax(top, 1).contiguous()
        self.gu = lib.quantize_fp8_blocks(torch.randn(held, 2 * i, h, generator=g, device="cuda") * 0.05)
        self.dn = lib.quantize_fp8_blocks(torch.randn(held, h, i, generator=g, device="cuda") * 0.05)

    def __call__(self):
        lib = self.lib
        q, s, off, perm, inv = lib.moe_dispatch_forward(self.x, self.ids, self.held, first=self.first, quantize=True)
        gu = lib.fp8_linear_forward(q, s, *self.gu, offsets=off, out_dtype=self.dt)
        q, s = lib.quantize_fp8_tokens(gu, gated=True, offsets=off)
        y = lib.fp8_linear_forward(q, s, *self.dn, offsets=off, out_dtype=self.dt)
        return lib.moe_combine_forward(y, inv, self.w)

    def ref(self):
        """64 bits from the tokens' codes on, nothing rounded between."""
        xd = rows_of(*row_ref(self.x))
        out = torch.zeros(self.x.shape, dtype=torch.float64, device="cuda")
        for z in range(self.held):
            tok, j = (self.ids == z + self.first).nonzero(as_tuple=True)
            gu = xd[tok] @ blocks_of(self.gu[0][z], self.gu[1][z]).T
            g, u = gu[:, :self.i], gu[:, self.i:]
            y = (g * torch.sigmoid(g) * u) @ blocks_of(self.dn[0][z], self.dn[1][z]).T
            out.index_add_(0, tok, y * self.w[tok, j, None].double())
        return out


SIZES = [(1, 256, 128, 2, 8, 0, 8), (64, 512, 272, 8, 64, 16, 24), (700, 1040, 256, 4, 16, 0, 16),
         (3000, 256, 384, 2, 8, 1, 6)]


@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16])
def test_block(lib, size, dt):
    """Against 64 bits: what the block rounds between is g and u to 16 bits and silu(g) u to e4m3,
    whose half step is 2^-4 of a value; over a product's many terms these errors of either sign add
    like their root, so the result's relative 2-norm error stays below that one half step."""
    block = Block(lib, *size, dt)
    out, ref = block(), block.ref()
    assert torch.isfinite(out).all()
    assert (out.double() - ref).norm() <= 2.0 ** -4 * ref.norm()
    unheld = ((block.ids < block.first) | (block.ids >= block.first + block.held)).all(dim=1)
    assert not out[unheld].any()
    assert torch.equal(out, block())


class Step:
    """A training step of one product over the experts."""

    def __init__(self, lib, t, h, n, k, e, dt, seed=2):
        g = gen_of(seed)
        self.lib, self.e, self.dt, self.k = lib, e, dt, k
        self.x = torch.randn(t, h, generator=g, device="cuda").to(dt)
        self.ids = torch.randint(0, e, (t, k), generator=g, device="cuda", dtype=torch.int32)
        self.w = torch.rand(t, k, generator=g, device="cuda")
        self.wq = lib.quantize_fp8_blocks(torch.randn(e, n, h, generator=g, device="cuda") * 0.05)
        self.dout = torch.randn(t, n, generator=g, device="cuda").to(dt)

    def __call__(self):
        lib = self.lib
        xp, off, perm, inv = lib.moe_dispatch_forward(self.x, self.ids, self.e)
        q, s, qc, sc = lib.quantize_fp8_tokens(xp, columns=True, offsets=off)
        y = lib.fp8_linear_forward(q, s, *self.wq, offsets=off, out_dtype=self.dt)
        out = lib.moe_combine_forward(y, inv, self.w)
        dy, dw = lib.moe_combine_backward(self.dout, y, inv, self.w)
        dxp, dwq = lib.fp8_linear_backward(dy, qc, sc, *self.wq, offsets=off)
        return out, dw, dwq, lib.moe_dispatch_backward(dxp, inv)


@pytest.mark.parametrize("size", [(60, 256, 144, 2, 4), (900, 528, 272, 3, 8)])
def test_training_step(lib, size):
    """Against autograd in 64 bits on the unquantised activations: every quantity is one product
    of e4m3 values, each half a step (2^-4) off, and the two factors' errors add."""
    step = Step(lib, *size, torch.bfloat16)
    out, dw, dwq, dx = step()
    x, w = step.x.double().requires_grad_(), step.w.double().requires_grad_()
    wd = blocks_of(*step.wq).requires_grad_()
    y = torch.einsum("th,enh->ten", x, wd)
    ref = (torch.gather(y, 1, step.ids.long()[:, :, None].expand(-1, -1, y.shape[2])) * w[:, :, None]).sum(1)
    ref.backward(step.dout.double())
    for got, want, what in ((out, ref, "out"), (dw, w.grad, "weights"), (dwq, wd.grad, "dw"), (dx, x.grad, "dx")):
        err = ((got.double() - want).norm() / want.norm()).item()
        assert err <= 2 * 2.0 ** -4, f"{what}: {err}"


@pytest.mark.parametrize("kind", ["block", "step"])
def test_graph(lib, kind):
    """Captured once and replayed on new inputs, with eager calls and synchronizations between:
    every replay equals the eager result."""
    make = (lambda seed: Block(lib, 64, 512, 272, 8, 64, 16, 24, torch.bfloat16, seed)) if kind == "block" else (
        lambda seed: Step(lib, 3000, 256, 144, 2, 4, torch.bfloat16, seed))
    held, others = make(3), [make(s) for s in (4, 5, 6)]
    tensors = lambda v: v if isinstance(v, tuple) else (v,)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        held()
    torch.cuda.current_stream().wait_stream(st)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = tensors(held())
    for other in others + others[:1]:
        want = [v.clone() for v in tensors(other())]
        torch.cuda.synchronize()
        for name in ("x", "ids", "w") + (("dout",) if kind == "step" else ()):
            getattr(held, name).copy_(getattr(other, name))
        for a, b in ((held.gu, other.gu), (held.dn, other.dn)) if kind == "block" else ((held.wq, other.wq),):
            for p, q in zip(a, b):
                p.view(torch.uint8).copy_(q.view(torch.uint8))
        graph.replay()
        other()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))


def test_graphs_beside_each_other(lib):
    """Two captured blocks with workspaces of their own, replayed at once on two streams."""
    blocks = [Block(lib, 200, 512, 272, 2, 8, 0, 8, torch.bfloat16, s) for s in (7, 8)]
    want = [b().clone() for b in blocks]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for b in blocks:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(b())
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in blocks]
    for _ in range(3):
        for g, st in zip(graphs, streams):
            st.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(st):
                g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))


def test_block_against_int4_layer(lib):
    """The FP8 experts and the INT4 layer made from the same weights agree as far as INT4 allows."""
    t, h, i, k, e = 64, 256, 128, 2, 8
    g = gen_of(9)
    gate, up = (torch.randn(e, i, h, generator=g, device="cuda") * 0.05 for _ in range(2))
    down = torch.randn(e, h, i, generator=g, device="cuda") * 0.05
    layer = lib.MoELayer(e, h, i, k)
    for z in range(e):
        layer.set_expert(z, gate[z], up[z], down[z])
    b = Block(lib, t, h, i, k, e, 0, e, torch.bfloat16, 10)
    b.gu, b.dn = lib.quantize_fp8_blocks(torch.cat([gate, up], 1).contiguous()), lib.quantize_fp8_blocks(down)
    want = lib.moe_int4_ffn_forward(layer, b.x, b.ids, b.w, mode=lib.Q4_W4A16).double()
    err = ((b().double() - want).norm() / want.norm()).item()
    # (INT4's half step is 1 / 14 of a group's largest value, e4m3's 2^-4 of each: three products)
    assert err <= 3 * (2.0 ** -4 + 1 / 14), err
    assert math.isfinite(err)
