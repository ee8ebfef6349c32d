"""GPU tests of the FP8 experts used together, against 64 bits that round and quantise where the calls
do, so that what is left is the products' own error and the last rounding.

A product's result is not the exact one rounded, but a neighbour, in about 1 % of bf16 results (the
matrix instruction's loss of 1.4e-5 of the norm against a step of 2^-7 to 2^-8 of the value), in fp16
in eight times as many by an eighth of that; both come to 0.011 2^-8 a result.  An e4m3 step is
2^-4 to 2^-3 of the value, so a code of silu(g) u changes for its g, its u or, twice as often at most, its
group's scale in 4 0.011 2^-8 / 2^-4 = 0.0028 of cases at most, by at most 2^-3: 0.0066 in root mean
square, and as much in the down product, whose terms' errors have either sign.  Without the loss (up
to 16 rows) fp32 sums change a hundredth as many results: 0.0007."""
import pytest
import torch

from tests.helpers import require_gpu
from tests.test_gpu_experts import SIZES, Block, Step
from tests.test_gpu_fp8 import TYPES, blocks_of, col_ref, cols_of, row_ref, rows_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lib():
    require_gpu()
    import int4_group_quantized_g128_amd as lib
    return lib


def off_by(got, ref):
    return ((got.double() - ref).norm() / ref.norm()).item()


def half(dt):
    return torch.finfo(dt).eps / 2


@pytest.mark.parametrize("size", SIZES + [(8, 1040, 272, 2, 16, 4, 8), (130, 2048, 528, 8, 40, 8, 24)])
@pytest.mark.parametrize("dt", TYPES)
def test_block_by_stages(lib, size, dt):
    block = Block(lib, *size, dt)
    x = rows_of(*row_ref(block.x))
    ref = torch.zeros(block.x.shape, dtype=torch.float64, device="cuda")
    for z in range(block.held):
        tok, j = (block.ids == z + block.first).nonzero(as_tuple=True)
        if not len(tok):
            continue
        gu = (x[tok] @ blocks_of(block.gu[0][z], block.gu[1][z]).T).to(dt).double()
        g, u = gu[:, :block.i], gu[:, block.i:]
        h = rows_of(*row_ref((g * torch.sigmoid(g) * u).float()))
        y = (h @ blocks_of(block.dn[0][z], block.dn[1][z]).T).to(dt).double()
        ref.index_add_(0, tok, y * block.w[tok, j, None].double())
    if not ref.any():
        return
    few = block.ids.numel() <= 16
    err = off_by(block(), ref)
    assert err <= half(dt) + (0.0007 if few else 0.0066), err


@pytest.mark.parametrize("size", [(60, 256, 144, 2, 4), (900, 528, 272, 3, 8), (3000, 1040, 528, 2, 8), (5, 256, 512, 2, 4)])
@pytest.mark.parametrize("dt", TYPES)
def test_training_step_by_stages(lib, size, dt):
    """The gradient that reaches the product, w dout, is rounded and quantised as the calls do.  What is
    left: out and the weights' gradients, sums over y's results of which 1 % are off by 2^-7 at most, 0.0008 in root
    mean square; dW one rounding; dx a sum over such results and one rounding."""
    step = Step(lib, *size, dt)
    out, dw, dwq, dx = step()
    t, k = step.ids.shape
    ref_out, ref_dx = torch.zeros_like(step.dout, dtype=torch.float64), torch.zeros_like(step.x, dtype=torch.float64)
    ref_dw, ref_dwq = torch.zeros(t, k, dtype=torch.float64, device="cuda"), torch.zeros(dwq.shape, dtype=torch.float64,
                                                                                         device="cuda")
    x = rows_of(*row_ref(step.x))
    for z in range(step.e):
        tok, j = (step.ids == z).nonzero(as_tuple=True)   # (in slot order)
        if not len(tok):
            continue
        w = blocks_of(step.wq[0][z], step.wq[1][z])
        y = (x[tok] @ w.T).to(dt).double()
        weight = step.w[tok, j, None]
        ref_out.index_add_(0, tok, y * weight.double())
        ref_dw[tok, j] = (y * step.dout[tok].double()).sum(1)
        dy = (weight * step.dout[tok].float()).to(dt)
        ref_dwq[z] = cols_of(*col_ref(dy)).T @ cols_of(*col_ref(step.x[tok]))
        ref_dx.index_add_(0, tok, (rows_of(*row_ref(dy)) @ w).to(dt).double())
    for what, got, ref, tol in (("out", out, ref_out, half(dt) + 0.0008), ("weights", dw, ref_dw, 0.0008),
                                ("dW", dwq, ref_dwq, half(dt) + 2e-5), ("dx", dx, ref_dx, half(dt) + 0.0008)):
        err = off_by(got, ref)
        assert err <= tol, f"{what}: {err} over {tol}"
