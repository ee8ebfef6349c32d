"""Block norms where every workgroup walks several rows, in every width class (rows of one to
sixteen waves, vectors and single columns): results, gradients and the sums over rows against
64 bits.

Sums over rows in fp32: a workgroup adds up to rows / workgroups rows one after another, then
groups / 16 sums and 16 of those, where groups are the workgroups of a pass (at most 2048 rows
at a time, at least 256): below rows / 256 + 2048 / 16 + 16 + 4 roundings in all, each of at
most u times the sum of magnitudes."""
import pytest
import torch

import tests.test_gpu_dense as base
from tests.helpers import require_gpu
from tests.test_gpu_dense import ALL_TYPES, U, Ref, gen_of, half_step, norm_grads, norm_inputs, randn, tiny, within

pytestmark = pytest.mark.gpu

# cols: waves a row, vectors (v) or single columns (s)
SHAPES = [(5000, 40), (5000, 77), (2100, 1000),        # 1v, 1s, 1v
          (1500, 1537), (2100, 2040), (900, 2040),     # 4s, 2v, 4v
          (1100, 4088), (700, 3001),                   # 4v, 8s
          (600, 4104), (600, 7168), (600, 4099),       # 8v, 8v, 16s
          (600, 8191),                                 # 16s
          (600, 9000), (600, 9001)]                    # 16v, 16s


@pytest.fixture(scope="module")
def lib():
    require_gpu()
    import int4_group_quantized_g128_amd as lib
    return lib


@pytest.mark.parametrize("dt", ALL_TYPES)
@pytest.mark.parametrize("t,c", SHAPES)
def test_many_rows(lib, t, c, dt):
    gen = gen_of(t + 3 * c)
    dr, dn = randn(gen, t, c).to(dt), randn(gen, t, c).to(dt)
    for gate in ("channel", "token") if c > 4104 else base.GATES:
        kw = norm_inputs(t, c, dt, gate, 6)
        f = base.norm_check(lib, kw)
        got = lib.block_norm_backward(dr, dn, alpha=0.75, **kw)
        ref = norm_grads(f, dr, dn, kw["y"], gate)
        # per row: rstd twice in every term, sums over the row (32), a dozen products
        row = 3 * f.e_rs / U + 64
        add = t / 256 + 2048 / 16 + 20
        for name, (v, mag) in ref.items():
            per = row if v.shape[0] == t else float(row.max()) + add
            tol = per * U * mag
            if got[name].dtype != torch.float32:
                tol = tol + half_step(got[name].dtype) * (v.abs() + tol) + tiny(got[name].dtype)
            assert got[name].shape == v.shape, name
            within(got[name], v, tol + 1e-37, f"{gate} {name}")


@pytest.mark.parametrize("dt", ALL_TYPES)
@pytest.mark.parametrize("t,c", [(1100, 77), (700, 3001), (600, 7168), (300, 9000), (300, 9001)])
def test_many_rows_codes_and_repeats(lib, t, c, dt):
    """INT8 codes of every row as of a call on the last rows alone, and equal bits again."""
    base.test_block_norm_codes(lib, t, c, dt)
    kw = norm_inputs(t, c, dt, "channel", 4)
    a, b = (lib.block_norm_backward(kw["y"], kw["res"], **kw) for _ in range(2))
    assert all(torch.equal(a[k], b[k]) for k in a)
    _, q, s = lib.block_norm_forward(quantize=True, **kw)
    tail = {k: v[-3:].clone() if v.shape[0] == t else v for k, v in kw.items()}
    _, q3, s3 = lib.block_norm_forward(quantize=True, **tail)
    assert torch.equal(q[-3:], q3) and torch.equal(s[-3:], s3)


def test_gate_that_is_no_tensor(lib):
    x = torch.zeros(4, 64, device="cuda")
    for gate in (0.5, [1.0] * 64):
        with pytest.raises(TypeError):
            lib.block_norm_forward(x, y=x, gate=gate)
        with pytest.raises(TypeError):
            lib.block_norm_backward(x, None, x, y=x, gate=gate)
