"""The residual norm and the router at calls beyond the ordinary ones: operands at any offset in
memory through autograd, rows that are not finite, more rows than one launch holds."""
import numpy as np
import pytest

import oracle
import synth
from tests.gpu_util import gpu, have_gpu, lib, to_dev_bf16
from tests.test_gpu_add_norm import EPS, NEPS, _bits, _forward, _inputs, _sum_bits

pytestmark = [gpu, pytest.mark.skipif(not have_gpu(), reason="needs an MI355X")]


@pytest.fixture(scope="module")
def f():
    oracle.build(force=False)
    synth.build(force=False)
    return lib()


def _randn(*shape, seed, scale=1.0):
    import torch
    g = torch.Generator(device="cuda:0").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda:0") * scale).to(torch.bfloat16)


# ---- offsets ------------------------------------------------------------------------------


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("with_res", [True, False])
def test_add_norm_operands_at_any_offset(f, kind, with_res):
    """Contiguous views that do not begin on 16 bytes: inputs and parameters cut from a longer
    buffer, and the gradients that the backward of a concatenation hands on. The bits are those
    of the same values in tensors of their own."""
    import torch
    from fp8_dynamic_scaling_amd.nn import AddNorm
    rows, cols, n = 5, 264, 5 * 264
    flat = _randn(3 + 2 * n + 2 * cols, seed=1)
    flat[3 + 2 * n:] += 1
    g = _randn(3 + 2 * n, seed=2)

    def step(cut):
        m = AddNorm(cols, kind, device="cuda:0")
        x, res = (cut(3 + i * n, n).view(rows, cols).requires_grad_(True) for i in range(2))
        m.weight = torch.nn.Parameter(cut(3 + 2 * n, cols))
        leaves = [x, m.weight]
        if kind == "layer":
            m.bias = torch.nn.Parameter(cut(3 + 2 * n + cols, cols))
            leaves.append(m.bias)
        if with_res:
            leaves.append(res)
        y, h = m(x, res if with_res else None)
        out = torch.cat([flat[:3], y.flatten(), h.flatten()])
        return [y, h, *torch.autograd.grad(out, leaves, g)]

    got = step(lambda at, size: flat[at:at + size].detach())
    want = step(lambda at, size: flat[at:at + size].detach().clone())
    assert all(torch.equal(a, b) for a, b in zip(got, want))
