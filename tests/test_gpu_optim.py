"""optim.AdamW on the GPU: runs that go on from a loaded state."""
import copy

import pytest
import torch

from tests.gpu_util import lib

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kw", [{}, dict(max_norm=float("inf")), dict(capturable=True)])
def test_goes_on_from_torchs_state(kw):
    """Two steps from the state that torch.optim.AdamW had after three, against torch's own: in each an update of at most
    5 lr to 16 roundings of 2^-24, and two of the parameter, on both sides."""
    lib()
    from fp8_dynamic_scaling_amd.optim import AdamW
    lr = 1e-2
    g = torch.Generator().manual_seed(1)
    ps = [torch.nn.Parameter(torch.randn(s, generator=g).cuda()) for s in ((33, 7), (1000,))]
    args = dict(lr=lr, betas=(0.8, 0.95), eps=1e-6, weight_decay=0.1)
    ref = torch.optim.AdamW(ps, **args)
    grads = [[torch.randn(p.shape, generator=g).cuda() for p in ps] for _ in range(5)]

    def step(opt, ps, gs):
        for p, x in zip(ps, gs):
            p.grad = x.clone()
        opt.step()

    for t in range(3):
        step(ref, ps, grads[t])
    qs = [torch.nn.Parameter(p.detach().clone()) for p in ps]
    opt = AdamW(qs, **args, **kw)
    opt.load_state_dict(copy.deepcopy(ref.state_dict()))
    for t in (3, 4):
        step(ref, ps, grads[t])
        step(opt, qs, grads[t])
    for p, q in zip(ps, qs):
        tol = 2 * 2 * 2.0 ** -24 * (16 * 5 * lr + 2 * p.abs())
        assert ((p - q).abs() <= tol).all()
    assert int(opt.state[qs[0]]["step"]) == 5
