"""The AdamW step and the norm at the ends of their ranges: roots of subnormal numbers, moments and factors that
overflow, tables whose workgroups take two pieces (GPU)."""
import numpy as np
import pytest
import torch

from tests.gpu_util import lib
from tests.test_gpu_adamw import B1, B2, F32, LR, WD, check, host, make, step

pytestmark = pytest.mark.gpu


def far_gradients(n, seed):
    """Groups of 32 of magnitudes 10^-24 to 10^-12 (squares down to fp32's last subnormal numbers and zero), every
    third one with magnitudes up to 10^18 among them."""
    g = torch.Generator().manual_seed(seed)
    e = torch.rand(n, generator=g) * 12 - 24
    large = (torch.arange(n) // 32 % 3 == 1) & (torch.rand(n, generator=g) < 0.5)
    e = torch.where(large, torch.rand(n, generator=g) * 28 - 10, e)
    return (torch.randint(0, 2, (n,), generator=g) * 2 - 1) * 10.0 ** e


@pytest.mark.parametrize("p16,master", [(False, False), (True, True)])
@pytest.mark.parametrize("mx8", [True, False])
@pytest.mark.parametrize("seed", [0, (3 << 32) + 5])
def test_adamw_far_second_moments(p16, master, mx8, seed):
    """Codes and scales bit for bit over three steps from zeroed states, the second and third with smaller gradients,
    so that the squares of small roots are subnormal too."""
    f = lib()
    s = make([96, 4099, 70001], p16, False, master, mx8)
    for k in ("m", "v", "ms", "vs"):
        for t in s[k] or ():
            t.zero_()
    for t in (1, 2, 3):
        for i, g in enumerate(s["grads"]):
            g.copy_(far_gradients(g.numel(), 10 * t + i) * 4.0 ** (1 - t))
        before = host(s)
        step(f, s, t, seed)
        check(f, before, s, t, seed, None, p16, master, mx8)


@pytest.mark.parametrize("mx8", [True, False])
def test_adamw_small_gradients_take_a_whole_first_step(mx8):
    """Without epsilon a first step moves by the rate, whatever the gradient's size. Relative error: two roundings of m,
    three of v (halved by the root), one each of the root, its factor, their product, the quotient, the step and the
    update, and two of the reciprocal (1 ulp): 11.5 of 2^-24."""
    f = lib()
    n = 4096
    # squares times 1 - b2 from 5e-36 on: normal numbers, so that each rounding is 2^-24
    g = (10.0 ** torch.linspace(-17, 2, n)).cuda()
    g[1::2] *= -1
    p = torch.zeros(n, device="cuda")
    kind = dict(dtype=torch.uint8 if mx8 else torch.float32, device="cuda")
    m, v = torch.zeros(n, **kind), torch.zeros(n, **kind)
    ms, vs = (torch.zeros(n // 32, dtype=torch.uint8, device="cuda") for _ in range(2))
    scales = dict(exp_avg_scales=[ms], exp_avg_sq_scales=[vs]) if mx8 else {}
    f.fp8_adamw([p], [g], [m], [v], LR, B1, B2, 0.0, 0.0, 1, **scales)
    want = -LR * g.sign().double()
    assert ((p.double() - want).abs() <= 12 * 2.0 ** -24 * LR).all()
    if mx8:
        assert (v != 0).all()  # a code above zero for each root above zero


@pytest.mark.parametrize("mx8", [True, False])
def test_adamw_smallest_epsilon(mx8):
    """Elements without gradients stay, beside one that has one."""
    f = lib()
    p, g = torch.ones(64, device="cuda"), torch.zeros(64, device="cuda")
    g[40] = 1e-3
    kind = dict(dtype=torch.uint8 if mx8 else torch.float32, device="cuda")
    ms, vs = (torch.zeros(2, dtype=torch.uint8, device="cuda") for _ in range(2))
    scales = dict(exp_avg_scales=[ms], exp_avg_sq_scales=[vs]) if mx8 else {}
    f.fp8_adamw([p], [g], [torch.zeros(64, **kind)], [torch.zeros(64, **kind)], LR, B1, B2, 2.0 ** -126, 0.0, 1, **scales)
    still = torch.arange(64, device="cuda") != 40
    assert (p[still] == 1).all() and abs(float(p[40]) - (1 - LR)) <= 2.0 ** -23


@pytest.mark.parametrize("mx8", [True, False])
def test_adamw_second_moment_that_overflows(mx8):
    """A finite gradient whose square is infinite: the root is infinite and the update 0, beside the decay."""
    f = lib()
    s = make([100], False, False, False, mx8)
    ref = make([100], False, False, False, mx8)
    s["grads"][0][37], s["grads"][0][70] = 1e20, -3e38
    step(f, s, 1)
    step(f, ref, 1)
    p, before = s["params"][0].cpu().numpy(), make([100], False, False, False, mx8)["params"][0].cpu().numpy()
    for i in (37, 70):
        assert p[i] == before[i] * F32(1.0 - LR * WD)
    others = [i for i in range(100) if i not in (37, 70)]
    assert np.array_equal(p[others], ref["params"][0].cpu().numpy()[others])
    if mx8:
        assert s["vs"][0].tolist()[1:3] == [255, 255] and (s["v"][0][32:96] == 0x7F).all()
        assert (s["ms"][0] != 255).all()
    else:
        assert torch.isinf(s["v"][0][[37, 70]]).all() and torch.isfinite(s["m"][0]).all()


@pytest.mark.parametrize("p16,g16,master", [(True, True, False), (True, False, True), (False, False, False)])
@pytest.mark.parametrize("seed", [0, (5 << 32) + 77])
def test_adamw_large_table(p16, g16, master, seed):
    """A table past 2^24 elements, whose workgroups take two pieces: each tensor as when it is stepped alone, at its place
    among empty ones (whose random bits go by the place), by workgroups of one."""
    f = lib()
    sizes = [1, 4096 * 1200 + 2047, 2048, 4096 * 700 + 2049, 33, 4096 * 900 + 1, 4097, 4096 * 1500 + 31, 0, 2047]
    assert sum(sizes) >= 8192 * 2048 and max(sizes) < 8192 * 2048
    s, ref = (make(sizes, p16, g16, master, False) for _ in range(2))
    for t in (s, ref):
        for k in "mv":
            t[k] = [torch.zeros(n, dtype=torch.uint8, device="cuda") for n in sizes]
            t[k + "s"] = [torch.zeros(-(-n // 32), dtype=torch.uint8, device="cuda") for n in sizes]
    mul = torch.tensor([0.37], device="cuda")
    for t in (1, 2):
        step(f, s, t, seed, mul)
        for i in range(len(sizes)):
            one = {k: v and [x if j == i else x[:0] for j, x in enumerate(v)] for k, v in ref.items()}
            step(f, one, t, seed, mul)
        for k, v in s.items():
            for i, (x, y) in enumerate(zip(v or (), ref[k] or ())):
                assert torch.equal(x.view(torch.uint8), y.view(torch.uint8)), (t, k, i)
    assert (s["v"][7] != 0).any()


def test_grad_norm_factor_that_overflows():
    """A factor past fp32 makes the step change nothing, and it is not counted either."""
    f = lib()
    g = torch.full((100,), 1e-30, device="cuda")
    norm, mul = torch.empty(1, device="cuda"), torch.empty(1, device="cuda")
    t = torch.zeros(1, dtype=torch.int32, device="cuda")
    for grads in ([g], [g] * 70):  # one launch and two
        ws = torch.empty(f.fp8_grad_norm_ws_bytes(grads), dtype=torch.uint8, device="cuda")
        f.fp8_grad_norm(grads, norm, mul, ws, grad_scale=1e39, step=t)
        want = 1e39 * float(g[0].double()) * (100 * len(grads)) ** 0.5
        assert abs(float(norm) - want) <= 2.0 ** -23 * want
        assert torch.isnan(mul).all() and int(t) == 0
        f.fp8_grad_norm(grads, norm, mul, ws, grad_scale=1e39, max_norm=1.0, step=t)  # clipped to a factor of 1e29
        assert abs(float(mul) * want / 1e39 - 1) <= 2.0 ** -23 and int(t) == 1
        t.zero_()
