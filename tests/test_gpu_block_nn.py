"""AddNorm and route through autograd on the GPU: outputs and gradients against the same
formulas in 64 bits, the chain of both with a Float8Linear, and a captured training step."""
import numpy as np
import pytest

from tests.gpu_util import gpu, have_gpu, lib

pytestmark = [gpu, pytest.mark.skipif(not have_gpu(), reason="needs an MI355X")]
U = 2.0 ** -24


@pytest.fixture(scope="module")
def f():
    return lib()


def _randn(*shape, seed, scale=1.0):
    import torch
    g = torch.Generator(device="cuda:0").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda:0") * scale).to(torch.bfloat16)


def _norm64(h, gamma, beta, layer):
    m = h.mean(-1, keepdim=True) if layer else 0.0
    y = (h - m) * (((h - m) ** 2).mean(-1, keepdim=True) + 1e-5).rsqrt() * gamma
    return y + beta if layer else y


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("with_res", [True, False])
def test_add_norm(f, kind, with_res):
    import torch
    from fp8_dynamic_scaling_amd.nn import AddNorm
    layer = kind == "layer"
    m = AddNorm(264, kind, device="cuda:0")
    with torch.no_grad():
        m.weight.add_(_randn(264, seed=1, scale=0.1))
        if layer:
            m.bias.copy_(_randn(264, seed=2, scale=0.1))
    x = _randn(2, 24, 264, seed=3).requires_grad_(True)
    res = _randn(2, 24, 264, seed=4).requires_grad_(True) if with_res else None
    y, h = m(x, res)
    dy, dh = _randn(2, 24, 264, seed=5), _randn(2, 24, 264, seed=6)
    torch.autograd.backward([y, h], [dy, dh])
    assert (h is x) if not with_res else torch.equal(h, (x.float() + res.float()).to(torch.bfloat16))
    h64 = h.detach().double().requires_grad_(True)
    g64, b64 = m.weight.detach().double().requires_grad_(True), None
    if layer:
        b64 = m.bias.detach().double().requires_grad_(True)
    y64 = _norm64(h64, g64, b64, layer)
    torch.autograd.backward([y64, h64], [dy.double(), dh.double()])
    # y: bf16's half step and some ten fp32 roundings of terms up to |y| + |beta|
    assert bool(((y - y64).abs() <= 2.0 ** -8 * y64.abs() + 16 * U * (y64.abs() + 1)).all())
    # dx without a residual is the sum of two bf16 gradients that autograd rounds once more
    mag = 8 * dh.double().abs().max() + 8 * dy.double().abs().max()
    halves = 2.0 ** -8 * h64.grad.abs() if with_res else 2.0 ** -8 * (h64.grad.abs() * 2 + dh.double().abs())
    assert bool(((x.grad - h64.grad).abs() <= halves + 64 * U * mag).all())
    assert not with_res or torch.equal(x.grad, res.grad)
    for got, want, terms in ((m.weight.grad, g64.grad, dy.double().abs().sum((0, 1)) * 8),
                             *(((m.bias.grad, b64.grad, dy.double().abs().sum((0, 1))),) if layer else ())):
        assert bool(((got - want).abs() <= 2.0 ** -8 * want.abs() + 64 * U * terms).all())


def test_add_norm_with_one_output_used(f):
    """The gradient of y alone, of h alone, and with frozen parameters."""
    import torch
    from fp8_dynamic_scaling_amd.nn import AddNorm
    m = AddNorm(64, device="cuda:0")
    x, res = (_randn(5, 64, seed=s).requires_grad_(True) for s in (1, 2))
    g = _randn(5, 64, seed=3)
    y, h = m(x, res)
    gy, = torch.autograd.grad(y, x, g, retain_graph=True)
    gh, gr = torch.autograd.grad(h, (x, res), g)
    assert torch.equal(gh, g) and torch.equal(gr, g)
    m.weight.requires_grad_(False)
    y, h = m(x, res)
    both, = torch.autograd.grad(y, x, g)
    assert torch.equal(both, gy)


def test_add_norm_outputs_changed_in_place(f):
    """y may be changed in place (its values are not kept); a changed stream, whose values are,
    is refused by the backward pass."""
    import torch
    from fp8_dynamic_scaling_amd.nn import AddNorm
    m = AddNorm(64, device="cuda:0")
    x, res = (_randn(2, 3, 64, seed=s).requires_grad_(True) for s in (1, 2))
    g = _randn(2, 3, 64, seed=3)
    y, h = m(x, res)
    want, = torch.autograd.grad(y, x, 2 * g)
    y, h = m(x, res)
    y.mul_(2)
    got, = torch.autograd.grad(y, x, g)
    assert torch.equal(got, want)
    y, h = m(x, res)
    h.add_(1)
    with pytest.raises(RuntimeError, match="inplace"):
        torch.autograd.grad(y, x, g)


def test_no_rows_and_no_second_derivatives(f):
    import torch
    from fp8_dynamic_scaling_amd.nn import AddNorm, route
    m = AddNorm(64, device="cuda:0")
    x = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda:0", requires_grad=True)
    y, h = m(x, x)
    (y.sum() + h.sum()).backward()
    assert y.shape == h.shape == x.grad.shape == (0, 64) and not bool(m.weight.grad.any())
    x = _randn(4, 64, seed=1).requires_grad_(True)
    dx, = torch.autograd.grad(m(x)[0].float().pow(2).sum(), x, create_graph=True)
    with pytest.raises(RuntimeError, match="differentiat"):
        dx.sum().backward()
    l = torch.randn(4, 8, device="cuda:0", requires_grad=True)
    dl, = torch.autograd.grad(route(l, 2).weights.pow(2).sum(), l, create_graph=True)
    with pytest.raises(RuntimeError, match="differentiat"):
        dl.sum().backward()


@pytest.mark.parametrize("gate", ["softmax", "softmax_topk", "sigmoid"])
def test_route(f, gate):
    import torch
    from fp8_dynamic_scaling_amd.nn import route
    T, E, k = 150, 20, 3
    l = _randn(T, E, seed=10, scale=1.5).float().requires_grad_(True)
    r = route(l, k, gate)
    assert r.offsets[-1] == T * k and not r.ids.requires_grad and r.weights.requires_grad
    v = _randn(T, k, seed=11).float()
    (r.weights * v).sum().backward()
    l64 = l.detach().double().requires_grad_(True)
    at = r.ids.long()
    if gate == "sigmoid":
        w = torch.sigmoid(l64.gather(1, at))
    elif gate == "softmax":
        w = torch.softmax(l64, 1).gather(1, at)
    else:
        w = torch.softmax(l64.gather(1, at), 1)
    (w * v.double()).sum().backward()
    # exp of arguments up to 16 and a few roundings; gradients are sums of k such terms
    assert bool(((r.weights - w).abs() <= 96 * U * w).all())
    terms = (w.detach() * v.double().abs()).sum(1, keepdim=True)
    assert bool(((l.grad - l64.grad).abs() <= 160 * U * terms).all())
    # the sorted rows: pair order[i] belongs to the expert whose range holds i
    pair = r.order.long()
    expert = torch.bucketize(torch.arange(T * k, device="cuda:0"), r.offsets[1:].long(), right=True)
    assert torch.equal(r.ids.reshape(-1)[pair].long(), expert)
    assert torch.equal(r.slot.reshape(-1)[pair], torch.arange(T * k, dtype=torch.int32, device="cuda:0"))


def test_refusals(f):
    import torch
    from fp8_dynamic_scaling_amd.nn import AddNorm, route
    m = AddNorm(64, device="cuda:0")
    x = _randn(3, 64, seed=1)
    with pytest.raises(TypeError, match="bfloat16"):
        m(x.float())
    with pytest.raises(RuntimeError, match="GPU"):
        m(x.cpu())
    with pytest.raises(ValueError, match="shape"):
        m(x, x[:2])
    with pytest.raises(ValueError, match="features"):
        m(x[:, :32])
    with pytest.raises(ValueError, match="kind"):
        AddNorm(64, "batch")
    with pytest.raises(ValueError, match="gate"):
        route(x.float(), 2, "top")
    with pytest.raises(ValueError, match="tokens"):
        route(x.float()[0], 2)
    with pytest.raises(RuntimeError, match="GPU"):
        route(x.cpu(), 2)
    with pytest.raises(f.Fp8Error):
        route(x, 65)  # more than there are experts


def _step(m, lin, x, res, dy, dh):
    import torch
    y, h = m(x, res)
    return torch.autograd.grad([lin(y), h], [x, res, m.weight, lin.weight], [dy, dh])


def test_training_step_captured(f):
    """Norm, residual and Float8Linear, forward and backward captured into one graph and
    replayed over new inputs with eager steps of the same leaves between: the eager bits."""
    import torch
    from fp8_dynamic_scaling_amd.nn import AddNorm, Float8Linear
    m, lin = AddNorm(256, device="cuda:0"), Float8Linear(256, 128, device="cuda:0")
    x, res = (torch.zeros(64, 256, dtype=torch.bfloat16, device="cuda:0", requires_grad=True) for _ in range(2))
    dy, dh = _randn(64, 128, seed=21), _randn(64, 256, seed=22)

    def fill(seed):
        with torch.no_grad():
            x.copy_(_randn(64, 256, seed=seed))
            res.copy_(_randn(64, 256, seed=seed + 100))

    fill(0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        _step(m, lin, x, res, dy, dh)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = _step(m, lin, x, res, dy, dh)
    for seed in range(1, 5):
        fill(seed)
        graph.replay()
        got = [t.clone() for t in out]
        want = _step(m, lin, x, res, dy, dh)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), seed


def test_route_backward_is_given_the_weights_gradient_alone(f, monkeypatch):
    """No zeros are made for the outputs without a gradient, and none are passed on where the
    weights have none."""
    import torch
    from fp8_dynamic_scaling_amd.nn import RouteFunction, route
    seen, backward = [], RouteFunction.backward

    def spy(ctx, *grads):
        seen.append([g is not None for g in grads])
        return backward(ctx, *grads)

    monkeypatch.setattr(RouteFunction, "backward", staticmethod(spy))
    l = torch.randn(70, 8, device="cuda:0", requires_grad=True)
    route(l, 2).weights.pow(2).sum().backward()
    assert seen == [[False, True, False, False, False]] and bool(l.grad.any())

    class Cut(torch.autograd.Function):
        @staticmethod
        def forward(ctx, w):
            return w.clone()

        @staticmethod
        def backward(ctx, g):
            return None

    l.grad = None
    Cut.apply(route(l, 2).weights).sum().backward()
    assert l.grad is None
