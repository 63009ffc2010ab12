"""nn.Float8GatedLinear, nn.Float8GatedMLP and optim.AdamW (GPU): the layers against the library's calls and against
the unquantized block, the optimizer against the call and torch's formula, and a training step of the norm, the
block and the optimizer, eager and captured."""
import copy

import pytest
import torch

from tests.gpu_util import lib

pytestmark = pytest.mark.gpu


def randn(*shape, seed=0, scale=1.0, dtype=torch.bfloat16):
    return (torch.randn(shape, generator=torch.Generator().manual_seed(seed)) * scale).to(dtype).cuda()


def act64(x, act):
    return x * torch.sigmoid(x if act == "silu" else (8 / torch.pi) ** 0.5 * (x + 0.044715 * x ** 3))


def rel(a, b):
    return float((a.double() - b.double()).norm() / b.double().norm())


# M, K, F: packed weights in both products, in the first only, in neither; one row; a rank-3 input below
SHAPES = [(300, 256, 192), (33, 128, 16), (7, 48, 24), (1, 128, 64), (1100, 1152, 128)]


@pytest.mark.parametrize("M,K,F", SHAPES)
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_gated_linear_is_the_calls(M, K, F, act):
    """Forward and backward are the quantizers', the gated product's and the GEMMs' own results."""
    f = lib()
    from fp8_dynamic_scaling_amd import nn
    m = nn.Float8GatedLinear(K, F, act, device="cuda")
    x = randn(M, K, seed=M).requires_grad_(True)
    dh = randn(M, F, seed=M + 1, scale=1e-2)
    h = m(x)
    dx, dw = torch.autograd.grad(h, (x, m.weight), dh)
    xd, w = x.detach(), m.weight.detach()
    codes = lambda *s: torch.empty(s, dtype=torch.uint8, device="cuda")  # noqa: E731
    fl = lambda n: torch.empty(n, device="cuda")  # noqa: E731
    xq, xs, xi, wq, ws, wi = codes(M, K), fl(M), fl(M), codes(2 * F, K), fl(2 * F), fl(2 * F)
    f.fp8_quant_row(xd, f.E4M3_NATIVE, 1e-12, xq, xs, xi)
    f.fp8_quant_row(w, f.E4M3_NATIVE, 1e-12, wq, ws, wi)
    a = f.ACT_SILU if act == "silu" else f.ACT_GELU_TANH
    out, gu = torch.empty_like(h), torch.empty((M, 2 * F), dtype=h.dtype, device="cuda")
    f.fp8_gated_mm(xq, wq, f.E4M3_NATIVE, f.SCALE_ROW, xi, wi, a, gu, out)
    # the row-major and the packed form may sum in another order: two bf16 neighbours at most, 2^-7 each
    assert ((h - out).abs() <= 2.0 ** -7 * out.abs() + 1e-2 * out.abs().mean()).all()
    dgu, q, s, inv = torch.empty_like(gu), codes(M, 2 * F), fl(M), fl(M)
    f.fp8_gated_bwd(dh, gu, a, f.E5M2_NATIVE, 1e-12, dgu, q, s, inv)
    want = torch.empty_like(w)
    f.fp8_wgrad_bf16(dgu, xd, want)
    assert rel(dw, want) <= 2.0 ** -7
    wt, ts, tinv = codes(K, 2 * F), fl(K), fl(K)
    f.fp8_quant_col(w, f.E4M3_NATIVE, 1e-12, wt, ts, tinv, codes(f.fp8_quant_col_ws_bytes(1, 2 * F, K)))
    want = torch.empty_like(xd)
    f.fp8_scaled_mm(q, f.E5M2_NATIVE, wt, f.E4M3_NATIVE, f.SCALE_ROW, inv, tinv, f.OUT_BF16, want, use_fast_accum=False)
    assert rel(dx, want) <= 2.0 ** -5  # an e5m2 code of a value next to a border moves by 2^-2 of it


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_gated_mlp_against_the_unquantized_block(act):
    """Outputs and gradients are those of the block in 64 bits but for the codes' roundings: a code's error is
    0.027 of its value in the mean for e4m3 (steps of 1/8 to 1/16, divided by the root of 12), 0.053 for e5m2.
    Forward: three quantized operands a path, x, w13 (twice each in g u) and h, w2: root of 6 x 0.027^2 = 0.066.
    Backward: the gradient's codes twice (0.053), three weights' and the forward's error: root of 2 x 0.053^2 +
    3 x 0.027^2 + 0.066^2 = 0.11. Twice that is the bound."""
    lib()
    from fp8_dynamic_scaling_amd import nn
    m = nn.Float8GatedMLP(256, 384, act, device="cuda")
    x = randn(2, 129, 256, seed=3).requires_grad_(True)
    dy = randn(2, 129, 256, seed=4)
    y = m(x)
    assert y.shape == x.shape
    got = torch.autograd.grad(y, (x, m.up.weight, m.down.weight), dy)
    x64, w13, w2 = (t.detach().cpu().double().requires_grad_(True) for t in (x, m.up.weight, m.down.weight))
    p = x64 @ w13.t()
    ref = (act64(p[..., :384], act) * p[..., 384:]) @ w2.t()
    want = torch.autograd.grad(ref, (x64, w13, w2), dy.cpu().double())
    assert rel(y.detach().cpu(), ref.detach()) <= 0.13
    for a, b in zip(got, want):
        assert rel(a.cpu(), b) <= 0.22


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_gate_gradient_against_differences(act):
    """The gate's gradient is the difference quotient of the product that the same call forms, at steps that bf16
    holds: off by the two products' roundings over the step and by a sixth of the step squared times the third
    derivative, at most 1.5 for both activations."""
    f = lib()
    M, F, d = 64, 256, 2.0 ** -4
    a = f.ACT_SILU if act == "silu" else f.ACT_GELU_TANH
    g = torch.linspace(-6, 6, M * F).view(M, F)
    g = (g / d).round() * d  # multiples of the step: g + d and g - d are bf16 values
    u = randn(M, F, seed=2).cpu().float()
    one = torch.ones((M, F), dtype=torch.bfloat16, device="cuda")

    def call(gg, uu):
        gu = torch.cat([gg, uu], 1).to(torch.bfloat16).cuda()
        assert torch.equal(gu.cpu().float(), torch.cat([gg, uu], 1).to(torch.bfloat16).float())
        dgu, h = torch.empty_like(gu), torch.empty_like(one)
        f.fp8_gated_bwd(one, gu, a, f.E5M2_NATIVE, 1e-12, dgu, None, None, h=h)
        return dgu.cpu().double(), h.cpu().double()

    dgu, h = call(g, u)
    (_, hp), (_, hm) = call(g + d, u), call(g - d, u)
    up = u.to(torch.bfloat16).double().abs()
    tol = 2.0 ** -8 * (hp.abs() + hm.abs()) / (2 * d) + d * d / 6 * 1.5 * up + 2.0 ** -8 * dgu[:, :F].abs() + 1e-6
    assert ((dgu[:, :F] - (hp - hm) / (2 * d)).abs() <= tol).all()
    # linear in u: h / u is the other half
    keep = up > 0.1
    err = (dgu[:, F:] - h / u.to(torch.bfloat16).double()).abs()[keep]
    assert (err <= (2.0 ** -7 * dgu[:, F:].abs() + 1e-6)[keep]).all()


def test_gated_linear_edges():
    lib()
    from fp8_dynamic_scaling_amd import nn
    m = nn.Float8GatedLinear(64, 32, device="cuda")
    e = m(torch.empty((0, 64), dtype=torch.bfloat16, device="cuda", requires_grad=True))
    assert e.shape == (0, 32)
    dw, = torch.autograd.grad(e, m.weight, torch.empty_like(e))
    assert (dw == 0).all()
    # a gradient that is a broadcast, an input that is a piece of a larger tensor, an output changed in place
    big = randn(5, 3, 80, seed=9)
    x = big[..., 8:72].detach().requires_grad_(True)
    y = m(x)
    y.mul_(2)
    dx, = torch.autograd.grad(y.sum(), x)
    xc = x.detach().contiguous().requires_grad_(True)
    want, = torch.autograd.grad(m(xc), xc, torch.full_like(y, 2.0))
    assert torch.equal(dx, want)
    with torch.no_grad():  # nothing is kept
        assert torch.equal(m(x), m(xc.detach()))
    # only one of the two gradients
    m.weight.requires_grad_(False)
    assert torch.equal(torch.autograd.grad(m(xc), xc, torch.full_like(y, 2.0))[0], want)
    m.weight.requires_grad_(True)
    g, = torch.autograd.grad(m(xc).float().pow(2).sum(), xc, create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        g.float().sum().backward()
    with pytest.raises(ValueError, match="features"):
        m(randn(2, 32))
    with pytest.raises(TypeError, match="bfloat16"):
        m(randn(2, 64).float())


# ---- optimizer --------------------------------------------------------------------------------------

def params(dtype=torch.bfloat16, seed=0):
    return [torch.nn.Parameter(randn(*s, seed=seed + i, scale=0.1, dtype=dtype)) for i, s in
            enumerate([(64, 48), (33,), (1,), (129, 65)])]


def set_grads(ps, seed, dtype=None):
    for i, p in enumerate(ps):
        p.grad = randn(*p.shape, seed=seed * 10 + i, scale=1e-2, dtype=dtype or p.dtype)


def test_adamw_is_torchs_formula():
    """fp32 parameters and states over 20 steps against torch's AdamW in 64 bits: each step adds at most some ten
    roundings of 2^-24 to a moment and to the parameter, so 20 steps stay within 2^-15 of an update's size."""
    lib()
    from fp8_dynamic_scaling_amd.optim import AdamW
    ps = params(torch.float32)
    ref = [torch.nn.Parameter(p.detach().cpu().double()) for p in ps]
    kw = dict(lr=1e-2, betas=(0.8, 0.95), eps=1e-6, weight_decay=0.1)
    a, b = AdamW(ps, **kw), torch.optim.AdamW(ref, **kw)
    for t in range(20):
        set_grads(ps, t)
        for p, r in zip(ps, ref):
            r.grad = p.grad.cpu().double()
        a.step()
        b.step()
    for p, r in zip(ps, ref):
        assert ((p.detach().cpu().double() - r).abs() <= 2.0 ** -15 * (r.abs() + 20 * 1e-2)).all()


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("master", [False, True])
def test_adamw_saves_and_loads(bits, master):
    """A run that is saved after two steps and loaded into a new optimizer goes on with the same bits."""
    lib()
    from fp8_dynamic_scaling_amd.optim import AdamW
    kw = dict(lr=1e-2, state_bits=bits, master_weights=master, seed=7)
    ps = params()
    a = AdamW(ps, **kw)
    for t in range(2):
        set_grads(ps, t)
        a.step()
    saved = copy.deepcopy(a.state_dict())
    qs = [torch.nn.Parameter(p.detach().clone()) for p in ps]
    b = AdamW(qs, **kw)
    b.load_state_dict(saved)
    for t in range(2, 5):
        set_grads(ps, t)
        set_grads(qs, t)
        a.step()
        b.step()
    assert all(torch.equal(p, q) for p, q in zip(ps, qs))
    for p, q in zip(ps, qs):
        assert a.state[p].keys() == b.state[q].keys()
        for k, v in a.state[p].items():
            assert (torch.equal(v, b.state[q][k]) and v.dtype == b.state[q][k].dtype) if torch.is_tensor(v) else v == b.state[q][k]


def test_adamw_kinds_in_one_optimizer():
    """bf16 and fp32 parameters, bf16 and fp32 gradients, groups of other rates, a parameter without a gradient."""
    lib()
    from fp8_dynamic_scaling_amd.optim import AdamW
    a, b = params(torch.bfloat16), params(torch.float32, seed=50)
    opt = AdamW([dict(params=a, lr=1e-2), dict(params=b, lr=1e-3, weight_decay=0.5)], state_bits=8, master_weights=True)
    before = [p.detach().clone() for p in a + b]
    versions = [p._version for p in a + b]
    set_grads(a, 1)
    set_grads(b, 2)
    a[1].grad = None
    opt.step()
    for i, (p, q) in enumerate(zip(a + b, before)):
        moved = not torch.equal(p, q)
        assert moved == (i != 1)
        assert (p._version > versions[i]) == (i != 1)  # autograd sees the change
    assert a[1] not in opt.state or "exp_avg" not in opt.state[a[1]]
    assert "master" in opt.state[a[0]] and "master" not in opt.state[b[0]]
    assert opt.state[a[0]]["exp_avg"].dtype == torch.uint8


def test_adamw_clips_and_skips():
    lib()
    from fp8_dynamic_scaling_amd.optim import AdamW
    ps = params()
    opt = AdamW(ps, lr=1e-2, max_norm=0.5)
    set_grads(ps, 1)
    want = float(torch.cat([p.grad.flatten().double() for p in ps]).norm())
    opt.step(grad_scale=0.25)
    assert abs(float(opt.grad_norm) - 0.25 * want) <= 1e-6 * want
    assert int(opt.state[ps[0]]["step"]) == 1
    before = [p.detach().clone() for p in ps]
    ps[2].grad[0] = float("inf")
    opt.step()
    assert all(torch.equal(p, q) for p, q in zip(ps, before)) and int(opt.state[ps[0]]["step"]) == 1
    set_grads(ps, 2)
    opt.step()
    assert not torch.equal(ps[0], before[0]) and int(opt.state[ps[0]]["step"]) == 2
    with pytest.raises(ValueError, match="max_norm"):
        AdamW(ps).step(grad_scale=0.5)


def test_adamw_closure_and_strided_gradients():
    lib()
    from fp8_dynamic_scaling_amd.optim import AdamW
    p, q = (torch.nn.Parameter(randn(32, 48, seed=1)) for _ in range(2))
    a, b = AdamW([p], seed=3), AdamW([q], seed=3)
    g = randn(48, 32, seed=2)
    p.grad = g.t()
    q.grad = g.t().contiguous()
    b.step()

    def closure():
        assert torch.is_grad_enabled()
        return 5.0

    assert a.step(closure) == 5.0
    assert torch.equal(p, q)


def test_adamw_eight_bits_follow_thirty_two():
    """With b2 = 0.999 and constant gradients 8-bit roots, rounded by chance, grow as the 32-bit ones do: after 300
    steps the mean update over 4096 equal elements is within 5% of the exact one (a root's spread of some 20% over
    4096 elements leaves 0.3%, its square's bias of at most 4% the rest). To nearest the root would have stopped
    after some ten steps, at a fifth of its value, and the update be several times as large."""
    lib()
    from fp8_dynamic_scaling_amd.optim import AdamW
    p = torch.nn.Parameter(torch.zeros(4096, device="cuda"))
    opt = AdamW([p], lr=1e-3, betas=(0.9, 0.999), weight_decay=0.0, state_bits=8)
    p.grad = torch.full((4096,), 0.01, device="cuda")
    for _ in range(300):
        before = p.detach().clone()
        opt.step()
    update = float((before - p.detach()).mean())
    assert abs(update / 1e-3 - 1) <= 0.05


# ---- together ---------------------------------------------------------------------------------------

def block(seed):
    from fp8_dynamic_scaling_amd import nn
    torch.manual_seed(seed)
    m = torch.nn.ModuleDict(dict(norm=nn.AddNorm(128, device="cuda"), mlp=nn.Float8GatedMLP(128, 256, device="cuda")))
    return m


def train(m, opt, x, res, dy, dh):
    y, h = m["norm"](x, res)
    out = m["mlp"](y)
    ps = list(m.parameters())
    gs = torch.autograd.grad((out, h), ps, (dy, dh), allow_unused=True)
    for p, g in zip(ps, gs):
        p.grad = g
    opt.step()
    return out.detach()


@pytest.mark.parametrize("bits", [8, 32])
def test_training_steps_captured(bits):
    """Norm, gated block, clipping and the optimizer's step captured into one graph; its replays over new inputs give
    the bits of eager steps on a copy."""
    lib()
    from fp8_dynamic_scaling_amd.optim import AdamW
    a, b = block(0), block(0)
    lr = torch.tensor([1e-2], device="cuda")
    kw = dict(lr=lr, state_bits=bits, max_norm=1.0, capturable=True, seed=11)
    oa, ob = AdamW(a.parameters(), **kw), AdamW(b.parameters(), **kw)
    x, res, dy, dh = (randn(64, 128, seed=i) for i in range(4))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        train(a, oa, x, res, dy, dh)
    torch.cuda.current_stream().wait_stream(side)
    train(b, ob, x, res, dy, dh)
    torch.cuda.synchronize()
    for p, q in zip(a.parameters(), b.parameters()):
        assert torch.equal(p, q)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = train(a, oa, x, res, dy, dh)
    for step in range(4):
        x.copy_(randn(64, 128, seed=100 + step))
        res.copy_(randn(64, 128, seed=200 + step))
        lr.fill_(1e-2 / (step + 1))
        graph.replay()
        want = train(b, ob, x, res, dy, dh)
        torch.cuda.synchronize()
        assert torch.equal(out, want), step
        for p, q in zip(a.parameters(), b.parameters()):
            assert torch.equal(p, q), step
        assert torch.equal(oa.grad_norm, ob.grad_norm)
    assert int(oa.state[next(a.parameters())]["step"]) == 5


def test_two_streams_at_once():
    """Two blocks stepped on two streams at the same time give what they give one after the other."""
    lib()
    from fp8_dynamic_scaling_amd.optim import AdamW
    ms, refs = [block(1), block(2)], [block(1), block(2)]
    kw = dict(lr=1e-2, state_bits=8, max_norm=1.0)
    opts, ropts = [AdamW(m.parameters(), **kw) for m in ms], [AdamW(m.parameters(), **kw) for m in refs]
    x, res, dy, dh = (randn(300, 128, seed=i) for i in range(4))
    streams = [torch.cuda.Stream() for _ in ms]
    torch.cuda.synchronize()
    for _ in range(3):
        for m, o, s in zip(ms, opts, streams):
            with torch.cuda.stream(s):
                train(m, o, x, res, dy, dh)
    torch.cuda.synchronize()
    for _ in range(3):
        for m, o in zip(refs, ropts):
            train(m, o, x, res, dy, dh)
    for m, r in zip(ms, refs):
        for p, q in zip(m.parameters(), r.parameters()):
            assert torch.equal(p, q)
