"""The residual norm and the router at calls beyond the ordinary ones: operands at any offset in
memory through autograd, rows that are not finite, more rows than one launch holds."""
import numpy as np
import pytest

import oracle
import synth
from tests.gpu_util import gpu, have_gpu, lib
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


# ---- rows that are not finite ---------------------------------------------------------------

NAN, PINF, NINF, MAX = 0x7FC0, 0x7F80, 0xFF80, 0x7F7F
# rows of inputs that are not finite, and sums of finite ones that pass bf16's range: in the
# addition, and in its rounding (the largest value and half a step more, a tie)
BAD = {1: (0, NAN, 0), 2: (5, PINF, 0), 3: (7, NINF, 0), 5: (0, MAX, MAX), 6: (3, 0, NAN), 8: (2, MAX, 0x7B00),
       10: (1, 0xFFC0, PINF)}


def _bad_inputs(cols, layer):
    x, r, g, b = _inputs(12, cols, 4990 + cols, layer)
    for row, (at, xv, rv) in BAD.items():
        x[row, at - cols // 2], r[row, at - cols // 2] = xv, rv
    x[9, 0], r[9, 0], x[9, cols - 1], r[9, cols - 1] = PINF, 0, NINF, 0  # both infinities
    return x, r, g, b, sorted([*BAD, 9])


def _formula(h, g, b, layer):
    """y (fp32, before its rounding), mean and rstd of rows of h by IEEE arithmetic."""
    with np.errstate(all="ignore"):
        v = oracle.bf16_to_f32(h)
        n = v.shape[1]
        mean = v.astype(np.float64).sum(1) / n if layer else np.zeros(len(v))
        rstd = 1.0 / np.sqrt((v.astype(np.float64) ** 2).sum(1) / n - mean * mean + NEPS)
        y = (v - mean.astype(np.float32)[:, None]) * rstd.astype(np.float32)[:, None] * oracle.bf16_to_f32(g)
        if layer:
            y = y + oracle.bf16_to_f32(b)
    return y.astype(np.float32), mean.astype(np.float32), rstd.astype(np.float32)


# both numbers of threads a row, one and several pieces a lane
@pytest.mark.parametrize("cols", [64, 1032, 2056, 6000])
@pytest.mark.parametrize("layer", [False, True], ids=["rms", "layer"])
def test_norm_rows_that_are_not_finite(f, layer, cols):
    """A row whose h has a NaN or an infinity has the formula's statistics and outputs (all NaN,
    or with an infinity under RMS zeros beside the NaN), and an inverse scale of NaN, whether y
    is written or not; the rows beside it have their own bits."""
    x, r, g, b, bad = _bad_inputs(cols, layer)
    good = [i for i in range(len(x)) if i not in bad]
    with np.errstate(all="ignore"):
        h = _bits(oracle.bf16_to_f32(x) + oracle.bf16_to_f32(r))
    for fmt, name in ((f.E4M3_NATIVE, "e4m3fn"), (f.E5M2_NATIVE, "e5m2")):
        got = _forward(f, x, r, g, b, layer, fmt)
        ry, rq, rs, ri = oracle.norm_quant_row(h[good], g, b, layer, NEPS, name, EPS)
        assert np.array_equal(got["h"][good], h[good])
        assert np.array_equal(got["y"][good], ry) and np.array_equal(got["q"][good], rq)
        assert np.array_equal(got["scale"][good], rs) and np.array_equal(got["inv"][good], ri)
        v = oracle.bf16_to_f32(got["h"][bad])
        assert not np.isfinite(v).all(1).any()
        y, mean, rstd = _formula(got["h"][bad], g, b, layer)
        assert np.array_equal(got["rstd"][bad], rstd, equal_nan=True)
        assert not layer or np.array_equal(got["mean"][bad], mean, equal_nan=True)
        gy = oracle.bf16_to_f32(got["y"][bad])
        assert np.array_equal(gy, y, equal_nan=True) and np.isnan(gy).any(1).all()  # 0 and NaN: exact in bf16
        assert np.isnan(got["inv"][bad]).all() and np.isnan(got["scale"][bad]).all()
        codes = _forward(f, x, r, g, b, layer, fmt, want_y=False)
        for part in ("q", "scale", "inv", "rstd"):
            assert np.array_equal(got[part], codes[part], equal_nan=part != "q"), part


@pytest.mark.parametrize("cols", [264, 6000])
def test_norm_outputs_that_are_not_finite(f, cols):
    """Finite rows with a weight that is not, and a row of zeros without a norm_eps (0 times
    infinity): y is the formula's, an inverse scale is NaN where y has a NaN, else infinite."""
    x, r, g, _ = _inputs(6, cols, 4995, False)
    h = _sum_bits(x, r)
    ry = oracle.norm_quant_row(h, g, None, False, NEPS, "e4m3fn", EPS)[0]
    for bits, test in ((NAN, np.isnan), (PINF, np.isinf)):
        bad = g.copy()
        bad[5] = bits
        got = _forward(f, x, r, bad, None, False, f.E4M3_NATIVE)
        y = oracle.bf16_to_f32(got["y"])
        assert test(y[:, 5]).all() and test(got["inv"]).all()
        keep = [c for c in range(cols) if c != 5]
        assert np.array_equal(got["y"][:, keep], ry[:, keep])
    r[2] = x[2] ^ 0x8000
    got = _forward(f, x, r, g, None, False, f.E4M3_NATIVE, neps=0.0)
    assert np.isnan(oracle.bf16_to_f32(got["y"][2])).all() and np.isnan(got["inv"][2])
    assert np.isfinite(got["inv"][[0, 1, 3, 4, 5]]).all()


@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_add_norm_hides_no_fault(f, kind):
    """A NaN in one row of the stream: the row's y and gradient and the weight's gradient are
    NaN, the other rows' as without it."""
    import torch
    from fp8_dynamic_scaling_amd.nn import AddNorm
    m = AddNorm(264, kind, device="cuda:0")
    x, res, dy, dh = (_randn(6, 264, seed=s) for s in (1, 2, 3, 4))
    keep = [0, 1, 2, 4, 5]

    def step(x):
        x = x.clone().requires_grad_(True)
        y, h = m(x, res)
        return (y, *torch.autograd.grad([y, h], [x, m.weight], [dy, dh]))

    clean = step(x)
    x[3, 100] = float("nan")
    y, dx, dw = step(x)
    assert bool(y[3].isnan().all()) and bool(dx[3].isnan().all()) and bool(dw.isnan().all())
    assert torch.equal(y[keep], clean[0][keep]) and torch.equal(dx[keep], clean[1][keep])


# ---- more rows than a launch holds ----------------------------------------------------------


@pytest.mark.parametrize("rows,cols", [((1 << 26) + 5, 8), ((1 << 23) + 3, 2056)], ids=["wave", "workgroup"])
def test_norm_rows_past_a_grid(f, rows, cols):
    """A grid has fewer than 2^32 threads, 64 or 256 of them a row. Rows do not depend on each
    other, so those at both ends and where a second launch begins are those of calls alone."""
    import torch
    bf = dict(dtype=torch.bfloat16, device="cuda:0")
    x, gamma, beta = torch.empty(rows, cols, **bf).normal_(), _randn(cols, seed=5), _randn(cols, seed=6)

    def forward(x):
        n = len(x)
        q = torch.full((n, cols), 0xA5, dtype=torch.uint8, device="cuda:0")
        s = [torch.full((n,), -7.0, device="cuda:0") for _ in range(4)]
        f.fp8_add_norm_quant_row(x, None, gamma, beta, f.NORM_LAYER, NEPS, f.E4M3_NATIVE, EPS, None, None, q, *s[:2],
                                 mean=s[2], rstd=s[3])
        return q, *s

    whole = forward(x)
    assert bool((whole[1] > 0).all()) and bool((whole[4] > 0).all())
    for at in (0, 1 << 23, 1 << 24, 1 << 25, 1 << 26, rows):
        lo, hi = max(0, at - 9), min(rows, at + 9)
        if lo < hi:
            for a, b in zip(whole, forward(x[lo:hi].clone())):
                assert torch.equal(a[lo:hi], b), at


@pytest.mark.parametrize("T,E,k", [((1 << 30) + 70, 1, 1), ((1 << 25) + 5, 520, 2)])
def test_route_backward_tokens_past_a_grid(f, T, E, k):
    import torch
    l = torch.empty(T, E, dtype=torch.bfloat16, device="cuda:0").normal_()
    ids, w = torch.empty(T, k, dtype=torch.int32, device="cuda:0"), torch.empty(T, k, device="cuda:0")
    f.fp8_moe_route(l, f.GATE_SIGMOID, ids, w)
    dw = torch.empty(T, k, device="cuda:0").normal_()
    alone = {}
    for at in (0, 1 << 25, 1 << 29, 1 << 30, T):
        lo, hi = max(0, at - 70), min(T, at + 70)
        if lo < hi:
            part = [t[lo:hi].clone() for t in (l, ids, w, dw)]
            alone[lo, hi] = torch.full_like(part[0], 7.0)
            f.fp8_moe_route_bwd(part[0], f.GATE_SIGMOID, *part[1:], alone[lo, hi])
    f.fp8_moe_route_bwd(l, f.GATE_SIGMOID, ids, w, dw, l)  # in place
    for (lo, hi), b in alone.items():
        assert torch.equal(l[lo:hi], b), (lo, hi)
    # every token: w (1 - w) <= 1/4, so |dl| <= |dw| / 4, half a step of bf16 (2^-8 of it) and a few of
    # fp32 above that: 0.25 (1 + 2^-8) = 0.25098
    n = 1 << 22
    for a, d in zip(l.split(n), dw.split(n)):
        assert bool((a.abs().amax(1) <= 0.251 * d.abs().amax(1)).all())


# ---- codes in torch's float8 tensors ----------------------------------------------------------


def test_codes_in_float8_tensors(f):
    """The norm's codes and the expert layer's weights as torch.float8_e4m3fn: the same bytes."""
    import torch
    from tests.test_gpu_moe import Layer, _tokens
    x, res, gamma = _randn(5, 264, seed=1), _randn(5, 264, seed=2), _randn(264, seed=3)
    got = []
    for dtype in (torch.uint8, torch.float8_e4m3fn):
        q, s = torch.empty(5, 264, dtype=dtype, device="cuda:0"), torch.empty(5, device="cuda:0")
        f.fp8_add_norm_quant_row(x, res, gamma, None, f.NORM_RMS, NEPS, f.E4M3_NATIVE, EPS, None, None, q, s)
        got.append(q.view(torch.uint8))
    assert torch.equal(*got)
    layer = Layer(4, 128, 64, 800, False)
    x, ids, w = _tokens(3, 4, 2, 128, 801)
    ws = torch.empty(f.fp8_moe_few_ws_bytes(3, 2, 64), dtype=torch.uint8, device="cuda:0")
    out = []
    for view in (torch.uint8, torch.float8_e4m3fn):
        out.append(torch.empty_like(x))
        f.fp8_moe_few(x, ids, w, layer.w13.view(view), layer.i13, layer.w2.view(view), layer.i2, f.E4M3_NATIVE, out[-1],
                      ws)
    assert torch.equal(*out)


def test_add_norm_refuses_parameters_of_another_size(f):
    import torch
    from fp8_dynamic_scaling_amd.nn import AddNorm
    x = _randn(3, 64, seed=1)
    for name in ("weight", "bias"):
        for size in (56, 72):
            m = AddNorm(64, "layer", device="cuda:0")
            setattr(m, name, torch.nn.Parameter(_randn(size, seed=2)))
            with torch.no_grad(), pytest.raises(ValueError, match="64 features, " + name):
                m(x)
