"""The residual norm on the GPU: fp8_add_norm_quant_row bit for bit against the oracle's
normalization and rowwise quantization of h = bf16(x + res), and fp8_add_norm_bwd against
its formula in 64 bits and against differences of the forward."""
import numpy as np
import pytest

import oracle
import synth
from tests.gpu_util import gpu, have_gpu, lib, to_dev, to_dev_bf16

pytestmark = [gpu, pytest.mark.skipif(not have_gpu(), reason="needs an MI355X")]
EPS, NEPS = 1e-12, 1e-5


@pytest.fixture(scope="module")
def f():
    oracle.build(force=False)
    synth.build(force=False)
    return lib()


def _bits(v):
    """float64 -> nearest bf16 (ties to even) as uint16, through fp32."""
    u = np.asarray(v, np.float32).view(np.uint32)
    return ((u + 0x7FFF + ((u >> 16) & 1)) >> 16).astype(np.uint16)


def _val(b):
    return oracle.bf16_to_f32(b).astype(np.float64)


def _inputs(rows, cols, seed, layer):
    x = synth.normal_bf16((rows, cols), seed, 1.0)
    r = synth.normal_bf16((rows, cols), seed + 1, 2.0)
    g = _bits(oracle.bf16_to_f32(synth.normal_bf16((1, cols), seed + 2, 0.1).reshape(cols)) + np.float32(1.0))
    b = synth.normal_bf16((1, cols), seed + 3, 0.1).reshape(cols) if layer else None
    return x, r, g, b


def _sum_bits(x, r):
    return _bits(oracle.bf16_to_f32(x) + oracle.bf16_to_f32(r))


def _forward(f, x, r, g, b, layer, fmt, h="new", want_y=True, want_q=True, neps=NEPS):
    import torch
    rows, cols = x.shape
    f32 = dict(dtype=torch.float32, device="cuda:0")
    xd, rd = to_dev_bf16(x), None if r is None else to_dev_bf16(r)
    hd = {"new": torch.empty_like(xd), "x": xd, "res": rd, None: None}[h]
    y = torch.empty_like(xd) if want_y else None
    q = torch.empty((rows, cols), dtype=torch.uint8, device="cuda:0") if want_q else None
    sc, iv = torch.empty(rows, **f32), torch.empty(rows, **f32)
    mean, rstd = torch.empty(rows, **f32) if layer else None, torch.empty(rows, **f32)
    f.fp8_add_norm_quant_row(xd, rd, to_dev_bf16(g), None if b is None else to_dev_bf16(b),
                             f.NORM_LAYER if layer else f.NORM_RMS, neps, fmt, EPS, hd, y, q, sc if want_q else None,
                             iv if want_q else None, mean=mean, rstd=rstd)
    torch.cuda.synchronize()
    n = lambda t: None if t is None else (t.view(torch.int16).cpu().numpy().view(np.uint16)  # noqa: E731
                                          if t.dtype == torch.bfloat16 else t.cpu().numpy())
    return dict(h=n(hd), y=n(y), q=n(q), scale=n(sc), inv=n(iv), mean=n(mean), rstd=n(rstd))


# rows held by one wavefront (up to 4096 columns) and by four, with a full and a ragged
# last piece, one row and row counts that leave part of a workgroup idle
SHAPES = [(1, 8), (1, 4096), (3, 1000), (5, 2056), (130, 1024), (7, 4104), (2, 7168), (3, 16384), (1025, 512)]


@pytest.mark.parametrize("layer", [False, True], ids=["rms", "layer"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_forward_bits(f, shape, layer):
    x, r, g, b = _inputs(*shape, 4100 + shape[1], layer)
    h = _sum_bits(x, r)
    for fmt, name in ((f.E4M3_NATIVE, "e4m3fn"), (f.E5M2_NATIVE, "e5m2")):
        got = _forward(f, x, r, g, b, layer, fmt)
        ry, rq, rs, ri = oracle.norm_quant_row(h, g, b, layer, NEPS, name, EPS)
        assert np.array_equal(got["h"], h)
        assert np.array_equal(got["y"], ry) and np.array_equal(got["q"], rq)
        assert np.array_equal(got["scale"], rs) and np.array_equal(got["inv"], ri)
    hv = _val(h)
    mean = hv.mean(1)
    var = (hv - mean[:, None] * layer).__pow__(2).mean(1)
    rstd = 1.0 / np.sqrt(var + NEPS)
    # fp32 values of statistics in 64 bits: half a step, 2^-24, and 2^-40 for this
    # reference's own sums; the mean's own sums cancel, so its error goes by mean |h|
    assert np.all(np.abs(got["rstd"] - rstd) <= rstd * (2.0 ** -24 + 2.0 ** -40))
    if layer:
        assert np.all(np.abs(got["mean"] - mean) <= np.abs(mean) * 2.0 ** -24 + np.abs(hv).mean(1) * 2.0 ** -40)


def test_forward_without_residual_is_the_plain_norm(f):
    x, _, g, b = _inputs(9, 520, 4300, True)
    got = _forward(f, x, None, g, b, True, f.E4M3_NATIVE, h=None)
    ry, rq, rs, ri = oracle.norm_quant_row(x, g, b, True, NEPS, "e4m3fn", EPS)
    assert np.array_equal(got["y"], ry) and np.array_equal(got["q"], rq)
    assert np.array_equal(got["scale"], rs) and np.array_equal(got["inv"], ri)


@pytest.mark.parametrize("cols", [264, 6000])
@pytest.mark.parametrize("h", ["x", "res", None])
def test_forward_in_place_and_partial_outputs(f, h, cols):
    x, r, g, _ = _inputs(11, cols, 4400, False)
    ref = _sum_bits(x, r)
    ry, rq, rs, _ = oracle.norm_quant_row(ref, g, None, False, NEPS, "e4m3fn", EPS)
    got = _forward(f, x, r, g, None, False, f.E4M3_NATIVE, h=h, want_y=False)
    assert np.array_equal(got["q"], rq) and np.array_equal(got["scale"], rs)
    assert h is None or np.array_equal(got["h"], ref)
    got = _forward(f, x, r, g, None, False, f.E4M3_NATIVE, h=h, want_q=False)
    assert np.array_equal(got["y"], ry) and (h is None or np.array_equal(got["h"], ref))


def test_forward_rows_that_cancel(f):
    """x + res = 0 in whole rows (statistics of zeros) and in all but one element."""
    x, r, g, b = _inputs(4, 1032, 4500, True)
    r[0] = x[0] ^ 0x8000
    r[1] = x[1] ^ 0x8000
    r[1, 7] = 0x4000
    for layer in (False, True):
        bb = b if layer else None
        got = _forward(f, x, r, g, bb, layer, f.E4M3_NATIVE)
        ry, rq, rs, ri = oracle.norm_quant_row(_sum_bits(x, r), g, bb, layer, NEPS, "e4m3fn", EPS)
        assert np.array_equal(got["y"], ry) and np.array_equal(got["q"], rq) and np.array_equal(got["scale"], rs)


# ---- backward ---------------------------------------------------------------------------

def _reference(dy, dh, h, g, mean, rstd, layer):
    """The formula in 64 bits on the kernel's inputs, and the sum of magnitudes that each
    output's fp32 operations act on."""
    r = rstd.astype(np.float64)[:, None]
    xh = (h - mean.astype(np.float64)[:, None]) * r if layer else h * r
    u = dy * g
    c1 = u.mean(1, keepdims=True) if layer else 0.0
    c2 = (u * xh).mean(1, keepdims=True)
    dx = dh + r * (u - c1 - xh * c2)
    mag = np.abs(dh) + r * (np.abs(u) + (np.abs(u).mean(1, keepdims=True) if layer else 0.0) +
                            np.abs(xh) * np.abs(u * xh).mean(1, keepdims=True))
    if layer:  # (h - mean) rounds relative to itself; its product with rstd once more
        mag = mag + r * np.abs(xh) * np.abs(u).mean(1, keepdims=True)
    return dx, mag, (dy * xh).sum(0), np.abs(dy * xh).sum(0), dy.sum(0), np.abs(dy).sum(0)


def _backward(f, dy, dh, h, g, mean, rstd, layer, dx="new", want_cols=True):
    import torch
    rows, cols = dy.shape
    kind = f.NORM_LAYER if layer else f.NORM_RMS
    dyd, dhd, hd = to_dev_bf16(dy), None if dh is None else to_dev_bf16(dh), to_dev_bf16(h)
    gd = to_dev_bf16(g)
    dxd = {"new": torch.empty_like(dyd), "dy": dyd, "dh": dhd}[dx]
    dg = torch.empty_like(gd) if want_cols else None
    db = torch.empty_like(gd) if layer and want_cols else None
    n = f.fp8_add_norm_bwd_ws_bytes(rows, cols, kind)
    ws = torch.full((n + 4096,), 0xA5, dtype=torch.uint8, device="cuda:0") if want_cols else None
    f.fp8_add_norm_bwd(dyd, dhd, hd, gd, to_dev(mean) if layer else None, to_dev(rstd), kind, dxd, dg, db,
                       ws[:n] if want_cols else None)
    torch.cuda.synchronize()
    if want_cols:
        assert bool((ws[n:] == 0xA5).all()), "write behind the workspace"
    c = lambda t: None if t is None else t.double().cpu().numpy()  # noqa: E731
    return c(dxd), c(dg), c(db)


def _check_backward(f, rows, cols, layer, seed, with_dh=True, dx="new"):
    x, r, g, _ = _inputs(rows, cols, seed, False)
    h = _sum_bits(x, r)
    hv = _val(h)
    mean = hv.mean(1).astype(np.float32)
    rstd = (1.0 / np.sqrt((hv - hv.mean(1, keepdims=True) * layer).__pow__(2).mean(1) + NEPS)).astype(np.float32)
    dy = synth.normal_bf16((rows, cols), seed + 7, 1e-2)
    dh = synth.normal_bf16((rows, cols), seed + 8, 1e-2) if with_dh else None
    got, dg, db = _backward(f, dy, dh, h, g, mean, rstd, layer, dx=dx)
    ref, mag, rg, mg, rb, mb = _reference(_val(dy), _val(dh) if with_dh else 0.0, hv, _val(g), mean, rstd, layer)
    # dx: the bf16 rounding, half a step, and fp32 operations: a row's sums have at most
    # 16 + 6 + 16 additions and each term some 8 roundings, 2^-24 each of the magnitudes
    assert np.all(np.abs(got - ref) <= 2.0 ** -8 * np.abs(ref) + 64 * 2.0 ** -24 * mag + 1e-38)
    # the column sums: the bf16 rounding, and at most 4 + rows / 256 additions in a
    # workgroup, 4 + 16 + 32 across them and 6 roundings of a term
    chain = (64 + rows / 256) * 2.0 ** -24
    assert np.all(np.abs(dg - rg) <= 2.0 ** -8 * np.abs(rg) + chain * mg + 1e-38)
    if layer:
        assert np.all(np.abs(db - rb) <= 2.0 ** -8 * np.abs(rb) + chain * mb + 1e-38)


@pytest.mark.parametrize("layer", [False, True], ids=["rms", "layer"])
@pytest.mark.parametrize("shape", [(1, 8), (1, 4096), (5, 72), (17, 1024), (130, 1032), (301, 4096), (33, 5120),
                                   (6, 16384), (2100, 200)], ids=str)
def test_backward(f, shape, layer):
    _check_backward(f, *shape, layer, 4700 + shape[1])


@pytest.mark.parametrize("dx", ["dy", "dh"])
@pytest.mark.parametrize("cols", [512, 4096, 8200])
def test_backward_in_place(f, cols, dx):
    _check_backward(f, 40, cols, True, 4800, dx=dx)


def test_backward_without_stream_gradient(f):
    _check_backward(f, 19, 640, False, 4850, with_dh=False)


def test_backward_dx_alone_needs_no_workspace(f):
    x, r, g, _ = _inputs(12, 512, 4860, False)
    h = _sum_bits(x, r)
    rstd = (1.0 / np.sqrt(_val(h).__pow__(2).mean(1) + NEPS)).astype(np.float32)
    dy = synth.normal_bf16((12, 512), 4861, 1e-2)
    a, _, _ = _backward(f, dy, None, h, g, None, rstd, False)
    b, dg, _ = _backward(f, dy, None, h, g, None, rstd, False, want_cols=False)
    assert dg is None and np.array_equal(a, b)


def test_backward_of_no_rows_writes_zeros(f):
    import torch
    e = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda:0")
    g = torch.ones(64, dtype=torch.bfloat16, device="cuda:0")
    s = torch.empty(0, dtype=torch.float32, device="cuda:0")
    dg, db = torch.ones_like(g), torch.ones_like(g)
    f.fp8_add_norm_bwd(e, None, e, g, s, s, f.NORM_LAYER, e, dg, db, None)
    assert not bool(dg.any()) and not bool(db.any())


@pytest.mark.parametrize("layer", [False, True], ids=["rms", "layer"])
def test_backward_against_differences(f, layer):
    """sum(dx * v) against the central difference of sum(y * dy) + sum(h * dh) along v, in
    64 bits. The difference quotient at step 1e-4 is good to about 1e-7 of the terms'
    magnitudes; dx is rounded to bf16, half a step each."""
    rows, cols = 6, 328
    x, r, g, _ = _inputs(rows, cols, 4900, False)
    h = _sum_bits(x, r)
    hv, gv = _val(h), _val(g)
    dyb, dhb = synth.normal_bf16((rows, cols), 4901, 1.0), synth.normal_bf16((rows, cols), 4902, 1.0)
    dy, dh = _val(dyb), _val(dhb)
    v = np.random.default_rng(5).standard_normal((rows, cols))

    def loss(z):
        m = z.mean(1, keepdims=True) if layer else 0.0
        return ((z - m) / np.sqrt((z - m).__pow__(2).mean(1, keepdims=True) + NEPS) * gv * dy).sum() + (z * dh).sum()

    want = (loss(hv + 1e-4 * v) - loss(hv - 1e-4 * v)) / 2e-4
    mean = hv.mean(1).astype(np.float32)
    rstd = (1.0 / np.sqrt((hv - hv.mean(1, keepdims=True) * layer).__pow__(2).mean(1) + NEPS)).astype(np.float32)
    dx, _, _ = _backward(f, dyb, dhb, h, g, mean, rstd, layer)
    assert abs((dx * v).sum() - want) <= 2.0 ** -8 * np.abs(dx * v).sum() + 1e-6 * np.abs(dx * v).sum()


def test_two_calls_at_once_on_two_streams(f):
    """Backward calls on two streams with a workspace each: the bits of calls in turn."""
    import torch
    rows, cols = 700, 2048
    kind = f.NORM_RMS
    g = torch.Generator(device="cuda:0").manual_seed(3)
    mk = lambda *s: torch.randn(*s, generator=g, device="cuda:0").to(torch.bfloat16)  # noqa: E731
    sets = []
    for _ in range(2):
        h = mk(rows, cols)
        sets.append(dict(dy=mk(rows, cols), dh=mk(rows, cols), h=h, gamma=mk(cols),
                         rstd=torch.rsqrt(h.float().square().mean(1) + NEPS)))

    def call(s, stream=None):
        o = (torch.empty_like(s["dy"]), torch.empty_like(s["gamma"]))
        ws = torch.empty(f.fp8_add_norm_bwd_ws_bytes(rows, cols, kind), dtype=torch.uint8, device="cuda:0")
        torch.cuda.synchronize()
        f.fp8_add_norm_bwd(s["dy"], s["dh"], s["h"], s["gamma"], None, s["rstd"], kind, *o, None, ws, stream=stream)
        return o, ws

    want = [call(s)[0] for s in sets]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [call(s, st) for s, st in zip(sets, streams)]
    torch.cuda.synchronize()
    for a, (b, _) in zip(want, got):
        assert all(torch.equal(p, q) for p, q in zip(a, b))
