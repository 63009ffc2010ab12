"""The gated product and its backward against their formulas in 64 bits (GPU)."""
import numpy as np
import pytest
import torch

from tests.gpu_util import kpack, lib

pytestmark = pytest.mark.gpu

ACTS = {"silu": 0, "gelu": 1}
# half a step of bf16, relative to the value
BF16 = torch.finfo(torch.bfloat16).eps / 2
# sums: full precision rounds each of K additions to 24 bits; the FP8 instructions keep some 12 bits
# below an instruction's largest product, 2^-9 of the sum of magnitudes with an eightfold margin
FAST = 2.0 ** -9
# a sigmoid below fp32's smallest normal number, 2^-126, may come out as zero: that much absolute error
# in it, times what it is multiplied by; and as much in results that are themselves below it
TINY = 2.0 ** -126


def act64(x, act):
    """In 64 bits; GELU's (1 + tanh(z / 2)) / 2 as sigmoid(z): the sum would cancel to 2^-53, which is 1% of
    a value of 1e-14."""
    return x * torch.sigmoid(x if act == "silu" else (8 / np.pi) ** 0.5 * (x + 0.044715 * x ** 3))


def codes(g, shape, scale):
    """e4m3 codes [.., K] of N(0, scale) rows, their inverse scales and the values in 64 bits."""
    x = torch.randn(shape, generator=g) * scale
    inv = x.abs().amax(-1).clamp_min(1e-6) / 448.0
    q = (x / inv[..., None]).to(torch.float8_e4m3fn)
    return q.view(torch.uint8), inv, q.double() * inv.double()[..., None]


def check(out, gu, a, w, act, fast, label):
    """out and gu ([M][F], [M][2F] bf16 or None) against a [M][K], w [2F][K] in 64 bits."""
    F = w.shape[0] // 2
    p, S = a @ w.t(), a.abs() @ w.abs().t()
    acc = (FAST if fast else (a.shape[1] + 16) * 2.0 ** -23) * S + 2.0 ** -22 * p.abs()
    g, u, eg, eu = p[:, :F], p[:, F:], acc[:, :F], acc[:, F:]
    r = act64(g, act) * u
    # |act'| <= 1.13, |act(g)| <= |g|; the activation's exp2 of a rounded argument: 2^-22 (1 + |z|)
    z = g.abs() if act == "silu" else 1.6 * (g.abs() + 0.045 * g.abs() ** 3)
    tol = 1.13 * (eg * u.abs() + g.abs() * eu + eg * eu) + (BF16 + 2.0 ** -22 * (2 + z)) * r.abs() + TINY * (1 + (g * u).abs())
    bad = (out.double() - r).abs() / tol
    assert torch.isfinite(out).all() and bad.max() <= 1.0, (label, float(bad.max()))
    if gu is not None:
        bad = (gu.double() - p).abs() / (acc + BF16 * p.abs() + TINY)
        assert bad.max() <= 1.0, (label, "gu", float(bad.max()))


# M, F, K, packed: one token, tile borders, odd sizes and odd F, K of any multiple of 16, more tiles than CUs
DENSE = [(1, 16, 128, True), (1, 1, 16, False), (3, 7, 48, False), (5, 129, 256, False), (64, 48, 128, True),
         (255, 144, 256, True), (257, 272, 384, True), (300, 80, 640, False), (513, 515, 720, False),
         (260, 1000, 128, False), (1024, 1040, 256, True), (2048, 2064, 128, False), (33, 8192, 256, True),
         (17, 8200, 256, False), (2, 4096, 1040, False),
         # the large kernel's last stage of 64: one of 16, 32 and 48, with two stages, three and more
         (1500, 1000, 80, False), (1500, 1001, 144, False), (1500, 1000, 176, False), (1301, 1200, 224, False),
         (1500, 1000, 304, False), (1500, 1000, 720, False), (1500, 1008, 128, True)]


@pytest.mark.parametrize("M,F,K,packed", DENSE)
@pytest.mark.parametrize("fast", [True, False])
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_gated_mm(M, F, K, packed, fast, act):
    f = lib()
    g = torch.Generator().manual_seed(M * 7 + F * 3 + K)
    a, ai, av = codes(g, (M, K), 1.0)
    b, bi, bv = codes(g, (2 * F, K), 2.0 / K ** 0.5)
    bd = torch.from_numpy(kpack(b.numpy())) if packed else b
    guard = 256
    full = torch.full((M * F + 2 * guard,), 7.5, dtype=torch.bfloat16, device="cuda")
    full2 = torch.full((2 * M * F + 2 * guard,), 7.5, dtype=torch.bfloat16, device="cuda")
    out, gu = full[guard:-guard].view(M, F), full2[guard:-guard].view(M, 2 * F)
    f.fp8_gated_mm(a.cuda(), bd.cuda(), f.E4M3_NATIVE, f.SCALE_ROW, ai.cuda(), bi.cuda(), ACTS[act], gu, out,
                   packed=packed, use_fast_accum=fast)
    check(out.cpu(), gu.cpu(), av, bv, act, fast, (M, F, K))
    for t in (full, full2):
        assert (t[:guard] == 7.5).all() and (t[-guard:] == 7.5).all(), "write outside the output"
    again = torch.empty_like(out)  # the projections are not wanted: the same product
    f.fp8_gated_mm(a.cuda(), bd.cuda(), f.E4M3_NATIVE, f.SCALE_ROW, ai.cuda(), bi.cuda(), ACTS[act], None, again,
                   packed=packed, use_fast_accum=fast)
    assert torch.equal(again.view(torch.int16), out.view(torch.int16))


@pytest.mark.parametrize("M,F,K,packed", [(5, 48, 128, True), (300, 80, 144, False), (700, 1040, 256, True),
                                          (1030, 1100, 128, False)])
@pytest.mark.parametrize("fast", [True, False])
def test_gated_mm_tensorwise(M, F, K, packed, fast):
    f = lib()
    g = torch.Generator().manual_seed(M + F + K)
    a, _, av = codes(g, (M, K), 1.0)
    b, _, bv = codes(g, (2 * F, K), 2.0 / K ** 0.5)
    sa, sb = torch.tensor([0.02]), torch.tensor([0.004])
    av, bv = a.view(torch.float8_e4m3fn).double() * sa.double(), b.view(torch.float8_e4m3fn).double() * sb.double()
    bd = torch.from_numpy(kpack(b.numpy())) if packed else b
    out = torch.empty((M, F), dtype=torch.bfloat16, device="cuda")
    gu = torch.empty((M, 2 * F), dtype=torch.bfloat16, device="cuda")
    f.fp8_gated_mm(a.cuda(), bd.cuda(), f.E4M3_NATIVE, f.SCALE_TENSOR, sa.cuda(), sb.cuda(), f.ACT_SILU, gu, out,
                   packed=packed, use_fast_accum=fast)
    check(out.cpu(), gu.cpu(), av, bv, "silu", fast, (M, F, K))


# rows of each expert (empty ones among them), rows of none at the end
GROUPED = [([0, 1, 0, 3], 0, 16, 128, True), ([5, 0, 250, 9], 6, 144, 256, True), ([300, 257, 0, 1], 2, 80, 128, True),
           ([0, 0, 0], 4, 48, 128, True), ([7, 0, 3], 0, 33, 48, False), ([129, 130, 0, 4], 3, 136, 272, False),
           ([300, 0, 2], 1, 200, 384, False), ([1, 513, 0], 2, 264, 208, False)]


@pytest.mark.parametrize("rows,pad,F,K,packed", GROUPED)
@pytest.mark.parametrize("fast", [True, False])
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_grouped_gated_mm(rows, pad, F, K, packed, fast, act):
    f = lib()
    E, M = len(rows), sum(rows) + pad
    g = torch.Generator().manual_seed(M * 5 + F + K)
    a, ai, av = codes(g, (M, K), 1.0)
    b, bi, bv = codes(g, (E, 2 * F, K), 2.0 / K ** 0.5)
    off = torch.tensor([0] + list(np.cumsum(rows)), dtype=torch.int32)
    ad = torch.from_numpy(kpack(a.numpy(), 2)).view(M, K) if packed else a
    bd = torch.from_numpy(kpack(b.numpy())) if packed else b
    out = torch.full((M, F), 7.5, dtype=torch.bfloat16, device="cuda")
    gu = torch.full((M, 2 * F), 7.5, dtype=torch.bfloat16, device="cuda")
    f.fp8_grouped_gated_mm(ad.cuda(), bd.cuda(), f.E4M3_NATIVE, ai.cuda(), bi.cuda(), off.cuda(), ACTS[act], gu, out,
                           packed=packed, use_fast_accum=fast)
    out, gu = out.cpu(), gu.cpu()
    for e in range(E):
        lo, hi = int(off[e]), int(off[e + 1])
        if lo < hi:
            check(out[lo:hi], gu[lo:hi], av[lo:hi], bv[e], act, fast, (rows, e))
    assert (out[sum(rows):] == 7.5).all() and (gu[sum(rows):] == 7.5).all(), "rows behind the last expert were written"


def test_gated_mm_empty_sum():
    f = lib()
    out = torch.full((3, 5), 7.5, dtype=torch.bfloat16, device="cuda")
    gu = torch.full((3, 10), 7.5, dtype=torch.bfloat16, device="cuda")
    a, b = torch.empty((3, 0), dtype=torch.uint8, device="cuda"), torch.empty((10, 0), dtype=torch.uint8, device="cuda")
    f.fp8_gated_mm(a, b, f.E4M3_NATIVE, f.SCALE_ROW, None, None, f.ACT_SILU, gu, out)
    assert (out == 0).all() and (gu == 0).all()


@pytest.mark.parametrize("offsets", [(0, 2, 2, 4), (0, 0, 0, 0), (0, 0, 7, 7)])
def test_grouped_gated_mm_empty_sum(offsets):
    """No terms: zeros in the experts' rows, and nothing behind them."""
    f = lib()
    M, F, E = 7, 5, len(offsets) - 1
    out = torch.full((M, F), 7.5, dtype=torch.bfloat16, device="cuda")
    gu = torch.full((M, 2 * F), 7.5, dtype=torch.bfloat16, device="cuda")
    a = torch.empty((M, 0), dtype=torch.uint8, device="cuda")
    b = torch.empty((E, 2 * F, 0), dtype=torch.uint8, device="cuda")
    off = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    for g in (gu, None):
        f.fp8_grouped_gated_mm(a, b, f.E4M3_NATIVE, None, None, off, f.ACT_SILU, g, out)
        n = offsets[-1]
        assert (out[:n] == 0).all() and (out[n:] == 7.5).all()
        assert (gu[:n] == 0).all() and (gu[n:] == 7.5).all()


def test_gated_mm_large_gates():
    """Gates far out on both sides: act goes to 0 and to the gate, without overflow of the exponential."""
    f = lib()
    K, F = 128, 32
    a = torch.full((2, K), 0x7E, dtype=torch.uint8)  # 448
    a[1] = 0xFE  # -448
    b = torch.full((2 * F, K), 0x38, dtype=torch.uint8)  # 1
    inv_a, inv_b = torch.ones(2), torch.full((2 * F,), 0.05)
    for act in ACTS:
        out = torch.empty((2, F), dtype=torch.bfloat16, device="cuda")
        f.fp8_gated_mm(a.cuda(), b.cuda(), f.E4M3_NATIVE, f.SCALE_ROW, inv_a.cuda(), inv_b.cuda(), ACTS[act], None, out)
        x = 448.0 * K * 0.05
        assert (out[1].float() == 0).all()
        assert ((out[0].double() - x * x).abs() <= (BF16 + 2.0 ** -20) * x * x).all()


# ---- backward -------------------------------------------------------------------------------------

def bwd64(dh, gu, act):
    F = dh.shape[1]
    x = gu.double().requires_grad_(True)
    y = act64(x[:, :F], act) * x[:, F:]
    return torch.autograd.grad(y, x, dh.double())[0], y.detach()


def run_bwd(f, dh, gu, act, e5, want_h=True):
    M, F = dh.shape
    bf = dict(dtype=torch.bfloat16, device="cuda")
    dgu, h = torch.empty((M, 2 * F), **bf), torch.empty((M, F), **bf) if want_h else None
    q = torch.empty((M, 2 * F), dtype=torch.uint8, device="cuda")
    sc, inv = torch.empty(M, device="cuda"), torch.empty(M, device="cuda")
    f.fp8_gated_bwd(dh, gu, ACTS[act], f.E5M2_NATIVE if e5 else f.E4M3_NATIVE, 1e-12, dgu, q, sc, inv, h=h)
    return dgu, q.view(torch.float8_e5m2 if e5 else torch.float8_e4m3fn), sc, inv, h


@pytest.mark.parametrize("M,F", [(1, 8), (3, 504), (4, 512), (5, 520), (2, 1024), (7, 1032), (2, 8192), (3, 8200),
                                 (2, 14336), (1, 16392), (2, 32768), (301, 2056)])
@pytest.mark.parametrize("act,e5", [("silu", True), ("gelu", False)])
def test_gated_bwd(M, F, act, e5):
    f = lib()
    g = torch.Generator().manual_seed(M + F)
    gu = (torch.randn((M, 2 * F), generator=g) * 2).to(torch.bfloat16)
    dh = (torch.randn((M, F), generator=g) * 1e-3).to(torch.bfloat16)
    dgu, q, sc, inv, h = run_bwd(f, dh.cuda(), gu.cuda(), act, e5)
    d, y = bwd64(dh, gu, act)
    # fp32 steps: act' is a sum of terms up to 1 + |g| whose cancellation leaves an absolute error; the
    # factor |dh u| or |dh| goes with it
    G = gu[:, :F].double().abs()
    z = G if act == "silu" else 1.6 * (G + 0.045 * G ** 3)
    each = 2.0 ** -21 * (1 + G) * (2 + z) + TINY * (1 + G) * (3 + 3 * z)
    slack = torch.cat([each * (dh.double() * gu[:, F:].double()).abs(), each * dh.double().abs()], 1)
    assert ((dgu.cpu().double() - d).abs() <= BF16 * d.abs() + slack + TINY).all()
    eh = (BF16 + 2.0 ** -21 * (2 + z)) * y.abs() + TINY * (1 + (gu[:, :F].double() * gu[:, F:].double()).abs())
    assert ((h.cpu().double() - y).abs() <= eh).all()
    top = 57344.0 if e5 else 448.0
    amax = d.abs().amax(1)
    near = slack.amax(1) / amax + 2.0 ** -22
    assert ((inv.cpu().double() * top / amax - 1).abs() <= near).all()
    assert ((sc.cpu().double() * inv.cpu().double() - 1).abs() <= 2.0 ** -22).all()
    half, least = (2.0 ** -3, 2.0 ** -17) if e5 else (2.0 ** -4, 2.0 ** -10)
    back = q.cpu().double() * inv.cpu().double()[:, None]
    tol = half * d.abs() + least * inv.cpu().double()[:, None] + 2 * slack + near[:, None] * d.abs()
    assert ((back - d).abs() <= tol).all()


def test_gated_bwd_parts_and_in_place():
    """Each output alone gives the same bits; dgu may take gu's place and h dh's."""
    f = lib()
    g = torch.Generator().manual_seed(5)
    gu = (torch.randn((9, 2 * 1032), generator=g)).to(torch.bfloat16).cuda()
    dh = (torch.randn((9, 1032), generator=g)).to(torch.bfloat16).cuda()
    dgu, q, sc, inv, h = run_bwd(f, dh, gu, "silu", True)
    bits = lambda t: t.view(torch.int16)  # noqa: E731
    one = torch.empty_like(dgu)
    f.fp8_gated_bwd(dh, gu, f.ACT_SILU, f.E5M2_NATIVE, 1e-12, one, None, None)
    assert torch.equal(bits(one), bits(dgu))
    q1, s1 = torch.empty(q.shape, dtype=torch.uint8, device="cuda"), torch.empty_like(sc)
    f.fp8_gated_bwd(dh, gu, f.ACT_SILU, f.E5M2_NATIVE, 1e-12, None, q1, s1)
    assert torch.equal(q1, q.view(torch.uint8)) and torch.equal(s1, sc)
    gu2, dh2 = gu.clone(), dh.clone()
    f.fp8_gated_bwd(dh2, gu2, f.ACT_SILU, f.E5M2_NATIVE, 1e-12, gu2, q1, s1, h=dh2)
    assert torch.equal(bits(gu2), bits(dgu)) and torch.equal(bits(dh2), bits(h)) and torch.equal(q1, q.view(torch.uint8))


@pytest.mark.parametrize("F", [64, 2056])
@pytest.mark.parametrize("e5", [True, False])
def test_gated_bwd_rows_of_zeros_and_not_finite(F, e5):
    f = lib()
    g = torch.Generator().manual_seed(F)
    gu, dh = torch.randn((6, 2 * F), generator=g).to(torch.bfloat16), torch.randn((6, F), generator=g).to(torch.bfloat16)
    dh[0] = 0
    dh[2, 5] = float("nan")
    dh[4, F - 1] = float("inf")
    clean = run_bwd(f, dh[[1, 3, 5]].cuda().contiguous(), gu[[1, 3, 5]].cuda().contiguous(), "silu", e5)
    dgu, q, sc, inv, h = run_bwd(f, dh.cuda(), gu.cuda(), "silu", e5)
    top = 57344.0 if e5 else 448.0
    assert (q[0].float() == 0).all() and float(sc[0]) == np.float32(top / 1e-12)
    assert torch.isnan(sc[[2, 4]]).all() and torch.isnan(inv[[2, 4]]).all()
    assert torch.isnan(dgu[2, 5]) and torch.isinf(dgu[4, F - 1])
    for a, b in zip((dgu, q, sc, inv, h), clean):  # the other rows are not touched by it
        assert torch.equal(a[[1, 3, 5]].view(torch.uint8), b.view(torch.uint8))


def test_gated_bwd_empty_rows():
    f = lib()
    sc, inv = torch.empty(3, device="cuda"), torch.empty(3, device="cuda")
    e = torch.empty((3, 0), dtype=torch.bfloat16, device="cuda")
    f.fp8_gated_bwd(e, e, f.ACT_SILU, f.E5M2_NATIVE, 1e-12, None, torch.empty((3, 0), dtype=torch.uint8, device="cuda"),
                    sc, inv)
    assert (sc == np.float32(57344.0 / 1e-12)).all()


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_gated_bwd_gates_far_out(act):
    """Gates up to bf16's largest: act' is 1 or 0, nothing overflows on the way."""
    f = lib()
    g = torch.tensor([[3e38, 1e20, 1e13, 100.0, -100.0, -1e13, -1e20, -3e38]]).to(torch.bfloat16)
    u = torch.full_like(g, 0.5)
    dh = torch.ones_like(g)
    dgu, q, sc, inv, h = run_bwd(f, dh.cuda(), torch.cat([g, u], 1).cuda(), act, False)
    dgu = dgu.cpu().float()
    assert torch.equal(dgu[0, :4], torch.full((4,), 0.5)) and (dgu[0, 4:8] == 0).all()
    assert torch.equal(dgu[0, 8:12], g[0, :4].float()) and (dgu[0, 12:] == 0).all()
    assert torch.isfinite(inv).all()


def test_formats_that_are_refused():
    f = lib()
    out = torch.empty((2, 16), dtype=torch.bfloat16, device="cuda")
    a, b = (torch.zeros((n, 128), dtype=torch.uint8, device="cuda") for n in (2, 32))
    inv = torch.ones(32, device="cuda")
    for fmt in (f.E5M2_NATIVE, f.E4M3FNUZ):
        with pytest.raises(f.Fp8Error) as e:
            f.fp8_gated_mm(a, b, fmt, f.SCALE_ROW, inv, inv, f.ACT_SILU, None, out)
        assert e.value.status == f.ERR_UNSUPPORTED
    dh = torch.zeros((2, 16), dtype=torch.bfloat16, device="cuda")
    gu = torch.zeros((2, 32), dtype=torch.bfloat16, device="cuda")
    q = torch.empty((2, 32), dtype=torch.uint8, device="cuda")
    with pytest.raises(f.Fp8Error) as e:
        f.fp8_gated_bwd(dh, gu, f.ACT_SILU, f.E5M2FNUZ, 1e-12, None, q, inv[:2].clone())
    assert e.value.status == f.ERR_UNSUPPORTED


@pytest.mark.parametrize("grouped", [False, True])
def test_past_32_bits_of_elements(grouped):
    """Projections of more than 2^31 elements: rows at both ends, forward and backward."""
    f = lib()
    M, F, K = 76000, 14336, 128
    g = torch.Generator().manual_seed(4)
    a, ai, av = codes(g, (M, K), 1.0)
    b, bi, bv = codes(g, (2 * F, K), 2.0 / K ** 0.5)
    out = torch.empty((M, F), dtype=torch.bfloat16, device="cuda")
    gu = torch.empty((M, 2 * F), dtype=torch.bfloat16, device="cuda")
    assert gu.numel() > 1 << 31
    if grouped:
        off = torch.tensor([0, 70000, M], dtype=torch.int32, device="cuda")
        bb, bbi = torch.stack([b, b]).cuda(), torch.stack([bi, bi]).cuda()
        f.fp8_grouped_gated_mm(a.cuda(), bb, f.E4M3_NATIVE, ai.cuda(), bbi, off, f.ACT_SILU, gu, out)
    else:
        f.fp8_gated_mm(a.cuda(), b.cuda(), f.E4M3_NATIVE, f.SCALE_ROW, ai.cuda(), bi.cuda(), f.ACT_SILU, gu, out)
    rows = torch.tensor([0, 1, M // 2, 74899, 74900, M - 2, M - 1])
    check(out[rows.cuda()].cpu(), gu[rows.cuda()].cpu(), av[rows], bv, "silu", True, "far rows")
    if grouped:
        return
    q, sc = torch.empty((M, 2 * F), dtype=torch.uint8, device="cuda"), torch.empty(M, device="cuda")
    keep = gu[rows.cuda()].clone()
    dh = out  # any gradient will do
    f.fp8_gated_bwd(dh, gu, f.ACT_SILU, f.E5M2_NATIVE, 1e-12, gu, q, sc)
    few = run_bwd(f, dh[rows.cuda()].contiguous(), keep, "silu", True)
    assert torch.equal(gu[rows.cuda()].view(torch.int16), few[0].view(torch.int16))
    assert torch.equal(q[rows.cuda()], few[1].view(torch.uint8)) and torch.equal(sc[rows.cuda()], few[2])
