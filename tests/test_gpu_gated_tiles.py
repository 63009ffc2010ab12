"""The gated product on each form of its kernel for many rows (GPU): tiles of 64, 128 and 256 rows, row-major and packed
weights, dense and grouped, fast and full-precision sums, with six stages of K at least and more tiles than CUs, so that
the loop's steady part and the loads under an epilogue run; and products whose weights are past 32-bit offsets. That each
shape has the tile it is listed under is checked on the host (test_gated_tiles_host.py)."""
import numpy as np
import pytest
import torch

from tests.gpu_util import lib
from tests.test_gpu_gated import ACTS, check, codes

pytestmark = pytest.mark.gpu

# rows of a tile, M, F, K, packed. K past a stage of 64: 0, 16, 32, 48; F that leaves whole lines, and not
DENSE = [(64, 131, 16400, 512, True), (64, 150, 16408, 544, False), (64, 190, 16400, 560, False),
         (64, 131, 16402, 528, False),
         (128, 257, 16400, 384, True), (128, 257, 16402, 336, False), (128, 300, 16408, 352, False),
         (128, 370, 16400, 368, False),
         (256, 600, 16400, 384, True), (256, 1030, 8201, 336, False), (256, 1100, 8200, 368, False),
         (256, 2100, 4200, 352, False), (256, 2100, 8200, 1072, False)]

# rows of a tile, rows of each expert, rows of none, F, K, packed
GROUPED = [(64, (131, 0, 66, 1), 0, 16400, 512, True), (64, (70, 0, 131, 3), 1, 16402, 400, False),
           (64, (70, 0, 131, 3), 3, 16400, 432, False),
           (128, (140, 0, 257, 1), 0, 16400, 384, True), (128, (300, 0, 257, 1), 3, 16402, 336, False),
           (128, (300, 0, 300, 140), 2, 8200, 432, False),
           (256, (600, 0, 257, 1), 2, 16400, 384, True), (256, (1030, 2, 518), 0, 8208, 1152, True),
           (256, (1030, 0, 257), 3, 8200, 352, False), (256, (600, 1, 257), 2, 16402, 336, False),
           (256, (1030, 0, 1025), 3, 8200, 1072, False)]


def kpacked(b):
    """b [.., K] in the layout that the packed products take (16 rows by 64 of K, each KB together)."""
    return b.view(-1, 16, b.shape[-1] // 64, 64).transpose(1, 2).contiguous().view(b.shape)


def kpaired(a):
    M, K = a.shape
    return a.view(M // 2, 2, K // 64, 64).transpose(1, 2).contiguous().view(M, K)


def guarded(M, F):
    full = torch.full((M * F + 512,), 7.5, dtype=torch.bfloat16, device="cuda")
    return full, full[256:-256].view(M, F)


def operands(seed, M, rows_b, K):
    g = torch.Generator().manual_seed(seed)
    a, ai, av = codes(g, (M, K), 1.0)
    b, bi, bv = codes(g, (*rows_b, K), 2.0 / K ** 0.5)
    return [t.cuda() for t in (a, ai, av, b, bi, bv)]


@pytest.mark.parametrize("tile,M,F,K,packed", DENSE)
@pytest.mark.parametrize("fast", [True, False])
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_dense(tile, M, F, K, packed, fast, act):
    f = lib()
    a, ai, av, b, bi, bv = operands(M + F + K, M, (2 * F,), K)
    bd = kpacked(b) if packed else b
    (full, out), (full2, gu) = guarded(M, F), guarded(M, 2 * F)
    call = lambda gu, out: f.fp8_gated_mm(a, bd, f.E4M3_NATIVE, f.SCALE_ROW, ai, bi, ACTS[act], gu, out,  # noqa: E731
                                          packed=packed, use_fast_accum=fast)
    call(gu, out)
    check(out, gu, av, bv, act, fast, (M, F, K))
    for t in (full, full2):
        assert (t[:256] == 7.5).all() and (t[-256:] == 7.5).all(), "write outside the output"
    again, gu2 = torch.empty_like(out), torch.empty_like(gu)
    for g in (None, gu2):  # without the projections, and once more: the same bits
        call(g, again)
        assert torch.equal(again.view(torch.int16), out.view(torch.int16))
    assert torch.equal(gu2.view(torch.int16), gu.view(torch.int16))


@pytest.mark.parametrize("tile,M,F,K,packed", [DENSE[i] for i in (0, 1, 4, 6, 8, 9, 12)])
@pytest.mark.parametrize("fast", [True, False])
def test_dense_tensorwise(tile, M, F, K, packed, fast):
    f = lib()
    a, _, _, b, _, _ = operands(M + F + K + 1, M, (2 * F,), K)
    sa, sb = torch.tensor([0.02], device="cuda"), torch.tensor([0.004], device="cuda")
    av, bv = (q.view(torch.float8_e4m3fn).double() * s.double() for q, s in ((a, sa), (b, sb)))
    out = torch.empty((M, F), dtype=torch.bfloat16, device="cuda")
    gu = torch.empty((M, 2 * F), dtype=torch.bfloat16, device="cuda")
    f.fp8_gated_mm(a, kpacked(b) if packed else b, f.E4M3_NATIVE, f.SCALE_TENSOR, sa, sb, f.ACT_SILU, gu, out,
                   packed=packed, use_fast_accum=fast)
    check(out, gu, av, bv, "silu", fast, (M, F, K))


@pytest.mark.parametrize("tile,rows,pad,F,K,packed", GROUPED)
@pytest.mark.parametrize("fast", [True, False])
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_grouped(tile, rows, pad, F, K, packed, fast, act):
    f = lib()
    E, M, end = len(rows), sum(rows) + pad, sum(rows)
    a, ai, av, b, bi, bv = operands(M + F + K, M, (E, 2 * F), K)
    off = torch.tensor([0] + list(np.cumsum(rows)), dtype=torch.int32, device="cuda")
    (full, out), (full2, gu) = guarded(M, F), guarded(M, 2 * F)
    call = lambda gu, out: f.fp8_grouped_gated_mm(  # noqa: E731
        kpaired(a) if packed else a, kpacked(b) if packed else b, f.E4M3_NATIVE, ai, bi, off, ACTS[act], gu, out,
        packed=packed, use_fast_accum=fast)
    call(gu, out)
    lo = 0
    for e, n in enumerate(rows):
        if n:
            check(out[lo:lo + n], gu[lo:lo + n], av[lo:lo + n], bv[e], act, fast, (rows, e))
        lo += n
    assert (out[end:] == 7.5).all() and (gu[end:] == 7.5).all(), "rows behind the last expert were written"
    for t in (full, full2):
        assert (t[:256] == 7.5).all() and (t[-256:] == 7.5).all(), "write outside the output"
    again = torch.empty_like(out)
    call(None, again)
    assert torch.equal(again[:end].view(torch.int16), out[:end].view(torch.int16))


def test_tests_own_layouts():
    """kpacked and kpaired are the quantizers' layouts."""
    f = lib()
    x = torch.randn((48, 256), generator=torch.Generator().manual_seed(0)).to(torch.bfloat16).cuda()
    sc = torch.empty((2, 48), device="cuda")
    q, qk = (torch.empty((48, 256), dtype=torch.uint8, device="cuda") for _ in range(2))
    f.fp8_quant_row(x, f.E4M3_NATIVE, 1e-12, q, sc[0], sc[1])
    f.fp8_quant_row_kpacked(x, f.E4M3_NATIVE, 1e-12, qk, sc[0], sc[1])
    assert torch.equal(qk, kpacked(q))
    f.fp8_quant_row_kpaired(x, f.E4M3_NATIVE, 1e-12, qk, sc[0], sc[1])
    assert torch.equal(qk, kpaired(q))


@pytest.mark.parametrize("fast", [True, False])
def test_weights_past_32_bits(fast):
    """2F K of 2^31 and more, 300 rows dense and grouped: features at both ends and where offsets pass 31 and 32 bits."""
    f = lib()
    F, K, rows = 66000, 16400, (170, 0, 130)
    E, M = len(rows), sum(rows)
    assert 2 * F * K > 1 << 31
    g = torch.Generator(device="cuda").manual_seed(1)
    # codes of all finite values: anything but 0x7f and 0xff
    b = torch.randint(0, 127, (E, 2 * F, K), dtype=torch.uint8, device="cuda", generator=g)
    for e in range(E):
        b[e] |= torch.randint(0, 2, (2 * F, K), dtype=torch.uint8, device="cuda", generator=g) << 7
    a = torch.randint(0, 127, (M, K), dtype=torch.uint8, device="cuda", generator=g)
    a |= torch.randint(0, 2, (M, K), dtype=torch.uint8, device="cuda", generator=g) << 7
    # sums of K products of codes of some 80 by 80: to values of about 1
    ai = torch.full((M,), 1 / 80 / K ** 0.5, device="cuda") * (1 + torch.arange(M, device="cuda") / M)
    bi = torch.full((E, 2 * F), 1 / 80, device="cuda") * (1 + torch.arange(2 * F, device="cuda") / F)
    av = a.view(torch.float8_e4m3fn).double() * ai.double()[:, None]
    at = ((1 << 31) // K, (1 << 30) // K)
    cols = sorted({c for m in (0, F - 17, *at) for c in range(m, m + 17) if c < F})
    cols = torch.tensor(cols + [at[0] - F + i for i in range(17) if 0 <= at[0] - F + i < F], device="cuda").unique()

    def values(e):
        both = torch.cat([cols, cols + F])
        return b[e][both].view(torch.float8_e4m3fn).double() * bi[e][both].double()[:, None]

    def some(out, gu):
        return out[:, cols], torch.cat([gu[:, cols], gu[:, cols + F]], 1)

    out = torch.full((M, F), float("nan"), dtype=torch.bfloat16, device="cuda")
    gu = torch.full((M, 2 * F), float("nan"), dtype=torch.bfloat16, device="cuda")
    off = torch.tensor([0] + list(np.cumsum(rows)), dtype=torch.int32, device="cuda")
    f.fp8_grouped_gated_mm(a, b, f.E4M3_NATIVE, ai, bi, off, f.ACT_SILU, gu, out, use_fast_accum=fast)
    o, p = some(out, gu)
    check(o[:170], p[:170], av[:170], values(0), "silu", fast, "grouped, first")
    check(o[170:], p[170:], av[170:], values(2), "silu", fast, "grouped, last")
    assert torch.isfinite(out).all() and torch.isfinite(gu).all()
    out.fill_(float("nan"))
    gu.fill_(float("nan"))
    f.fp8_gated_mm(a, b[2], f.E4M3_NATIVE, f.SCALE_ROW, ai, bi[2], f.ACT_SILU, gu, out, use_fast_accum=fast)
    o, p = some(out, gu)
    check(o, p, av, values(2), "silu", False, "dense")
    assert torch.isfinite(out).all() and torch.isfinite(gu).all()
