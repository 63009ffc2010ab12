"""The residual norm, the router and the few-token expert layer at the ends of their ranges:
tensors past 2^31 elements, the most experts and choices, every token on one expert, and
calls captured into graphs that replay at the same time."""
import pytest

from tests.gpu_util import gpu, have_gpu, lib
from tests.test_gpu_moe import Layer, _tokens, check_few, check_route, few_reference, run_few, run_route

pytestmark = [gpu, pytest.mark.skipif(not have_gpu(), reason="needs an MI355X")]
EPS = 1e-12


@pytest.fixture(scope="module")
def f():
    return lib()


def test_norm_past_32_bits(f):
    """Each row's results do not depend on the rows before it: the last ones are those of a call alone."""
    import torch
    rows, cols, last = 262150, 8200, 9
    dev = dict(dtype=torch.bfloat16, device="cuda:0")
    x, res = torch.empty(rows, cols, **dev).normal_(), torch.empty(rows, cols, **dev).normal_()
    gamma = torch.empty(cols, **dev).normal_()

    def forward(x, res):
        n = x.shape[0]
        h, y = torch.empty_like(x), torch.empty_like(x)
        q = torch.empty(x.shape, dtype=torch.uint8, device="cuda:0")
        s = [torch.empty(n, device="cuda:0") for _ in range(2)]
        f.fp8_add_norm_quant_row(x, res, gamma, None, f.NORM_RMS, 1e-5, f.E4M3_NATIVE, EPS, h, y, q, s[0], rstd=s[1])
        return h, y, q, *s

    def backward(dy, h, rstd):
        dx = torch.empty_like(dy)
        f.fp8_add_norm_bwd(dy, None, h, gamma, None, rstd, f.NORM_RMS, dx, None, None, None)
        return dx

    whole, alone = forward(x, res), forward(x[-last:].clone(), res[-last:].clone())
    for a, b in zip(whole, alone):
        assert torch.equal(a[-last:], b)
    dx = backward(x, whole[0], whole[-1])
    assert torch.equal(dx[-last:], backward(x[-last:].clone(), alone[0], alone[-1]))


def test_route_past_32_bits(f):
    import torch
    T, E = (1 << 21) + 5, 1024
    l = torch.empty(T, E, dtype=torch.bfloat16, device="cuda:0").normal_()
    i32 = dict(dtype=torch.int32, device="cuda:0")
    ids, w = torch.empty(T, 1, **i32), torch.empty(T, 1, device="cuda:0")
    offsets, order, slot = torch.empty(E + 1, **i32), torch.empty(T, **i32), torch.empty(T, 1, **i32)
    ws = torch.empty(f.fp8_moe_route_ws_bytes(T, E, 1), dtype=torch.uint8, device="cuda:0")
    f.fp8_moe_route(l, f.GATE_SIGMOID, ids, w, offsets, order, slot, ws)
    top = torch.cat([c.float().amax(1) for c in l.split(1 << 18)])
    at = torch.cat([torch.gather(a.float(), 1, b.long())[:, 0]
                    for a, b in zip(l.split(1 << 18), ids.split(1 << 18))])
    assert torch.equal(at, top)
    flat = ids[:, 0].long()
    counts = torch.bincount(flat, minlength=E)
    assert torch.equal(offsets.long()[1:], counts.cumsum(0)) and int(offsets[0]) == 0
    want = torch.sort(flat, stable=True)[1]
    assert torch.equal(order.long(), want)
    assert torch.equal(slot[:, 0].long()[want], torch.arange(T, device="cuda:0"))
    dl = torch.full_like(l, 7.0)
    f.fp8_moe_route_bwd(l, f.GATE_SIGMOID, ids, w, torch.ones_like(w), dl)
    n = 1 << 18
    for a, b, c in zip(dl.split(n), ids.split(n), w.split(n)):
        v = torch.gather(a, 1, b.long()).float()
        s = (c.double() * (1 - c.double())).float()
        assert bool(((v - s).abs() <= 2.0 ** -8 * s + 1e-6).all())
        assert int((a != 0).sum()) <= len(a)


@pytest.mark.parametrize("packed", [False, True], ids=["rows", "packed"])
def test_few_past_32_bits(f, packed):
    import torch
    E, D, F = 68, 8192, 4096
    layer = Layer(2, D, F, 700, packed)
    big = Layer.__new__(Layer)
    big.E, big.D, big.F, big.packed = E, D, F, packed
    for n in ("c13", "c2"):
        t = getattr(layer, n)
        b = torch.full((E, *t.shape[1:]), 0x7F, dtype=torch.uint8, device="cuda:0")  # NaN wherever it is wrong
        b[0], b[E - 1] = t[0], t[1]
        setattr(big, n, b)
    for n in ("i13", "i2"):
        t = getattr(layer, n)
        b = torch.full((E, t.shape[1]), float("nan"), device="cuda:0")
        b[0], b[E - 1] = t[0], t[1]
        setattr(big, n, b)
    x, ids, w = _tokens(5, 2, 2, D, 701)
    got = run_few(f, big, x, torch.where(ids == 1, E - 1, ids).to(torch.int32), w)
    assert torch.equal(got, run_few(f, layer, x, ids, w))
    ref, err = few_reference(layer, x, ids, w)
    assert bool(((got.double() - ref).abs() <= err).all())


def test_few_most_experts_and_choices(f):
    check_few(f, Layer(1024, 64, 64, 710, True), *_tokens(64, 1024, 32, 64, 711))


@pytest.mark.parametrize("T", [64, 33, 17])
def test_few_every_token_on_one_expert(f, T):
    """Ids of one expert alone, named in every slot, with others that do not exist between."""
    import torch
    layer = Layer(3, 320, 192, 720, True)
    x, ids, w = _tokens(T, 3, 3, 320, 721)
    k = 32  # more choices than experts
    g = torch.Generator(device="cuda:0").manual_seed(722)
    ids = torch.full((T, k), 2, dtype=torch.int32, device="cuda:0")
    ids[:, ::3] = 3
    ids[:, 1::3] = -5
    w = torch.rand((T, k), generator=g, device="cuda:0")
    check_few(f, layer, x, ids, w)


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (700, 1, 1), (3, 1024, 32), (130, 33, 32), (70, 257, 8), (333, 512, 32),
                                   (150, 513, 5)])
def test_route_ends_of_the_range(f, T, E, k):
    import torch
    g = torch.Generator(device="cuda:0").manual_seed(T)
    l = torch.randn(T, E, generator=g, device="cuda:0")
    check_route(f, l.to(torch.bfloat16), k, "softmax_topk")  # many equal logits
    for gate in ("softmax", "softmax_topk", "sigmoid"):
        check_route(f, l, k, gate)


@pytest.mark.parametrize("T,pad", [(48, 7), (300, 111)])
def test_a_padded_batch_in_the_grouped_gemms(f, T, pad):
    """Tokens without an expert leave rows behind the last pair: the grouped GEMMs over all T k
    rows neither use what is there (NaN) nor write it."""
    import torch
    E, k, K, N = 8, 2, 256, 192
    g = torch.Generator(device="cuda:0").manual_seed(740 + T)
    l = torch.randn(T, E, generator=g, device="cuda:0")
    l[T - pad:] = -float("inf")
    ids, w, offsets, order, slot = run_route(f, l, k, "softmax")
    M, used = T * k, (T - pad) * k
    assert int(offsets[E]) == used and bool((order[used:] == -1).all()) and bool((slot[T - pad:] == -1).all())
    assert f.fp8_validate_offsets(offsets.cpu().numpy(), M) != f.OK  # the strict check of a full batch
    layer = Layer(E, N, K, 741, True)  # w2 codes [E][N][K]
    codes = torch.randint(0, 0x7f, (M, K), generator=g, device="cuda:0", dtype=torch.int32).to(torch.uint8)
    codes[used:] = 0x7F
    inv = torch.rand(M, generator=g, device="cuda:0") * 1e-2
    inv[used:] = float("nan")
    paired = codes.reshape(M // 2, 2, K // 64, 64).transpose(1, 2).contiguous().reshape(M, K)

    def gemm(call, a, b, rows, **shape):
        out = torch.full((rows, N), 9.0, dtype=torch.bfloat16, device="cuda:0")
        call(a[:rows], f.E4M3_NATIVE, b, f.E4M3_NATIVE, f.SCALE_ROW, inv[:rows], layer.i2, offsets, f.OUT_BF16, out,
             use_fast_accum=False, **shape)
        return out

    for call, a, b, shape in ((f.fp8_grouped_mm, codes, layer.w2, {}),
                              (f.fp8_grouped_mm_kpacked, paired, layer.c2, dict(N=N))):
        out = gemm(call, a, b, M, **shape)
        assert bool((out[used:] == 9.0).all())
        assert torch.equal(out[:used], gemm(call, a, b, used, **shape))
    gy, x = (torch.randn(M, n, generator=g, device="cuda:0").to(torch.bfloat16) for n in (N, K))
    gy[used:] = x[used:] = float("nan")
    gw = [torch.empty(E, N, K, dtype=torch.bfloat16, device="cuda:0") for _ in range(2)]
    f.fp8_grouped_wgrad_bf16(gy, x, offsets, gw[0])
    f.fp8_grouped_wgrad_bf16(gy[:used], x[:used], offsets, gw[1])
    assert torch.equal(*gw) and not bool(gw[0].isnan().any())


def test_split_tiles_and_placed_rows_captured(f):
    """The calls of two launches that hand counts or partial sums over, each in a graph of its
    own with a workspace of its own, replayed on two streams at once, and in turn."""
    import torch

    class Set:
        def __init__(self, seed):
            self.layer = Layer(8, 64, 8192, seed, True)
            self.x, self.ids, self.w = _tokens(4, 8, 8, 64, seed)
            self.out = torch.empty(4, 64, dtype=torch.bfloat16, device="cuda:0")
            self.ws = torch.empty(f.fp8_moe_few_ws_bytes(4, 8, 8192), dtype=torch.uint8, device="cuda:0")
            i32 = dict(dtype=torch.int32, device="cuda:0")
            self.l = torch.empty(3000, 40, device="cuda:0")
            self.r = [torch.empty(3000, 6, **i32), torch.empty(3000, 6, device="cuda:0"), torch.empty(41, **i32),
                      torch.empty(18000, **i32), torch.empty(3000, 6, **i32)]
            self.rws = torch.empty(f.fp8_moe_route_ws_bytes(3000, 40, 6), dtype=torch.uint8, device="cuda:0")

        def fill(self, seed):
            g = torch.Generator(device="cuda:0").manual_seed(seed)
            self.x.copy_(torch.randn(self.x.shape, generator=g, device="cuda:0"))
            self.l.copy_(torch.randn(self.l.shape, generator=g, device="cuda:0"))

        def run(self):
            L = self.layer
            f.fp8_moe_few(self.x, self.ids, self.w, L.c13, L.i13, L.c2, L.i2, f.E4M3_NATIVE, self.out, self.ws,
                          packed=True)
            f.fp8_moe_route(self.l, f.GATE_SOFTMAX, *self.r, self.rws)

        def results(self):
            return [t.clone() for t in (self.out, *self.r)]

    sets = [Set(730 + i) for i in range(2)]
    graphs = []
    for s in sets:
        s.fill(0)
        s.run()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            s.run()
        graphs.append(g)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for turn in range(4):
        want = []
        for i, s in enumerate(sets):
            s.fill(10 * turn + i)
            s.run()
            want.append(s.results())
            for t in (s.out, *s.r):
                t.zero_()
        torch.cuda.synchronize()
        for st, g in zip(streams, graphs):
            with torch.cuda.stream(st):
                g.replay()
        torch.cuda.synchronize()
        for s, w in zip(sets, want):
            assert all(torch.equal(a, b) for a, b in zip(s.results(), w))
