"""The expert router and the few-token expert layer on the GPU: choices, offsets and sorted
rows exactly, gate weights, gradients and the layer's outputs against 64 bits, at masks and
sizes where they can go wrong, and the whole chain from the residual norm on, captured and
replayed."""
import numpy as np
import pytest

import oracle
from tests.gpu_util import gpu, have_gpu, lib, kpack, to_dev

pytestmark = [gpu, pytest.mark.skipif(not have_gpu(), reason="needs an MI355X")]
EPS = 1e-12
U = 2.0 ** -24  # half a step of fp32
GATES = ["softmax", "softmax_topk", "sigmoid"]


@pytest.fixture(scope="module")
def f():
    oracle.build(force=False)
    return lib()


def _gate(f, name):
    return {"softmax": f.GATE_SOFTMAX, "softmax_topk": f.GATE_SOFTMAX_TOPK, "sigmoid": f.GATE_SIGMOID}[name]


# ---- router -------------------------------------------------------------------------------

def route_reference(l, k, gate):
    """ids, weights (64 bits), offsets, order, slot of logits l [T][E] float64."""
    T, E = l.shape
    usable = np.where(np.isnan(l), -np.inf, l) + 0.0
    rank = np.argsort(-usable, axis=1, kind="stable")[:, :k]  # equal: the lowest index first
    val = np.take_along_axis(usable, rank, 1)
    ok = val > -np.inf
    ids = np.where(ok, rank, -1)
    with np.errstate(all="ignore"):
        if gate == "sigmoid":
            w = 1.0 / (1.0 + np.exp(-val))
        else:
            top = val[:, :1]
            over = l if gate == "softmax" else val
            w = np.exp(val - top) / np.where(over > -np.inf, np.exp(over - top), 0.0).sum(1, keepdims=True)
    w = np.where(ok, w, 0.0)
    w = np.where(ok & np.isnan(l).any(1, keepdims=True), np.nan, w)
    flat = ids.reshape(-1)
    key = np.where(flat < 0, E, flat)
    sort = np.argsort(key, kind="stable")
    offsets = np.concatenate([[0], np.cumsum(np.bincount(key, minlength=E + 1)[:E])])
    slot = np.empty(T * k, np.int64)
    slot[sort] = np.arange(T * k)
    order = np.where(np.arange(T * k) < offsets[-1], sort, -1)
    return ids, w, offsets, order, np.where(flat < 0, -1, slot).reshape(T, k)


def run_route(f, l, k, gate, sort=True):
    import torch
    T, E = l.shape
    i32 = dict(dtype=torch.int32, device="cuda:0")
    full = lambda *s: torch.full(s, -77, **i32)  # noqa: E731
    ids, w = full(T, k), torch.full((T, k), -77.0, device="cuda:0")
    offsets, order, slot = (full(E + 1), full(T * k), full(T, k)) if sort else (None, None, None)
    n = f.fp8_moe_route_ws_bytes(T, E, k)
    ws = torch.full((n + 1024,), 0xA5, dtype=torch.uint8, device="cuda:0")
    f.fp8_moe_route(l, _gate(f, gate), ids, w, offsets, order, slot, ws[:n] if sort else None)
    torch.cuda.synchronize()
    assert bool((ws[n:] == 0xA5).all()), "write behind the workspace"
    return ids, w, offsets, order, slot


def check_route(f, l, k, gate):
    ids, w, offsets, order, slot = run_route(f, l, k, gate)
    lv = l.double().cpu().numpy()
    ri, rw, ro, rr, rs = route_reference(lv, k, gate)
    assert np.array_equal(ids.cpu().numpy(), ri)
    assert np.array_equal(offsets.cpu().numpy(), ro)
    assert np.array_equal(order.cpu().numpy(), rr)
    assert np.array_equal(slot.cpu().numpy(), rs)
    got = w.double().cpu().numpy()
    assert np.array_equal(np.isnan(got), np.isnan(rw))
    # l - top rounds once (relative to itself, up to 2^-24 |l - top| in the exponent), exp
    # and the quotient to a few steps, the sum has at most 22 additions; weights below the
    # normal range (2^-126) keep fewer bits
    with np.errstate(all="ignore"):
        top = np.where(lv > -np.inf, lv, np.nan)
        spread = np.nan_to_num(np.nanmax(np.abs(top), axis=1, keepdims=True, initial=0.0, where=np.isfinite(top)))
    tol = U * (64 + 4 * spread) * np.abs(rw) + 2.0 ** -125
    with np.errstate(invalid="ignore"):
        assert np.all((np.abs(got - rw) <= tol) | np.isnan(rw))
    return ids, w


def _logits(T, E, dtype, seed, scale=1.5):
    import torch
    g = torch.Generator(device="cuda:0").manual_seed(seed)
    return (torch.randn(T, E, generator=g, device="cuda:0") * scale).to(dtype)


# one block (up to 64 tokens) and several, every number of lanes a token, ragged E
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 32, 8), (3, 2, 2), (63, 16, 4), (64, 17, 3), (65, 33, 8),
                                   (257, 64, 6), (300, 100, 8), (1000, 256, 8), (129, 300, 32), (70, 1024, 16),
                                   (20011, 24, 2)])
@pytest.mark.parametrize("gate", GATES)
def test_route(f, T, E, k, gate):
    import torch
    for dtype in (torch.float32, torch.bfloat16):
        check_route(f, _logits(T, E, dtype, 31 * T + E), k, gate)


@pytest.mark.parametrize("gate", GATES)
def test_route_equal_logits_take_the_lowest_expert(f, gate):
    import torch
    l = _logits(200, 40, torch.float32, 9).round()  # a few distinct values, -0 among them
    l[7] = 0.0
    l[8] = -0.0
    l[9, ::2] = -0.0
    l[9, 1::2] = 0.0
    check_route(f, l, 8, gate)


@pytest.mark.parametrize("T", [50, 700])
@pytest.mark.parametrize("gate", GATES)
def test_route_masks(f, gate, T):
    """Masked experts, tokens with fewer experts than slots or none, the type's lowest value
    (an ordinary logit), NaN."""
    import torch
    l = _logits(T, 48, torch.float32, 10)
    inf = float("inf")
    l[3] = -inf
    l[T - 9:] = -inf          # padding behind the last token
    l[5, 2:] = -inf           # two experts left
    l[6, :47] = -inf          # the last one alone
    l[:, 11] = -inf           # an expert that nobody may take
    l[8] = torch.finfo(torch.float32).min
    l[9, :40] = torch.finfo(torch.float32).min
    l[10, 4] = float("nan")
    l[12, 1:] = float("nan")
    l[13] = float("nan")
    ids, w = check_route(f, l, 6, gate)
    assert not bool((ids == 11).any())
    assert bool((ids[T - 9:] == -1).all()) and not bool(w[T - 9:].any())


def test_route_all_tokens_masked(f):
    import torch
    l = torch.full((130, 8), float("-inf"), device="cuda:0")
    ids, w, offsets, order, slot = run_route(f, l, 2, "softmax")
    assert bool((ids == -1).all()) and bool((order == -1).all()) and bool((slot == -1).all())
    assert not bool(offsets.any()) and not bool(w.any())


def test_route_without_sorting_and_without_tokens(f):
    import torch
    l = _logits(100, 32, torch.bfloat16, 12)
    a = run_route(f, l, 4, "softmax")
    b = run_route(f, l, 4, "softmax", sort=False)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    _, _, offsets, _, _ = run_route(f, l[:0], 4, "softmax")
    assert not bool(offsets.any())


def bwd_reference(l, ids, w, dw, gate):
    T, E = l.shape
    ok = ids >= 0
    at = np.where(ok, ids, 0)
    wd = np.where(ok, w * dw, 0.0)
    S = wd.sum(1, keepdims=True)
    out, mag = np.zeros((T, E)), np.zeros((T, E))
    rows = np.arange(T)[:, None]
    if gate == "sigmoid":
        np.add.at(out, (rows, at), wd * (1.0 - w))
        np.add.at(mag, (rows, at), np.abs(wd))
    elif gate == "softmax_topk":
        np.add.at(out, (rows, at), np.where(ok, wd - w * S, 0.0))
        np.add.at(mag, (rows, at), np.abs(wd) + np.abs(w) * np.abs(wd).sum(1, keepdims=True))
    else:
        top = l.max(1, keepdims=True)
        with np.errstate(invalid="ignore"):
            p = np.where(l > -np.inf, np.exp(l - top), 0.0)
        p = p / np.maximum(p.sum(1, keepdims=True), 1e-300)
        out = -p * S
        np.add.at(out, (rows, at), wd)
        mag = p * np.abs(wd).sum(1, keepdims=True)
        np.add.at(mag, (rows, at), np.abs(wd))
    return out, mag


@pytest.mark.parametrize("T,E,k", [(1, 32, 8), (5, 1, 1), (130, 17, 3), (300, 100, 8), (77, 256, 8), (90, 257, 8),
                                   (33, 512, 8), (40, 1000, 32)])
@pytest.mark.parametrize("gate", GATES)
def test_route_backward(f, T, E, k, gate):
    import torch
    for dtype in (torch.float32, torch.bfloat16):
        l = _logits(T, E, dtype, 5 * T + E)
        if E > 8:
            l[0, :E - k + 2] = -float("inf")
            l[T - 1] = -float("inf") if T > 1 else l[T - 1]
        ids, w = run_route(f, l, k, gate, sort=False)[:2]
        dw = _logits(T, k, torch.float32, 77, 0.3)
        dl = torch.full_like(l, 7.0)
        f.fp8_moe_route_bwd(l, _gate(f, gate), ids, w, dw, dl)
        ref, mag = bwd_reference(l.double().cpu().numpy(), ids.cpu().numpy(), w.double().cpu().numpy(),
                                 dw.double().cpu().numpy(), gate)
        got = dl.double().cpu().numpy()
        # fp32: products and a sum of at most 32 terms over the lanes, and the softmax's
        # own (as above: |l - top| up to 16 here); then the type's half step
        half = U if dtype == torch.float32 else 2.0 ** -8
        assert np.all(np.abs(got - ref) <= half * np.abs(ref) + 160 * U * mag + 1e-38)
        # in place
        f.fp8_moe_route_bwd(l, _gate(f, gate), ids, w, dw, l)
        assert torch.equal(l, dl)


@pytest.mark.parametrize("gate", GATES)
def test_route_backward_against_differences(f, gate):
    """sum(dl * v) against the central difference of sum(w * dw) along v in 64 bits, the
    chosen experts held (logits a step apart, so that no step changes the choice)."""
    import torch
    T, E, k = 7, 24, 4
    g = np.random.default_rng(8)
    l = np.stack([g.permutation(E) for _ in range(T)]) * 0.25
    dw, v = g.standard_normal((T, k)).astype(np.float32), g.standard_normal((T, E))
    loss = lambda z: (route_reference(z, k, gate)[1] * dw).sum()  # noqa: E731
    want = (loss(l + 1e-5 * v) - loss(l - 1e-5 * v)) / 2e-5
    ld = to_dev(l.astype(np.float32))
    ids, w = run_route(f, ld, k, gate, sort=False)[:2]
    dl = torch.empty_like(ld)
    f.fp8_moe_route_bwd(ld, _gate(f, gate), ids, w, to_dev(dw), dl)
    got = dl.double().cpu().numpy()
    # the quotient's error, 1e-5^2 of third derivatives below 1 and 2^-52 / 1e-5 of the sum
    assert abs((got * v).sum() - want) <= 1e-6 * (np.abs(got * v).sum() + 1.0)


# ---- the few-token layer --------------------------------------------------------------------

class Layer:
    def __init__(self, E, D, F, seed, packed):
        import torch
        g = torch.Generator(device="cuda:0").manual_seed(seed)
        self.E, self.D, self.F, self.packed = E, D, F, packed

        def make(N, K):
            codes = torch.randint(0, 256, (E, N, K), generator=g, device="cuda:0", dtype=torch.int32)
            codes = torch.where((codes & 0x7f) == 0x7f, codes ^ 1, codes).to(torch.uint8)  # no NaN
            inv = torch.rand((E, N), generator=g, device="cuda:0") * 2e-4 + 1e-5
            return codes, inv

        self.w13, self.i13 = make(2 * F, D)
        self.w2, self.i2 = make(D, F)
        if packed:
            pk = lambda c: to_dev(kpack(c.cpu().numpy())).reshape(c.shape)  # noqa: E731
            self.c13, self.c2 = pk(self.w13), pk(self.w2)
        else:
            self.c13, self.c2 = self.w13, self.w2

    def dense(self, e):
        import torch
        d = lambda c, i: c[e].view(torch.float8_e4m3fn).double() * i[e].double()[:, None]  # noqa: E731
        return d(self.w13, self.i13), d(self.w2, self.i2)


def few_reference(layer, x, ids, w):
    """out in 64 bits and a bound of the kernel's error, per element."""
    import torch
    T, D, F = x.shape[0], layer.D, layer.F
    xd = x.double()
    out, err = torch.zeros(T, D, dtype=torch.float64, device=x.device), torch.zeros(T, D, dtype=torch.float64,
                                                                                    device=x.device)
    for e in range(layer.E):
        share = torch.where(ids == e, w.double(), 0.0).sum(1)
        t = (ids == e).any(1).nonzero()[:, 0]
        if len(t) == 0:
            continue
        m13, m2 = layer.dense(e)
        p, s = xd[t] @ m13.t(), xd[t].abs() @ m13.abs().t()
        g, u, sg, su = p[:, :F], p[:, F:], s[:, :F], s[:, F:]
        silu = g * torch.sigmoid(g)
        sh = share[t, None]
        a = sh * silu * u
        # fp32 sums of D products (any order: D roundings of the magnitudes' sum), silu'
        # at most 1.1, a few roundings and expf (relative to its argument) for the rest
        dg, du = (D + 4) * U * sg, (D + 4) * U * su
        da = sh.abs() * (1.1 * dg * u.abs() + silu.abs() * du + dg * du) + (32 + 4 * g.abs()) * U * a.abs()
        da = da + 2.0 ** -16 * (a.abs() + da)  # stored as a bf16 value and that of what is left
        out[t] += a @ m2.t()
        err[t] += da @ m2.abs().t() + (F + 64) * U * ((a.abs() + da) @ m2.abs().t())
    return out, err + 2.0 ** -8 * (out.abs() + err)


def run_few(f, layer, x, ids, w, guard=True):
    import torch
    T, k = ids.shape
    out = torch.full((T + 2, layer.D), 9.0, dtype=torch.bfloat16, device="cuda:0")
    n = f.fp8_moe_few_ws_bytes(T, k, layer.F)
    ws = torch.full((n + 1024,), 0xFF, dtype=torch.uint8, device="cuda:0")  # NaN patterns
    f.fp8_moe_few(x, ids, w, layer.c13, layer.i13, layer.c2, layer.i2, f.E4M3_NATIVE, out[:T], ws[:n],
                  packed=layer.packed)
    torch.cuda.synchronize()
    assert bool((out[T:] == 9.0).all()) and bool((ws[n:] == 0xFF).all()), "write out of range"
    return out[:T]


def check_few(f, layer, x, ids, w):
    import torch
    got = run_few(f, layer, x, ids, w)
    ref, err = few_reference(layer, x, ids, w)
    off = (got.double() - ref).abs()
    assert bool((off <= err + 1e-30).all()), float((off / (err + 1e-30)).max())
    assert torch.equal(got, run_few(f, layer, x, ids, w)), "another run, other bits"
    return got


def _tokens(T, E, k, D, seed):
    import torch
    g = torch.Generator(device="cuda:0").manual_seed(seed)
    x = torch.randn(T, D, generator=g, device="cuda:0").to(torch.bfloat16)
    ids = torch.rand(T, E, generator=g, device="cuda:0").argsort(1)[:, :k].to(torch.int32).contiguous()
    w = torch.rand(T, k, generator=g, device="cuda:0")
    return x, ids, w


# token tiles of 16, 32 and 64 full and ragged, D and F below, at and past a unit of 128,
# more waves than units and fewer
@pytest.mark.parametrize("packed", [False, True], ids=["rows", "packed"])
@pytest.mark.parametrize("T,E,k,D,F", [(1, 8, 2, 64, 64), (1, 32, 8, 1024, 256), (5, 8, 2, 1088, 704),
                                       (16, 4, 4, 128, 192), (17, 4, 2, 320, 128), (33, 3, 1, 256, 320),
                                       (64, 2, 2, 192, 1152), (64, 16, 8, 512, 64), (40, 200, 8, 128, 128),
                                       (2, 1, 1, 2176, 64)])
def test_few(f, T, E, k, D, F, packed):
    check_few(f, Layer(E, D, F, 100 + D, packed), *_tokens(T, E, k, D, T))


# many units of F an output tile: the down product's tiles are shared by workgroups and
# their sums joined; tiles that begin and end inside a workgroup's share, a tile of half
# the rows, every number of loads for an expert's tokens
@pytest.mark.parametrize("packed", [False, True], ids=["rows", "packed"])
@pytest.mark.parametrize("T,E,k,D,F", [(1, 8, 8, 64, 8192), (4, 8, 8, 64, 8256), (7, 40, 8, 576, 1088),
                                       (33, 40, 8, 192, 1024), (64, 6, 6, 128, 5632), (24, 3, 2, 448, 12800)])
def test_few_with_tiles_shared_by_workgroups(f, T, E, k, D, F, packed):
    check_few(f, Layer(E, D, F, 400 + D, packed), *_tokens(T, E, k, D, T))


@pytest.mark.parametrize("D,F", [(80, 8192), (1040, 5136), (16, 12816)])
def test_few_with_shared_tiles_row_major_odd_sizes(f, D, F):
    check_few(f, Layer(9, D, F, 450 + D, False), *_tokens(5, 9, 8, D, 6))


@pytest.mark.parametrize("D,F", [(16, 16), (48, 16), (16, 176), (1040, 720), (208, 144)])
def test_few_row_major_odd_sizes(f, D, F):
    check_few(f, Layer(5, D, F, 200 + D, False), *_tokens(9, 5, 3, D, 4))


@pytest.mark.parametrize("T,D,F,packed", [(1, 4096, 128, True), (1, 4112, 128, False), (20, 4112, 272, False),
                                          (20, 4160, 320, True), (50, 4160, 64, True), (50, 4096, 144, False)])
def test_few_either_side_of_narrow_tiles(f, T, D, F, packed):
    """Whole tiles of 16 rows up to 4096 rows of few units, of 32 above."""
    check_few(f, Layer(6, D, F, 460 + T, packed), *_tokens(T, 6, 2, D, T))


def test_few_tokens_without_experts_and_repeated_ids(f):
    import torch
    layer = Layer(6, 256, 192, 300, True)
    x, ids, w = _tokens(20, 6, 4, 256, 301)
    ids[0] = -1
    ids[1, 1:] = -1
    ids[2, :3] = torch.tensor([6, 1 << 30, -(1 << 31)], dtype=torch.int32)
    ids[3] = 2                       # four times the same expert: the weights add up
    ids[4, 1] = ids[4, 3]
    ids[19] = -1
    got = check_few(f, layer, x, ids, w)
    assert not bool(got[0].any()) and not bool(got[19].any())
    ids.fill_(-1)
    assert not bool(run_few(f, layer, x, ids, w).any())


@pytest.mark.parametrize("T", [3, 40])
def test_few_a_nan_stays_with_its_token(f, T):
    """NaN in one token's x, and NaN codes in an expert that another token takes alone."""
    import torch
    layer = Layer(4, 128, 128, 310, False)
    x, ids, w = _tokens(T, 3, 2, 128, 311)  # expert 3 unused
    clean = run_few(f, layer, x, ids, w)
    x[1, 5] = float("nan")
    ids[2] = 3
    layer.c13[3, 7, 9] = 0x7F
    layer.c2[3, 11] = 0xFF
    got = run_few(f, layer, x, ids, w)
    assert bool(got[1].isnan().all()) and bool(got[2, 11].isnan())
    keep = [t for t in range(T) if t not in (1, 2)]
    assert torch.equal(got[keep], clean[keep])


@pytest.mark.parametrize("T", [3, 40])
def test_few_an_infinite_activation_is_the_formulas(f, T):
    """Activations that overflow with codes of one sign behind them: an infinity, not a NaN."""
    import torch
    layer = Layer(4, 128, 128, 312, False)
    x, ids, w = _tokens(T, 3, 1, 128, 313)  # expert 3 unused
    clean = run_few(f, layer, x, ids, w)
    layer.c13[3], layer.c2[3] = 0x38, 0x38  # ones
    layer.i13[3], layer.i2[3] = 1.0, 1.0
    layer.c2[3, 5] = 0xB8
    ids[1], w[1], x[1] = 3, 0.5, 1e30  # 128e30 squared
    got = run_few(f, layer, x, ids, w)
    want = torch.full((128,), float("inf"), device="cuda:0")
    want[5] = -want[5]
    assert torch.equal(got[1].float(), want)
    keep = [t for t in range(T) if t != 1]
    assert torch.equal(got[keep], clean[keep])


def test_few_alone_is_as_in_a_batch(f):
    """A token's output does not depend on the tokens beside it (same tile, same sums)."""
    import torch
    layer = Layer(8, 384, 256, 320, True)
    x, ids, w = _tokens(16, 8, 2, 384, 321)
    whole = run_few(f, layer, x, ids, w)
    ref, err = few_reference(layer, x, ids, w)
    for t in (0, 15):
        one = run_few(f, layer, x[t:t + 1].contiguous(), ids[t:t + 1].contiguous(), w[t:t + 1].contiguous())
        assert bool(((one[0].double() - ref[t]).abs() <= err[t]).all())
        assert bool(((whole[t].double() - ref[t]).abs() <= err[t]).all())


def test_few_without_intermediate_columns_is_the_empty_sum(f):
    import torch
    x, ids, w = _tokens(4, 3, 2, 64, 330)
    u8 = dict(dtype=torch.uint8, device="cuda:0")
    e = torch.empty((3, 0), device="cuda:0")
    out = torch.ones((4, 64), dtype=torch.bfloat16, device="cuda:0")
    f.fp8_moe_few(x, ids, w, torch.empty((3, 0, 64), **u8), e, torch.empty((3, 64, 0), **u8),
                  torch.ones((3, 64), device="cuda:0"), f.E4M3_NATIVE, out, None)
    assert not bool(out.any())


# ---- the operators together --------------------------------------------------------------------

class Block:
    """The feed-forward half of a block: residual norm, router, experts (few tokens)."""

    def __init__(self, f, T, D, E, k, F, seed):
        import torch
        self.f, self.T, self.E, self.k = f, T, E, k
        self.layer = Layer(E, D, F, seed, True)
        g = torch.Generator(device="cuda:0").manual_seed(seed + 1)
        self.gamma = (1 + 0.1 * torch.randn(D, generator=g, device="cuda:0")).to(torch.bfloat16)
        self.wr = (0.05 * torch.randn(E, D, generator=g, device="cuda:0"))
        bf, dev = torch.bfloat16, "cuda:0"
        self.x, self.res = torch.zeros(T, D, dtype=bf, device=dev), torch.zeros(T, D, dtype=bf, device=dev)
        self.y, self.out = torch.empty_like(self.x), torch.empty_like(self.x)
        self.ids = torch.empty((T, k), dtype=torch.int32, device=dev)
        self.w = torch.empty((T, k), device=dev)
        self.logits = torch.empty((T, E), device=dev)
        self.sorted = [torch.empty(n, dtype=torch.int32, device=dev) for n in (E + 1, T * k, T * k)]
        self.ws = torch.empty(f.fp8_moe_few_ws_bytes(T, k, F), dtype=torch.uint8, device=dev)

    def fill(self, seed):
        import torch
        g = torch.Generator(device="cuda:0").manual_seed(seed)
        self.x.copy_(torch.randn(self.x.shape, generator=g, device="cuda:0"))
        self.res.copy_(torch.randn(self.x.shape, generator=g, device="cuda:0"))

    def run(self):
        import torch
        f, L = self.f, self.layer
        f.fp8_add_norm_quant_row(self.x, self.res, self.gamma, None, f.NORM_RMS, 1e-5, f.E4M3_NATIVE, EPS, self.res,
                                 self.y, None, None)
        torch.mm(self.y.float(), self.wr.t(), out=self.logits)
        f.fp8_moe_route(self.logits, f.GATE_SOFTMAX_TOPK, self.ids, self.w, *self.sorted)
        f.fp8_moe_few(self.y, self.ids, self.w, L.c13, L.i13, L.c2, L.i2, f.E4M3_NATIVE, self.out, self.ws, packed=True)

    def outputs(self):
        return [t.clone() for t in (self.res, self.y, self.logits, self.ids, self.w, *self.sorted, self.out)]


def test_block_against_64_bits(f):
    import torch
    b = Block(f, 24, 512, 16, 4, 256, 500)
    b.fill(1)
    x, res = b.x.clone(), b.res.clone()
    b.run()
    h = (x.float() + res.float()).to(torch.bfloat16)
    assert torch.equal(b.res, h)
    y = h.double() * torch.rsqrt(h.double().square().mean(1, keepdim=True) + 1e-5) * b.gamma.double()
    # two fp32 products and the statistics' rounding before the bf16 rounding
    assert bool(((b.y.double() - y).abs() <= y.abs() * (2.0 ** -8 + 8 * U)).all())
    ids, w, off, order, slot = route_reference(b.logits.double().cpu().numpy(), 4, "softmax_topk")
    assert np.array_equal(b.ids.cpu().numpy(), ids) and np.array_equal(b.sorted[0].cpu().numpy(), off)
    ref, err = few_reference(b.layer, b.y, b.ids, b.w)
    assert bool(((b.out.double() - ref).abs() <= err).all())


def test_block_captured_and_replayed(f):
    """The chain captured into a graph, replayed over new inputs with eager work between:
    the eager bits every time. Two graphs with a workspace each run on two streams."""
    import torch
    blocks = [Block(f, 24, 512, 16, 4, 256, 510 + i) for i in range(2)]
    graphs = []
    for b in blocks:
        b.fill(0)
        b.run()  # probe and libraries are warm before the capture
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            b.run()
        graphs.append(g)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for seed in range(2, 6):
        want = []
        for b in blocks:
            b.fill(seed)
            b.run()
            want.append(b.outputs())
            b.fill(seed)
        torch.cuda.synchronize()
        for b, g, s in zip(blocks, graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for b, w in zip(blocks, want):
            assert all(torch.equal(p, q) for p, q in zip(b.outputs(), w)), seed


def test_route_feeds_the_grouped_gemm(f):
    """The sorted rows and offsets as the grouped GEMM takes them: the same experts' products
    as the few-token layer's, up to the FP8 rounding of the activations that only the
    grouped path quantizes (each e4m3 rounding half a step, 2^-4 relative, of a random
    sign: far below 2^-4 in the norm of a row)."""
    import torch
    T, D, E, k, F = 48, 512, 8, 2, 256
    layer = Layer(E, D, F, 520, False)
    x, _, _ = _tokens(T, E, k, D, 521)
    l = _logits(T, E, torch.float32, 522)
    ids, w, offsets, order, slot = run_route(f, l, k, "softmax_topk")
    assert f.fp8_validate_offsets(offsets.cpu().numpy(), T * k) == f.OK
    rows = x[(order // k).long()].contiguous()

    def gemm(a, codes, inv, N):
        M, K = a.shape
        q = torch.empty((M, K), dtype=torch.uint8, device="cuda:0")
        s, i = torch.empty(M, device="cuda:0"), torch.empty(M, device="cuda:0")
        out = torch.empty((M, N), dtype=torch.bfloat16, device="cuda:0")
        f.fp8_quant_row(a, f.E4M3_NATIVE, EPS, q, s, i)
        f.fp8_grouped_mm(q, f.E4M3_NATIVE, codes, f.E4M3_NATIVE, f.SCALE_ROW, i, inv, offsets, f.OUT_BF16, out,
                         use_fast_accum=False)
        return out

    p = gemm(rows, layer.c13, layer.i13, 2 * F).float()
    a = (torch.nn.functional.silu(p[:, :F]) * p[:, F:]).to(torch.bfloat16)
    o = gemm(a, layer.c2, layer.i2, D).float()
    many = (o[slot.long()] * w[:, :, None]).sum(1)
    few = run_few(f, layer, x, ids, w).float()
    assert float((many - few).norm() / few.norm()) < 2.0 ** -4
