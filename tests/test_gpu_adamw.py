"""The AdamW step and the gradients' norm against their definitions (GPU): 32-bit states against 64 bits,
8-bit states bit for bit against the definition's fp32 operations in numpy."""
import math

import numpy as np
import pytest
import torch

from tests.gpu_util import lib

pytestmark = pytest.mark.gpu

LR, B1, B2, EPS, WD = 1e-3, 0.9, 0.95, 1e-8, 0.1
F32 = np.float32


def mix(x):
    """Wellons' lowbias32 on uint64 arrays or Python ints of 32-bit values."""
    m = 0xFFFFFFFF
    x = x & m
    x = ((x ^ (x >> 16)) * 0x7FEB352D) & m
    x = ((x ^ (x >> 15)) * 0x846CA68B) & m
    return x ^ (x >> 16)


def bits_of(n, seed, index, t):
    key = mix((seed >> 32) ^ mix((seed & 0xFFFFFFFF) ^ mix(index)))
    i = np.arange(n, dtype=np.uint64)
    return mix((i + np.uint64(mix(key + t))).astype(np.uint64)).astype(np.uint32)


def e4m3(y):
    """fp32 values of magnitude at most 448 to e4m3 codes, to nearest even."""
    return torch.from_numpy(np.ascontiguousarray(y)).to(torch.float8_e4m3fn).view(torch.uint8).numpy()


def mx(x, rnd, lift):
    n = x.size
    pad = np.zeros(-(-n // 32) * 32, F32)
    pad[:n] = x
    top = np.abs(pad).reshape(-1, 32).max(1).view(np.uint32).astype(np.int64)
    e = np.maximum((top >> 23) - 8 + ((top & 0x7FFFFF) > 0x600000), 12)
    inv = ((254 - e) << 23).astype(np.uint32).view(F32)
    y = (pad.reshape(-1, 32) * inv[:, None]).reshape(-1)[:n]
    if rnd is not None:
        a = np.abs(y)
        r20 = rnd * np.uint32(16) + np.uint32(8)
        t = ((a.view(np.uint32) + r20) & np.uint32(0xFFF00000)).view(F32)
        # below 2^-6 codes are 2^-9 apart: in 64 bits, which hold the 20 bits below them
        small = np.floor(a.astype(np.float64) * 512 + r20 * 2.0 ** -20) / 512
        y = np.copysign(np.where(a < F32(2.0 ** -6), small, t).astype(F32), y)
    if lift:
        y = np.where((x > 0) & (y < F32(2.0 ** -9)), F32(2.0 ** -9), y)
    return e4m3(y), e.astype(np.uint8)


def unmx(q, e):
    v = torch.from_numpy(q).view(torch.float8_e4m3fn).float().numpy()
    return v * np.repeat((e.astype(np.uint32) << np.uint32(23)).view(F32), 32)[:q.size]


def reference(p, g, m, v, ms, vs, t, seed, index, mul, mx8, bf16, master):
    """One step in numpy, fp32 operation by operation (the quotient in 64 bits)."""
    g = g * F32(mul) if mul is not None else g
    if mx8:
        m, r = unmx(m, ms), unmx(v, vs)
        v = r * r
    m = m * F32(B1) + g * F32(1.0 - B1)
    v = v * F32(B2) + (g * g) * F32(1.0 - B2)
    r = np.sqrt(v)
    c2, step = F32(1.0 / math.sqrt(1.0 - B2 ** t)), F32(LR / (1.0 - B1 ** t))
    d = r * c2 + F32(EPS)
    up = m.astype(np.float64) / d * step
    kept = p * F32(1.0 - LR * WD)
    new = kept.astype(np.float64) - up
    # the reciprocal to 1 ulp and three roundings of the update, one of the sum and, with bf16 kept, half a step
    tol = 4 * 2.0 ** -23 * np.abs(up) + 2.0 ** -24 * (np.abs(kept) + np.abs(new)) + 1e-38
    rnd = bits_of(p.size, seed, index, t) if seed else None
    if mx8:
        qm, ems = mx(m, None if rnd is None else rnd & np.uint32(0xFFFF), False)
        qv, evs = mx(r, None if rnd is None else rnd >> np.uint32(16), True)
        return new, tol, qm, qv, ems, evs, rnd
    return new, tol, m, v, None, None, rnd


SIZES = [1, 7, 8, 31, 32, 33, 100, 2047, 2048, 2049, 4096, 10007, 70001]


def make(sizes, p16, g16, master, mx8, seed=0, off=0):
    """Lists of device tensors; off: elements by which each begins behind a 16-byte line."""
    g = torch.Generator().manual_seed(len(sizes) + seed)
    def dev(x, dt):  # noqa: E306
        big = torch.empty(x.numel() + off, dtype=dt, device="cuda")
        big[off:] = x.to(dt).cuda()
        return big[off:]
    full = [torch.randn(n, generator=g) * 0.02 for n in sizes]
    s = dict(params=[dev(x, torch.bfloat16 if p16 else torch.float32) for x in full],
             grads=[dev(torch.randn(n, generator=g) * 1e-2, torch.bfloat16 if g16 else torch.float32) for n in sizes],
             masters=[dev(x, torch.float32) for x in full] if master else None, ms=None, vs=None)
    m = [torch.randn(n, generator=g) * 1e-3 * 10.0 ** torch.randint(-5, 1, (n,), generator=g) for n in sizes]
    r = [torch.randn(n, generator=g).abs() * 1e-2 * 10.0 ** torch.randint(-6, 1, (n,), generator=g) for n in sizes]
    if mx8:
        for k, xs, lift in (("m", m, False), ("v", r, True)):
            got = [mx(x.numpy(), None, lift) for x in xs]
            s[k] = [dev(torch.from_numpy(q), torch.uint8) for q, _ in got]
            s[k + "s"] = [torch.from_numpy(e).cuda() for _, e in got]
    else:
        s["m"], s["v"] = [dev(x, torch.float32) for x in m], [dev(x * x, torch.float32) for x in r]
    return s


def host(s):
    c = lambda ts: None if ts is None else [t.cpu().float().numpy() if t.dtype == torch.bfloat16 else t.cpu().numpy()  # noqa: E731
                                            for t in ts]
    return {k: c(v) for k, v in s.items()}


def step(f, s, t, seed=0, mul=None, **kw):
    f.fp8_adamw(s["params"], s["grads"], s["m"], s["v"], LR, B1, B2, EPS, WD, t, exp_avg_scales=s["ms"],
                exp_avg_sq_scales=s["vs"], masters=s["masters"], seed=seed, grad_mul=mul, **kw)


def check(f, before, s, t, seed, mul, p16, master, mx8):
    after = host(s)
    for i in range(len(s["params"])):
        p0 = before["masters"][i] if master else before["params"][i]
        new, tol, m, v, ms, vs, rnd = reference(
            p0, before["grads"][i], before["m"][i], before["v"][i], before["ms"] and before["ms"][i],
            before["vs"] and before["vs"][i], t, seed, i, mul, mx8, p16, master)
        if mx8:
            for name, want, got in (("m", m, after["m"][i]), ("v", v, after["v"][i]), ("m_scale", ms, after["ms"][i]),
                                    ("v_scale", vs, after["vs"][i])):
                assert np.array_equal(want, got), (name, i, int((want != got).sum()))
        else:  # the same operations: the same bits
            assert np.array_equal(m, after["m"][i]) and np.array_equal(v, after["v"][i]), i
        if master:
            assert (np.abs(after["masters"][i] - new) <= tol).all(), i
            want = torch.from_numpy(after["masters"][i]).to(torch.bfloat16).float().numpy()
            assert np.array_equal(want, after["params"][i])
        elif not p16:
            assert (np.abs(after["params"][i] - new) <= tol).all(), i
        elif rnd is None:
            assert (np.abs(after["params"][i] - new) <= tol + 2.0 ** -8 * np.abs(new)).all(), i
        else:  # one of the two neighbours: less than a whole step off, and the one the bits choose where
            # the value is not within its own error of the choice
            assert (np.abs(after["params"][i] - new) <= tol + 2.0 ** -7 * np.abs(new)).all(), i
            b = ((rnd ^ (rnd >> np.uint32(16))) & np.uint32(0xFFFF))
            pick = lambda x: ((x.astype(F32).view(np.uint32) + b) & np.uint32(0xFFFF0000)).view(F32)  # noqa: E731
            lo, hi = pick(new - tol), pick(new + tol)
            got = after["params"][i]
            # truncation after adding the same bits is monotone, so the value's own error gives an interval (near
            # zero, where the update cancels the parameter, of several bf16 steps)
            assert ((lo <= got) & (got <= hi)).all(), i
            assert got.size < 100 or (lo == hi).mean() > 0.9


KINDS = [(True, True, False), (True, True, True), (True, False, True), (True, False, False), (False, False, False),
         (False, True, False)]


@pytest.mark.parametrize("p16,g16,master", KINDS)
@pytest.mark.parametrize("mx8", [False, True])
@pytest.mark.parametrize("seed", [0, (5 << 32) + 77])
def test_adamw_step(p16, g16, master, mx8, seed):
    f = lib()
    s = make(SIZES, p16, g16, master, mx8)
    mul = torch.tensor([0.37], device="cuda")
    for t, m in ((1, None), (2, mul), (1000, mul)):
        before = host(s)
        step(f, s, t, seed, m)
        check(f, before, s, t, seed, None if m is None else 0.37, p16, master, mx8)


@pytest.mark.parametrize("mx8", [False, True])
@pytest.mark.parametrize("off", [1, 4])
def test_adamw_unaligned(mx8, off):
    """Tensors that begin anywhere in a larger buffer."""
    f = lib()
    s = make([1, 33, 2049, 5000], True, False, True, mx8, off=off)
    before = host(s)
    step(f, s, 3, 9)
    check(f, before, s, 3, 9, None, True, True, mx8)


def test_adamw_many_tensors():
    """More tensors than one launch takes, empty ones among them: each has the random bits of its place."""
    f = lib()
    s = make([(37 * i) % 300 for i in range(120)], True, True, False, True)
    before = host(s)
    step(f, s, 2, 123)
    check(f, before, s, 2, 123, None, True, False, True)


@pytest.mark.parametrize("mx8", [False, True])
def test_adamw_step_and_rate_on_the_device(mx8):
    f = lib()
    a, b = (make([100, 5000], True, True, True, mx8) for _ in range(2))
    t, lr = torch.tensor([7], dtype=torch.int32, device="cuda"), torch.tensor([LR], device="cuda")
    step(f, a, 7, 11)
    f.fp8_adamw(b["params"], b["grads"], b["m"], b["v"], float("nan"), B1, B2, EPS, WD, 0, exp_avg_scales=b["ms"],
                exp_avg_sq_scales=b["vs"], masters=b["masters"], seed=11, step_dev=t, lr_dev=lr)
    for k in ("m", "v") + (("ms", "vs") if mx8 else ()):
        assert all(torch.equal(x, y) for x, y in zip(a[k], b[k])), k
    for x, y in zip(a["masters"], b["masters"]):  # lr was rounded to fp32: 2^-24 of the update and the decay
        assert ((x - y).abs() <= 2.0 ** -22 * x.abs() + 2.0 ** -22 * 0.1).all()


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("mx8", [False, True])
def test_adamw_skips_a_step_that_is_not_finite(bad, mx8):
    f = lib()
    s = make([33, 4097], True, True, True, mx8)
    before = host(s)
    step(f, s, 1, 5, torch.tensor([bad], device="cuda"))
    after = host(s)
    for k, v in before.items():
        assert v is None or all(np.array_equal(x, y) for x, y in zip(v, after[k])), k


def test_adamw_first_step_and_zeros():
    """From zeroed states; elements whose gradients are zero keep codes of zero and do not move but by decay."""
    f = lib()
    n = 96
    p = torch.full((n,), 0.5, device="cuda")
    g = torch.zeros(n, device="cuda")
    g[40] = 1e-3
    m, v = (torch.zeros(n, dtype=torch.uint8, device="cuda") for _ in range(2))
    ms, vs = (torch.zeros(3, dtype=torch.uint8, device="cuda") for _ in range(2))
    f.fp8_adamw([p], [g], [m], [v], LR, B1, B2, EPS, WD, 1, exp_avg_scales=[ms], exp_avg_sq_scales=[vs])
    still = torch.ones(n, dtype=torch.bool)
    still[40] = False
    assert (m[still] == 0).all() and (v[still] == 0).all()
    assert (p[still.cuda()] == np.float32(0.5) * np.float32(1 - LR * WD)).all()
    assert abs(float(p[40]) - (0.5 * (1 - LR * WD) - LR)) < 1e-6
    assert m[40] != 0 and v[40] != 0


def test_adamw_small_second_moments_keep_a_code():
    """A root far below its group's largest keeps the smallest code, not zero: its next step stays bounded."""
    f = lib()
    for seed in (0, 3):
        g = torch.full((32,), 1e-9, device="cuda")
        g[0] = 1.0
        p = torch.zeros(32, device="cuda")
        m, v = (torch.zeros(32, dtype=torch.uint8, device="cuda") for _ in range(2))
        ms, vs = (torch.zeros(1, dtype=torch.uint8, device="cuda") for _ in range(2))
        args = dict(exp_avg_scales=[ms], exp_avg_sq_scales=[vs], seed=seed)
        f.fp8_adamw([p], [g], [m], [v], LR, B1, B2, 0.0, 0.0, 1, **args)
        assert (v[1:] == 1).all()
        g.zero_()
        f.fp8_adamw([p], [g], [m], [v], LR, B1, B2, 0.0, 0.0, 2, **args)
        assert torch.isfinite(p).all() and (p.abs() <= 3 * LR).all()


def test_adamw_group_that_is_not_finite():
    """A NaN or an infinity takes its group of 32 with it, and no other."""
    f = lib()
    s = make([128], False, False, False, True)
    s["grads"][0][40], s["grads"][0][100] = float("nan"), float("inf")
    ref = make([128], False, False, False, True)
    step(f, s, 1)
    step(f, ref, 1)
    for k in ("m", "v"):
        assert (s[k][0][32:64] == 0x7F).all() and s[k + "s"][0][1] == 255
        assert torch.equal(s[k][0][:32], ref[k][0][:32]) and torch.equal(s[k][0][64:96], ref[k][0][64:96])
        assert (s[k][0][96:] == 0x7F).all() and s[k + "s"][0][3] == 255
    step(f, s, 2)
    assert torch.isnan(s["params"][0][32:64]).all() and torch.isfinite(s["params"][0][:32]).all()


def test_stochastic_rounding_is_right_in_the_mean():
    """Over many steps' random bits a code between two neighbours is each of them with its share: the mean of n
    draws is within six standard errors (at most half a step over sqrt(n)) of the value."""
    f = lib()
    n = 1 << 16
    # a moment of 1.3 and one below the smallest normal code, in groups whose largest is 448 (scale 1)
    for value, spacing in ((1.3, 2.0 ** -3), (0.0101, 2.0 ** -9), (-1.3, 2.0 ** -3)):
        g = torch.full((n,), value, device="cuda") * 10
        g[::32] = 4480.0
        p = torch.zeros(n, device="cuda")
        m, v = (torch.zeros(n, dtype=torch.uint8, device="cuda") for _ in range(2))
        ms, vs = (torch.zeros(n // 32, dtype=torch.uint8, device="cuda") for _ in range(2))
        f.fp8_adamw([p], [g], [m], [v], LR, B1, B2, EPS, 0.0, 1, exp_avg_scales=[ms], exp_avg_sq_scales=[vs], seed=42)
        got = m.view(torch.float8_e4m3fn).double() * torch.exp2(ms.double() - 127).repeat_interleave(32)
        got = got.view(-1, 32)[:, 1:]
        assert got.unique().numel() == 2
        assert abs(float(got.mean()) - value) <= 6 * 0.5 * spacing / math.sqrt(got.numel()) + 1e-6 * abs(value)


def test_adamw_past_32_bits():
    """A tensor of more than 2^31 elements: its last ones as those of a short tensor of the same values."""
    f = lib()
    n, k = (1 << 31) + 4096 + 77, 4096 + 77
    short = make([k], True, True, False, True, seed=1)
    long = {}
    for key, big in (("params", n), ("grads", n), ("m", n), ("v", n), ("ms", -(-n // 32)), ("vs", -(-n // 32))):
        t = short[key][0]
        x = torch.zeros(big, dtype=t.dtype, device="cuda")
        x[x.numel() - t.numel():] = t
        long[key] = [x]
    long["masters"] = None
    step(f, short, 3)
    step(f, long, 3)
    for key in ("params", "m", "v", "ms", "vs"):
        t = short[key][0]
        assert torch.equal(long[key][0][-t.numel():].view(torch.uint8), t.view(torch.uint8)), key
    norm, mul = torch.empty(1, device="cuda"), torch.empty(1, device="cuda")
    ws = torch.empty(f.fp8_grad_norm_ws_bytes(long["grads"]), dtype=torch.uint8, device="cuda")
    f.fp8_grad_norm(long["grads"], norm, mul, ws)
    want = float(short["grads"][0].double().norm())
    assert abs(float(norm) - want) <= 2.0 ** -23 * want


def test_adamw_refuses_a_parameter_twice():
    f = lib()
    s = make([40], True, True, False, False)
    two = {k: v and v * 2 for k, v in s.items()}
    with pytest.raises(ValueError, match="twice"):
        step(f, two, 1)


# ---- norm ------------------------------------------------------------------------------------------

@pytest.mark.parametrize("sizes", [[1], [0, 5], SIZES, [32767, 32768, 32769, 200001], [11] * 300])
@pytest.mark.parametrize("off", [0, 1])
def test_grad_norm(sizes, off):
    f = lib()
    g = torch.Generator().manual_seed(len(sizes))
    grads, total = [], 0.0
    for i, n in enumerate(sizes):
        x = (torch.randn(n + off, generator=g) * 10.0 ** (i % 5 - 2)).to(torch.bfloat16 if i % 2 else torch.float32)
        grads.append(x.cuda()[off:])
        total += float(x[off:].double().square().sum())
    norm, mul, t = torch.empty(1, device="cuda"), torch.empty(1, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = torch.empty(f.fp8_grad_norm_ws_bytes(grads) + 8, dtype=torch.uint8, device="cuda")
    for scale, most in ((1.0, math.inf), (0.125, 1e-3), (2.0, 1e9)):
        f.fp8_grad_norm(grads, norm, mul, ws, grad_scale=scale, max_norm=most, step=t)
        want = scale * math.sqrt(total)
        assert abs(float(norm) - want) <= 2.0 ** -23 * want
        clip = scale * min(1.0, most / (want + 1e-6))
        assert abs(float(mul) - clip) <= 2.0 ** -23 * clip
    assert int(t) == 3


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_grad_norm_not_finite(bad):
    f = lib()
    x = torch.ones(1000, dtype=torch.bfloat16, device="cuda")
    x[777] = bad
    norm, mul, t = torch.empty(1, device="cuda"), torch.empty(1, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = torch.empty(f.fp8_grad_norm_ws_bytes([x]), dtype=torch.uint8, device="cuda")
    f.fp8_grad_norm([x], norm, mul, ws, step=t)
    assert not math.isfinite(float(norm)) and math.isnan(float(mul)) and int(t) == 0


def test_grad_norm_of_nothing():
    f = lib()
    norm, mul = torch.empty(1, device="cuda"), torch.empty(1, device="cuda")
    f.fp8_grad_norm([], norm, mul, None, max_norm=1.0)
    assert float(norm) == 0.0 and float(mul) == 1.0


def test_clipped_step_as_used():
    """The norm's factor goes to the step on the device."""
    f = lib()
    s, ref = (make([5000, 33], True, True, True, False) for _ in range(2))
    norm, mul = torch.empty(1, device="cuda"), torch.empty(1, device="cuda")
    ws = torch.empty(f.fp8_grad_norm_ws_bytes(s["grads"]), dtype=torch.uint8, device="cuda")
    f.fp8_grad_norm(s["grads"], norm, mul, ws, max_norm=0.1)
    step(f, s, 1, mul=mul)
    step(f, ref, 1, mul=torch.tensor([float(mul)], device="cuda"))
    assert float(norm) > 0.1 and float(mul) < 1.0
    assert all(torch.equal(x, y) for k in ("params", "m", "v", "masters") for x, y in zip(s[k], ref[k]))
