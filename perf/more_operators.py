"""Cases of the operators of an FP8 feed-forward block's training step: the gated product (both
projections, the activation and their product in one FP8 GEMM), its backward with the rowwise
quantization of the gradient, the AdamW step over many tensors with 32-bit or 8-bit states, and
the gradients' norm that clips them.

Each operator is here in its plain form, elementary torch operations in 32 bits (64 for the
norm's sums), and, where `own` is true, as the library's calls. `exact` computes the same results
in 64 bits.
"""
import math

import torch

own = False

EPS = 1e-12
E4M3_MAX = 448.0
E5M2_MAX = 57344.0
LR, BETA1, BETA2, ADAM_EPS, DECAY = 3e-4, 0.9, 0.95, 1e-8, 0.1
MLP = "58720256,58720256,58720256,4096,4096"  # gate, up and down weights of 14336 x 4096, two norms


def listed():
    return [
        # one token through the block's first half, 14336 features of a 4096-wide model: reads weights
        dict(name="gated 1 token 14336x4096", op="gated", rows=1, F=14336, K=4096, E=0, act="silu", packed=True,
             save=False, fast=True, pad=0),
        # a training step's 8192 tokens, both projections kept for the backward
        dict(name="gated 8192x14336x4096", op="gated", rows=8192, F=14336, K=4096, E=0, act="silu", packed=True,
             save=True, fast=True, pad=0),
        # a ragged batch of a small GELU model, row-major weights, sums of full precision
        dict(name="gated 333x1040x720", op="gated", rows=333, F=1040, K=720, E=0, act="gelu", packed=False,
             save=True, fast=False, pad=0),
        # 32768 sorted rows of 32 experts of [2048, 7168], the last 512 slots empty
        dict(name="gated 32 experts 32768 rows", op="gated", rows=32768, F=2048, K=7168, E=32, act="silu",
             packed=True, save=True, fast=True, pad=512),
        # the training step's gradient through the gate, its codes for the grad-input product
        dict(name="gate bwd 8192x14336", op="gate_bwd", rows=8192, F=14336, act="silu", e5=True, h=False),
        # a short ragged batch, the activations computed again for the down weight's gradient
        dict(name="gate bwd 301x2056", op="gate_bwd", rows=301, F=2056, act="gelu", e5=False, h=True),
        # norm weights and biases only: latency
        dict(name="adamw 6 vectors", op="adamw", sizes="4096,4096,14336,4096,256,1", bits=32, params=16, grads=16,
             master=False, seed=0, scaled=False),
        # the weights of one feed-forward block, bf16 with an fp32 copy
        dict(name="adamw block 32-bit", op="adamw", sizes=MLP, bits=32, params=16, grads=16, master=True, seed=0,
             scaled=True),
        # the same block with 8-bit states and stochastic rounding, no copy
        dict(name="adamw block 8-bit", op="adamw", sizes=MLP, bits=8, params=16, grads=16, master=False, seed=12345,
             scaled=True),
        # odd tensors in fp32 with 8-bit states to nearest
        dict(name="adamw ragged 8-bit", op="adamw", sizes="1,31,33,4097,100003,65537,77777,513,12289,999983", bits=8,
             params=32, grads=32, master=False, seed=0, scaled=False),
        # the norm of that block's gradients
        dict(name="norm of a block", op="norm", sizes=MLP, grads=16, max_norm=1.0),
        # and of odd fp32 tensors
        dict(name="norm ragged", op="norm", sizes="1,31,33,4097,100003,65537,77777,513,12289,999983", grads=32,
             max_norm=1e9),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["gated", "gated", "gated", "gate_bwd", "gate_bwd", "adamw", "adamw", "adamw", "norm"])
    if op == "gated":
        packed = rng.random() < 0.6
        K = 128 * _log(rng, 2, 56) if packed else 16 * _log(rng, 4, 448)
        F = 16 * _log(rng, 4, 896)
        most = int(1.9e12 / (4 * F * K))
        E = rng.choice([0, 0, _log(rng, 2, 64)])
        if E and E * 2 * F * K > 2_000_000_000:
            E = max(2, 2_000_000_000 // (2 * F * K))
        rows = _log(rng, 1, max(1, min(16384, most)))
        if E:
            rows += rows % 2  # pairs of rows share a line of the packed layout
        return dict(op=op, rows=rows, F=F, K=K, E=E, act=rng.choice(["silu", "silu", "gelu"]), packed=packed,
                    save=rng.random() < 0.6, fast=rng.random() < 0.7, pad=rng.randint(0, rows // 8) if E else 0)
    if op == "gate_bwd":
        F = 8 * _log(rng, 4, 2048)
        return dict(op=op, rows=_log(rng, 1, min(32768, 8192 * 14336 // F)), F=F,
                    act=rng.choice(["silu", "silu", "gelu"]), e5=rng.random() < 0.7, h=rng.random() < 0.5)
    sizes = ",".join(str(_log(rng, 1, 8_000_000)) for _ in range(_log(rng, 1, 40)))
    if op == "norm":
        return dict(op=op, sizes=sizes, grads=rng.choice([16, 32]), max_norm=rng.choice([1.0, 1e9]))
    params = rng.choice([16, 16, 32])
    return dict(op=op, sizes=sizes, bits=rng.choice([8, 32]), params=params, grads=rng.choice([16, params]),
                master=params == 16 and rng.random() < 0.5, seed=rng.choice([0, rng.randint(1, 1 << 30)]),
                scaled=rng.random() < 0.5)


def _sizes(case):
    return [int(n) for n in case["sizes"].split(",")]


def work(case):
    op = case["op"]
    if op == "gated":
        M, F, K, E = case["rows"] - case["pad"], case["F"], case["K"], max(1, case["E"])
        read = M * K + E * 2 * F * K + 4 * (M + E * 2 * F) + (4 * (E + 1) if case["E"] else 0)
        return dict(bytes=read + M * F * (6 if case["save"] else 2), flops=4.0 * M * F * K + 8.0 * M * F)
    if op == "gate_bwd":
        M, F = case["rows"], case["F"]
        return dict(bytes=M * F * (12 + (2 if case["h"] else 0)) + 4 * M, flops=20.0 * M * F)
    n, g = sum(_sizes(case)), case["grads"] // 8
    if op == "norm":
        return dict(bytes=n * g, flops=2.0 * n)
    state = 16 if case["bits"] == 32 else 4 + 4 / 32
    return dict(bytes=n * (g + state + (8 + 2 if case["master"] else 2 * case["params"] // 8)), flops=16.0 * n)


# ---- inputs ---------------------------------------------------------------------------


def _codes(g, shape, scale):
    """e4m3 codes of N(0, scale) rows and their inverse scales."""
    x = torch.randn(shape, generator=g, device="cuda") * scale
    amax = x.abs().amax(-1, keepdim=True)
    return (x * (E4M3_MAX / amax)).to(torch.float8_e4m3fn).view(torch.uint8), (amax / E4M3_MAX).squeeze(-1)


def _pack(codes):
    """The k-packed layout: 1 KB chunks of 16 rows x 64 columns."""
    E, N, K = codes.shape
    return codes.reshape(E, N // 16, 16, K // 64, 64).permute(0, 1, 3, 2, 4).contiguous().reshape(E, N, K)


def _unpack(codes):
    E, N, K = codes.shape
    return codes.reshape(E, N // 16, K // 64, 16, 64).permute(0, 1, 3, 2, 4).reshape(E, N, K)


def _pair(codes):
    """The pair-interleaved layout: rows 2i and 2i + 1 share each 128-byte line of 64 columns."""
    M, K = codes.shape
    return codes.reshape(M // 2, 2, K // 64, 64).permute(0, 2, 1, 3).contiguous().reshape(M, K)


def _unpair(codes):
    M, K = codes.shape
    return codes.reshape(M // 2, K // 64, 2, 64).permute(0, 2, 1, 3).reshape(M, K)


def _split(case, g):
    """Rows per expert: uneven, the first expert empty, `pad` rows of none at the end."""
    E, used = case["E"], case["rows"] - case["pad"]
    share = torch.rand(E, generator=g, device="cuda") + 0.25
    share[0] = 0.0
    cut = (share.cumsum(0) / share.sum() * used).round().to(torch.int32)
    cut[-1] = used
    return torch.cat([torch.zeros_like(cut[:1]), cut])


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s, op = dict(case), case["op"]
    f32, bf = dict(dtype=torch.float32, device="cuda"), dict(dtype=torch.bfloat16, device="cuda")
    if op == "gated":
        M, F, K, E = case["rows"], case["F"], case["K"], case["E"]
        s["a"], s["a_inv"] = _codes(g, (M, K), 1.0)
        w = [_codes(g, (2 * F, K), 0.02) for _ in range(max(1, E))]
        s["b"], s["b_inv"] = torch.stack([c for c, _ in w]), torch.stack([i for _, i in w])
        if case["packed"]:
            s["b"] = _pack(s["b"])
        if E:
            s["offsets"] = _split(case, g)
            s["most"] = int((s["offsets"][1:] - s["offsets"][:-1]).max())
            if case["packed"]:
                s["a"] = _pair(s["a"])
        else:
            s["b"], s["b_inv"] = s["b"][0], s["b_inv"][0]
        s["out"] = torch.zeros((M, F), **bf)
        s["gu"] = torch.zeros((M, 2 * F), **bf) if case["save"] else None
        return s
    if op == "gate_bwd":
        M, F = case["rows"], case["F"]
        s["gu"] = (torch.randn((M, 2 * F), generator=g, device="cuda") * 1.5).to(torch.bfloat16)
        s["dh"] = (torch.randn((M, F), generator=g, device="cuda") * 1e-3).to(torch.bfloat16)
        s["dgu"], s["h"] = torch.empty((M, 2 * F), **bf), torch.empty((M, F), **bf) if case["h"] else None
        s["q"] = torch.empty((M, 2 * F), dtype=torch.uint8, device="cuda")
        s["scale"], s["inv"] = torch.empty(M, **f32), torch.empty(M, **f32)
        return s
    gt = torch.bfloat16 if case["grads"] == 16 else torch.float32
    s["grads"] = [(torch.randn(n, generator=g, device="cuda") * 1e-2).to(gt) for n in _sizes(case)]
    if op == "norm":
        s["norm"], s["mul"] = torch.empty(1, **f32), torch.empty(1, **f32)
        s["step"] = torch.zeros(1, dtype=torch.int32, device="cuda")
        return s
    full = [torch.randn(n, generator=g, device="cuda") * 0.02 for n in _sizes(case)]
    s["params"] = [p.to(torch.bfloat16) if case["params"] == 16 else p for p in full]
    s["masters"] = full if case["master"] else None
    m = [torch.randn(n, generator=g, device="cuda") * 1e-3 for n in _sizes(case)]
    r = [torch.randn(n, generator=g, device="cuda").abs() * 1e-2 for n in _sizes(case)]
    if case["bits"] == 8:
        s["m"], s["ms"] = (list(x) for x in zip(*(_mx(x, None) for x in m)))
        s["v"], s["vs"] = (list(x) for x in zip(*(_mx(x, None, lift=True) for x in r)))
    else:
        s["m"], s["v"], s["ms"], s["vs"] = m, [x * x for x in r], None, None
    s["t"] = 1000  # steps taken before
    s["mul"] = torch.full((1,), 0.37, **f32) if case["scaled"] else None
    return s


# ---- the plain forms ---------------------------------------------------------------------


def _gate(g, act):
    """The activation and its derivative, x * sigmoid(z(x)) for both kinds."""
    c = math.sqrt(8.0 / math.pi)
    z, dz = (g, 1.0) if act == "silu" else (c * (g + 0.044715 * g * g * g), c * (1.0 + 3 * 0.044715 * g * g))
    sg = 1.0 / (1.0 + torch.exp(-z))
    return g * sg, sg + g * sg * (1.0 - sg) * dz


def _gated(s):
    E, F, K = s["E"], s["F"], s["K"]
    w = s["b"] if E else s["b"][None]
    w = (_unpack(w) if s["packed"] else w).view(torch.float8_e4m3fn).float() * s["b_inv"].reshape(-1, 2 * F, 1)
    a = _unpair(s["a"]) if E and s["packed"] else s["a"]
    a = a.view(torch.float8_e4m3fn).float() * s["a_inv"][:, None]
    if not E:
        p = torch.matmul(a, w[0].t())
    else:  # every expert's rows, filled up to the longest; rows of no expert stay as they were
        off = s["offsets"].long()
        at = torch.arange(s["most"], device=a.device)[None] + off[:-1, None]
        live = at < off[1:, None]
        p = torch.matmul(a[torch.where(live, at, 0)], w.transpose(1, 2).contiguous())[live]
    g, u = p[:, :F], p[:, F:]
    n = p.shape[0]
    s["out"][:n] = (_gate(g, s["act"])[0] * u).to(torch.bfloat16)
    if not s["save"]:
        return dict(out=s["out"])
    s["gu"][:n] = p.to(torch.bfloat16)
    return dict(out=s["out"], gu=s["gu"])


def _gate_bwd(s):
    F, top = s["F"], E5M2_MAX if s["e5"] else E4M3_MAX
    g, u, dh = s["gu"][:, :F].float(), s["gu"][:, F:].float(), s["dh"].float()
    a, da = _gate(g, s["act"])
    d = torch.cat([dh * u * da, dh * a], 1)
    scale = top / d.abs().amax(1).double().clamp_min(EPS)
    q = (d * scale.float()[:, None]).clamp(-top, top).to(torch.float8_e5m2 if s["e5"] else torch.float8_e4m3fn)
    out = dict(dgu=d.to(torch.bfloat16), q=q, inv=(1.0 / scale).float())
    if s["h"] is not None:
        out["h"] = (a * u).to(torch.bfloat16)
    return out


def _mix(x):
    """Wellons' 32-bit integer hash with the low bias, on int64 tensors or Python numbers."""
    x = x & 0xFFFFFFFF
    x = ((x ^ (x >> 16)) * 0x7FEB352D) & 0xFFFFFFFF
    x = ((x ^ (x >> 15)) * 0x846CA68B) & 0xFFFFFFFF
    return x ^ (x >> 16)


def _random(n, seed, index, step):
    """32 random bits for each element of the index-th tensor at a step."""
    key = _mix((seed >> 32) ^ _mix(seed ^ _mix(index)))
    return _mix(torch.arange(n, device="cuda") + _mix(key + step))


def _mx(x, bits, lift=False):
    """MXFP8: a power of two for each 32 values, the smallest with which the largest is at most 448;
    codes to nearest, or with 16 random bits below the code's last place. lift: a value above zero
    keeps a code above zero."""
    n = x.numel()
    pad = torch.zeros(-(-n // 32) * 32, device=x.device)
    pad[:n] = x
    top = pad.reshape(-1, 32).abs().amax(1).view(torch.int32)
    e8 = ((top >> 23) - 8 + ((top & 0x7FFFFF) > 0x600000)).clamp_min(12)
    inv = ((254 - e8) << 23).view(torch.float32)
    y = (pad.reshape(-1, 32) * inv[:, None]).reshape(-1)[:n]
    if bits is not None:
        small = y.abs() < 2.0 ** -6  # below the smallest normal, codes are 2^-9 apart, as they are just above it
        t = torch.where(small, y.abs() + 2.0 ** -6, y.abs())
        t = ((t.view(torch.int32) + bits.to(torch.int32) * 16 + 8) & ~0xFFFFF).view(torch.float32)
        y = torch.copysign(torch.where(small, t - 2.0 ** -6, t), y)
    if lift:
        y = torch.where((x > 0) & (y < 2.0 ** -9), 2.0 ** -9, y)
    return y.to(torch.float8_e4m3fn), e8.to(torch.uint8)


def _unmx(codes, e8):
    n = codes.numel()
    return codes.float() * (e8.to(torch.int32) << 23).view(torch.float32).repeat_interleave(32)[:n]


def _adamw(s):
    s["t"] += 1
    step, c2 = LR / (1.0 - BETA1 ** s["t"]), 1.0 / math.sqrt(1.0 - BETA2 ** s["t"])
    eight = s["bits"] == 8
    for i, param in enumerate(s["params"]):
        bits = _random(param.numel(), s["seed"], i, s["t"]) if s["seed"] else None
        g = s["grads"][i].float()
        if s["mul"] is not None:
            g = g * s["mul"]
        m = _unmx(s["m"][i], s["ms"][i]) if eight else s["m"][i]
        v = _unmx(s["v"][i], s["vs"][i]).square() if eight else s["v"][i]
        m = m * BETA1 + g * (1.0 - BETA1)
        v = v * BETA2 + (g * g) * (1.0 - BETA2)
        r = torch.sqrt(v)
        p = s["masters"][i] if s["master"] else param.float()
        p = p * (1.0 - LR * DECAY) - (m / (r * c2 + ADAM_EPS)) * step
        if s["master"]:
            s["masters"][i].copy_(p)
        if param.dtype == torch.bfloat16 and bits is not None and not s["master"]:
            p = ((p.view(torch.int32) + ((bits ^ (bits >> 16)) & 0xFFFF).to(torch.int32)) & ~0xFFFF).view(torch.float32)
        param.copy_(p)
        if eight:
            lo, hi = (None, None) if bits is None else (bits & 0xFFFF, bits >> 16)
            for kind, x, b in (("m", m, lo), ("v", r, hi)):
                codes, e8 = _mx(x, b, lift=kind == "v")
                s[kind][i].copy_(codes)
                s[kind + "s"][i].copy_(e8)
        else:
            s["m"][i].copy_(m)
            s["v"][i].copy_(v)
    return _states(s)


def _cat(ts):
    """Many tensors as one output (codes have no concatenation of their own)."""
    if ts[0].dtype == torch.float8_e4m3fn:
        return torch.cat([t.view(torch.uint8) for t in ts]).view(torch.float8_e4m3fn)
    return torch.cat(ts)


def _states(s):
    if len(s["params"]) > 10:
        return {k: _cat(s[k]) for k in ("params", "masters", "m", "v", "ms", "vs") if s[k] is not None}
    return {k: s[k] for k in ("params", "masters", "m", "v", "ms", "vs") if s[k] is not None}


def _norm(s):
    norm = torch.stack([g.double().square().sum() for g in s["grads"]]).sum().sqrt()
    s["step"] += 1
    return dict(norm=norm.float().reshape(1), mul=(s["max_norm"] / (norm + 1e-6)).clamp_max(1.0).float().reshape(1),
                step=s["step"])


def run(s):
    if own:
        return _run_own(s)
    return dict(gated=_gated, gate_bwd=_gate_bwd, adamw=_adamw, norm=_norm)[s["op"]](s)


# ---- the library's calls -----------------------------------------------------------------


def _run_own(s):
    import fp8_dynamic_scaling_amd as f
    op = s["op"]
    if op in ("gated", "gate_bwd"):
        act = f.ACT_SILU if s["act"] == "silu" else f.ACT_GELU_TANH
    if op == "gated":
        if s["E"]:
            f.fp8_grouped_gated_mm(s["a"], s["b"], f.E4M3_NATIVE, s["a_inv"], s["b_inv"], s["offsets"], act, s["gu"],
                                   s["out"], packed=s["packed"], use_fast_accum=s["fast"])
        else:
            f.fp8_gated_mm(s["a"], s["b"], f.E4M3_NATIVE, f.SCALE_ROW, s["a_inv"], s["b_inv"], act, s["gu"], s["out"],
                           packed=s["packed"], use_fast_accum=s["fast"])
        return dict(out=s["out"], gu=s["gu"]) if s["save"] else dict(out=s["out"])
    if op == "gate_bwd":
        f.fp8_gated_bwd(s["dh"], s["gu"], act, f.E5M2_NATIVE if s["e5"] else f.E4M3_NATIVE, EPS, s["dgu"], s["q"],
                        s["scale"], s["inv"], h=s["h"])
        out = dict(dgu=s["dgu"], q=s["q"].view(torch.float8_e5m2 if s["e5"] else torch.float8_e4m3fn), inv=s["inv"])
        if s["h"] is not None:
            out["h"] = s["h"]
        return out
    if op == "norm":
        if "ws" not in s:
            s["ws"] = torch.empty(f.fp8_grad_norm_ws_bytes(s["grads"]), dtype=torch.uint8, device="cuda")
        f.fp8_grad_norm(s["grads"], s["norm"], s["mul"], s["ws"], max_norm=s["max_norm"], step=s["step"])
        return dict(norm=s["norm"], mul=s["mul"], step=s["step"])
    s["t"] += 1
    f.fp8_adamw(s["params"], s["grads"], s["m"], s["v"], LR, BETA1, BETA2, ADAM_EPS, DECAY, s["t"],
                exp_avg_scales=s["ms"], exp_avg_sq_scales=s["vs"], masters=s["masters"], seed=s["seed"],
                grad_mul=s["mul"])
    return _states(s)


# ---- the results in 64 bits ----------------------------------------------------------------


def _act64(x, act):
    return torch.nn.functional.silu(x) if act == "silu" else torch.nn.functional.gelu(x, approximate="tanh")


def exact(case, seed):
    s, D64 = prepare(case, seed), torch.float64
    op = case["op"]
    if op == "gated":
        E, F, M = case["E"], case["F"], case["rows"]
        cut = s["offsets"].tolist() if E else [0, M]
        out, gu = torch.zeros((M, F), dtype=D64, device="cuda"), torch.zeros((M, 2 * F), dtype=D64, device="cuda")
        codes = s["b"] if E else s["b"].unsqueeze(0)
        codes = _unpack(codes) if case["packed"] else codes
        a = _unpair(s["a"]) if E and case["packed"] else s["a"]
        invs = s["b_inv"].reshape(-1, 2 * F)
        for e in range(len(cut) - 1):
            lo, hi = cut[e], cut[e + 1]
            if lo == hi:
                continue
            w = codes[e].view(torch.float8_e4m3fn).to(D64)
            p = a[lo:hi].view(torch.float8_e4m3fn).to(D64) @ w.t()
            p *= s["a_inv"][lo:hi].to(D64)[:, None] * invs[e].to(D64)
            gu[lo:hi] = p
            out[lo:hi] = _act64(p[:, :F], case["act"]) * p[:, F:]
        return dict(out=out, gu=gu) if case["save"] else dict(out=out)
    if op == "gate_bwd":
        F, top = case["F"], E5M2_MAX if case["e5"] else E4M3_MAX
        dgu = torch.empty((case["rows"], 2 * F), dtype=D64, device="cuda")
        h = torch.empty((case["rows"], F), dtype=D64, device="cuda")
        for lo in range(0, case["rows"], 1024):
            x = s["gu"][lo:lo + 1024].to(D64).requires_grad_(True)
            with torch.enable_grad():
                y = _act64(x[:, :F], case["act"]) * x[:, F:]
                dgu[lo:lo + 1024] = torch.autograd.grad(y, x, s["dh"][lo:lo + 1024].to(D64))[0]
            h[lo:lo + 1024] = y.detach()
        peak = torch.linalg.vector_norm(dgu, math.inf, dim=1).clamp(min=EPS)
        # e5m2's rounding, 0.053 in the mean, would hide what a value in 64 bits could show
        out = dict(dgu=dgu, q=None if case["e5"] else dgu * (top / peak)[:, None], inv=peak / top)
        if case["h"]:
            out["h"] = h
        return out
    if op == "norm":
        norm = torch.linalg.vector_norm(torch.cat([g.to(D64) for g in s["grads"]]))
        return dict(norm=norm.reshape(1), mul=torch.clamp(case["max_norm"] / (norm + 1e-6), max=1.0).reshape(1),
                    step=None)
    t = s["t"] + 1
    got = dict(params=[], masters=[], m=[], v=[])
    for i, param in enumerate(s["params"]):
        wide = lambda c, e: c.to(D64) * torch.exp2(e.to(D64) - 127).repeat_interleave(32)[:c.numel()]  # noqa: E731
        m0 = wide(s["m"][i], s["ms"][i]) if case["bits"] == 8 else s["m"][i].to(D64)
        v0 = wide(s["v"][i], s["vs"][i]) ** 2 if case["bits"] == 8 else s["v"][i].to(D64)
        g = s["grads"][i].to(D64) * (s["mul"].to(D64) if case["scaled"] else 1.0)
        m, v = torch.lerp(g, m0, BETA1), torch.lerp(g * g, v0, BETA2)
        w = (s["masters"][i] if case["master"] else param).to(D64)
        w = w - LR * DECAY * w - LR * (m / (1 - BETA1 ** t)) / (torch.sqrt(v / (1 - BETA2 ** t)) + ADAM_EPS)
        got["params"].append(w)
        got["masters"].append(w)
        if case["bits"] == 32:
            got["m"].append(m)
            got["v"].append(v)
            continue
        for k, x in (("m", m), ("v", v.sqrt())):
            full = torch.zeros(-(-x.numel() // 32), 32, dtype=D64, device="cuda")
            full.view(-1)[:x.numel()] = x
            peak = full.abs().amax(1, keepdim=True).clamp(min=2.0 ** -115 * E4M3_MAX)
            got[k].append((full / torch.exp2(torch.ceil(torch.log2(peak / E4M3_MAX)))).view(-1)[:x.numel()])
    if not case["master"]:
        del got["masters"]
    if len(s["params"]) > 10:
        got = {k: torch.cat(v) for k, v in got.items()}
    if case["bits"] == 8:
        got["ms"] = got["vs"] = None if len(s["params"]) > 10 else [None] * len(s["params"])
    return got
