"""Cases of the operators around the grouped expert products: the norm with the residual's
addition and an FP8 output (and its backward), the expert router (and its backward), and
the mixture-of-experts layer for a few tokens.

Each operator is here in its plain form, elementary torch operations in 32 bits (64 for
the norm's statistics, whose definition is in 64), and, where `own` is true, as the
library's calls. `exact` computes the same results in 64 bits.
"""
import math

import torch

own = False

NORM_EPS = 1e-5
EPS = 1e-12
E4M3_MAX = 448.0


def listed():
    return [
        # one token's residual stream between two layers of a 4096-wide model: latency
        dict(name="norm 1 token", op="norm", rows=1, cols=4096, kind="rms"),
        # a training step's 8192 tokens of the same model, before its MLP
        dict(name="norm 8192x4096", op="norm", rows=8192, cols=4096, kind="rms"),
        # an odd number of packed tokens of a 7168-wide model with LayerNorm
        dict(name="norm layer 2049x7168", op="norm", rows=2049, cols=7168, kind="layer"),
        # the backward of the training step's norm, residual gradient included
        dict(name="norm bwd 8192x4096", op="norm_bwd", rows=8192, cols=4096, kind="rms"),
        # the LayerNorm's backward over a short ragged batch
        dict(name="norm bwd layer 301x5120", op="norm_bwd", rows=301, cols=5120, kind="layer"),
        # a decode step's router: 64 tokens over 32 experts, the last 3 slots of the batch empty
        dict(name="route 64 tokens", op="route", tokens=64, experts=32, k=8, gate="softmax_topk", bits=16, pad=3),
        # the router of a training step: 16384 tokens, top 8 of 32
        dict(name="route 16384x32", op="route", tokens=16384, experts=32, k=8, gate="softmax", bits=32, pad=0),
        # its gradient, over many experts
        dict(name="route bwd 8192x256", op="route_bwd", tokens=8192, experts=256, k=8, gate="softmax", bits=32, pad=5),
        # a small layer, odd sizes, row-major weights: latency
        dict(name="moe 5 tokens small", op="moe", tokens=5, experts=8, k=2, D=1040, F=720, packed=False),
        # single-token decode, top 8 of 32 experts of [2048, 7168]
        dict(name="moe 1 token 32x2048x7168", op="moe", tokens=1, experts=32, k=8, D=7168, F=2048, packed=True),
        # a decode batch of 16 over the same layer: nearly every expert is read
        dict(name="moe 16 tokens 32x2048x7168", op="moe", tokens=16, experts=32, k=8, D=7168, F=2048, packed=True),
        # 64 tokens, top 1 of 16 experts of [8192, 5120], row-major weights
        dict(name="moe 64 tokens 16x8192x5120", op="moe", tokens=64, experts=16, k=1, D=5120, F=8192, packed=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm_bwd", "route", "route_bwd", "moe", "moe"])
    if op in ("norm", "norm_bwd"):
        cols = 8 * _log(rng, 8, 2048)
        rows = _log(rng, 1, min(65536, 8192 * 4096 // cols))
        return dict(op=op, rows=rows, cols=cols, kind=rng.choice(["rms", "rms", "layer"]))
    if op in ("route", "route_bwd"):
        experts = _log(rng, 4, 512)
        tokens = _log(rng, 1, min(65536, (1 << 24) // experts))
        return dict(op=op, tokens=tokens, experts=experts, k=rng.randint(1, min(8, experts)),
                    gate=rng.choice(["softmax", "softmax_topk", "sigmoid"]), bits=rng.choice([16, 32]),
                    pad=rng.randint(0, tokens // 4))
    packed = rng.random() < 0.5
    step = 64 if packed else 16
    experts = _log(rng, 4, 128)
    D = step * _log(rng, 256 // step, 7168 // step)
    F = step * _log(rng, max(1, 128 // step), max(2, min(8192, 1_800_000_000 // (3 * experts * D)) // step))
    return dict(op="moe", tokens=_log(rng, 1, 64), experts=experts, k=rng.randint(1, min(8, experts)), D=D, F=F,
                packed=packed)


def work(case):
    op = case["op"]
    if op in ("norm", "norm_bwd"):
        rows, cols, layer = case["rows"], case["cols"], case["kind"] == "layer"
        if op == "norm":  # x, res -> h, y, q; gamma (beta); scale's inverse and the statistics
            return dict(bytes=rows * cols * 9 + cols * (4 if layer else 2) + rows * (12 if layer else 8),
                        flops=rows * cols * (10 if layer else 8))
        return dict(bytes=rows * cols * 8 + cols * (6 if layer else 4) + rows * (8 if layer else 4),
                    flops=rows * cols * (14 if layer else 11))
    if op in ("route", "route_bwd"):
        T, E, k, esz = case["tokens"], case["experts"], case["k"], case["bits"] // 8
        if op == "route":
            return dict(bytes=T * E * esz + 16 * T * k + 4 * (E + 1), flops=T * E * (k + 3))
        return dict(bytes=2 * T * E * esz + 12 * T * k, flops=T * (5 * E + 3 * k))
    T, E, k, D, F = (case[n] for n in ("tokens", "experts", "k", "D", "F"))
    active = E * (1.0 - (1.0 - k / E) ** T)  # the experts that some token chooses, in the mean
    return dict(bytes=active * (3 * F * D + 4 * (2 * F + D)) + 4 * T * D + 8 * T * k, flops=6.0 * T * k * F * D)


# ---- inputs ---------------------------------------------------------------------------


def _bf(g, shape, scale=1.0, shift=0.0):
    return (torch.randn(shape, generator=g, device="cuda") * scale + shift).to(torch.bfloat16)


def _logits(case, g):
    T, E = case["tokens"], case["experts"]
    l = torch.randn((T, E), generator=g, device="cuda") * 1.5
    l = l.to(torch.bfloat16 if case.get("bits", 32) == 16 else torch.float32)
    if case.get("pad", 0):
        l[T - case["pad"]:] = -math.inf  # the empty slots of a padded batch: no expert
    return l


def _experts(g, E, N, K):
    """[E][N][K] e4m3 codes of N(0, 0.02) weights and their inverse scales [E][N]."""
    codes = torch.empty((E, N, K), dtype=torch.uint8, device="cuda")
    inv = torch.empty((E, N), device="cuda")
    for e in range(E):
        w = torch.randn((N, K), generator=g, device="cuda") * 0.02
        amax = w.abs().amax(1)
        codes[e] = (w * (E4M3_MAX / amax)[:, None]).to(torch.float8_e4m3fn).view(torch.uint8)
        inv[e] = amax / E4M3_MAX
    return codes, inv


def _pack(codes):
    """The k-packed layout: 1 KB chunks of 16 rows x 64 columns."""
    E, N, K = codes.shape
    return codes.reshape(E, N // 16, 16, K // 64, 64).permute(0, 1, 3, 2, 4).contiguous().reshape(E, N, K)


def _unpack(codes):
    E, N, K = codes.shape
    return codes.reshape(E, N // 16, K // 64, 16, 64).permute(0, 1, 3, 2, 4).reshape(E, N, K)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = dict(case)
    f32 = dict(dtype=torch.float32, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    op = case["op"]
    if op in ("norm", "norm_bwd"):
        rows, cols, layer = case["rows"], case["cols"], case["kind"] == "layer"
        s["gamma"] = _bf(g, (cols,), 0.1, 1.0)
        s["beta"] = _bf(g, (cols,), 0.1) if layer else None
        s["x"], s["res"] = _bf(g, (rows, cols)), _bf(g, (rows, cols), 2.0, 0.25 if layer else 0.0)
        s["h"] = torch.empty_like(s["x"])
        s["mean"] = torch.empty(rows, **f32) if layer else None
        s["rstd"] = torch.empty(rows, **f32)
        if op == "norm":
            s["y"] = torch.empty_like(s["x"])
            s["q"] = torch.empty((rows, cols), dtype=torch.uint8, device="cuda")
            s["scale"], s["inv"] = torch.empty(rows, **f32), torch.empty(rows, **f32)
        else:  # what the forward left behind, and the gradients that arrive
            h = (s["x"].float() + s["res"].float()).to(torch.bfloat16)
            mean, rstd = _stats(h, layer)
            s["h"], s["rstd"] = h, rstd
            s["mean"] = mean if layer else None
            s["dy"], s["dh"] = _bf(g, (rows, cols), 1e-2), _bf(g, (rows, cols), 1e-2)
            s["dx"] = torch.empty_like(h)
            s["dgamma"] = torch.empty_like(s["gamma"])
            s["dbeta"] = torch.empty_like(s["gamma"]) if layer else None
            del s["x"], s["res"]
        return s
    T, E, k = case["tokens"], case["experts"], case["k"]
    s["logits"] = _logits(case, g)
    if op == "route":
        s["ids"], s["weights"] = torch.empty((T, k), **i32), torch.empty((T, k), **f32)
        s["offsets"], s["order"], s["slot"] = torch.empty(E + 1, **i32), torch.empty(T * k, **i32), torch.empty((T, k), **i32)
        return s
    if op == "route_bwd":
        s["ids"], s["weights"] = _choose(s["logits"], k, case["gate"])
        s["dweights"] = torch.randn((T, k), generator=g, device="cuda") * 0.1
        s["dlogits"] = torch.empty_like(s["logits"])
        return s
    D, F = case["D"], case["F"]
    s["ids"], s["weights"] = _choose(s.pop("logits"), k, "softmax_topk")
    s["x"] = _bf(g, (T, D))
    s["w13"], s["w13_inv"] = _experts(g, E, 2 * F, D)
    s["w2"], s["w2_inv"] = _experts(g, E, D, F)
    if case["packed"]:
        s["w13"], s["w2"] = _pack(s["w13"]), _pack(s["w2"])
    s["out"] = torch.empty((T, D), dtype=torch.bfloat16, device="cuda")
    return s


# ---- the plain forms ---------------------------------------------------------------------


def _stats(h, layer):
    """mean and 1 / sqrt(var + eps) of each row: sums in 64 bits, rounded once."""
    hd = h.double()
    mean = hd.mean(1) if layer else torch.zeros_like(hd[:, 0])
    var = hd.square().mean(1) - mean.square()
    return mean.float(), (1.0 / (var + NORM_EPS).sqrt()).float()


def _norm(s):
    layer = s["kind"] == "layer"
    h = (s["x"].float() + s["res"].float()).to(torch.bfloat16)
    mean, rstd = _stats(h, layer)
    y = ((h.float() - mean[:, None]) * rstd[:, None]) * s["gamma"].float()
    if layer:
        y = y + s["beta"].float()
    y = y.to(torch.bfloat16)
    scale = E4M3_MAX / y.float().abs().amax(1).double().clamp_min(EPS)
    q = (y.float() * scale.float()[:, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    return dict(h=h, y=y, q=q, inv=(1.0 / scale).float(), rstd=rstd, **(dict(mean=mean) if layer else {}))


def _norm_bwd(s):
    layer = s["kind"] == "layer"
    dy, h, rstd = s["dy"].float(), s["h"].float(), s["rstd"][:, None]
    xh = (h - s["mean"][:, None]) * rstd if layer else h * rstd
    g = dy * s["gamma"].float()
    d = g - xh * (g * xh).mean(1, keepdim=True)
    if layer:
        d = d - g.mean(1, keepdim=True)
    out = dict(dx=(s["dh"].float() + rstd * d).to(torch.bfloat16), dgamma=(dy * xh).sum(0).to(torch.bfloat16))
    if layer:
        out["dbeta"] = dy.sum(0).to(torch.bfloat16)
    return out


def _gates(logits, chosen, valid, gate):
    """Gate weights of the chosen logits [T][k]; 0 where there is no expert."""
    if gate == "sigmoid":
        w = 1.0 / (1.0 + torch.exp(-chosen))
    else:
        top = chosen[:, :1]
        over = logits if gate == "softmax" else torch.where(valid, chosen, -math.inf)
        w = torch.exp(chosen - top) / torch.exp(over - top).sum(1, keepdim=True)
    return torch.where(valid, w, 0.0)


def _choose(logits, k, gate):
    lf = logits.float()
    val, idx = torch.sort(lf, dim=1, descending=True, stable=True)  # equal logits: the lowest index first
    val, idx = val[:, :k], idx[:, :k]
    valid = val > -math.inf
    return torch.where(valid, idx, -1).to(torch.int32), _gates(lf, val, valid, gate)


def _route(s):
    E = s["experts"]
    ids, w = _choose(s["logits"], s["k"], s["gate"])
    flat = ids.reshape(-1).long()
    key = torch.where(flat < 0, E, flat)
    order = torch.sort(key, stable=True)[1]
    counts = torch.zeros(E + 1, dtype=torch.int64, device=flat.device).index_add_(0, key, torch.ones_like(key))
    offsets = torch.cat([torch.zeros_like(counts[:1]), counts[:E].cumsum(0)])
    slot = torch.empty_like(order)
    slot[order] = torch.arange(order.numel(), device=order.device)
    used = torch.arange(order.numel(), device=order.device) < offsets[E]
    return dict(ids=ids, weights=w, offsets=offsets.to(torch.int32),
                order=torch.where(used, order, -1).to(torch.int32),
                slot=torch.where(flat < 0, -1, slot).to(torch.int32).reshape(ids.shape))


def _route_bwd(s):
    lf, ids, w, dw = s["logits"].float(), s["ids"].long(), s["weights"], s["dweights"]
    valid = ids >= 0
    at = ids.clamp_min(0)
    wd = torch.where(valid, w * dw, 0.0)
    out = torch.zeros_like(lf)
    if s["gate"] == "sigmoid":
        out.scatter_add_(1, at, wd * (1.0 - w))
    elif s["gate"] == "softmax_topk":
        out.scatter_add_(1, at, wd - w * wd.sum(1, keepdim=True))
    else:
        top = lf.amax(1, keepdim=True)
        p = torch.exp(lf - top)
        p = torch.where(top > -math.inf, p / p.sum(1, keepdim=True), 0.0)
        out = -p * wd.sum(1, keepdim=True)
        out.scatter_add_(1, at, wd)
    return dict(dlogits=out.to(s["logits"].dtype))


def _moe(s):
    T, E, D, F = s["tokens"], s["experts"], s["D"], s["F"]
    w13, w2 = (_unpack(s["w13"]), _unpack(s["w2"])) if s["packed"] else (s["w13"], s["w2"])
    w13 = w13.view(torch.float8_e4m3fn).float() * s["w13_inv"][:, :, None]
    w2 = w2.view(torch.float8_e4m3fn).float() * s["w2_inv"][:, :, None]
    p = torch.matmul(s["x"].float(), w13.reshape(E * 2 * F, D).t()).reshape(T, E, 2, F)
    gate, up = p[:, :, 0], p[:, :, 1]
    share = torch.zeros((T, E), device=p.device)
    share.scatter_add_(1, s["ids"].long().clamp_min(0), torch.where(s["ids"] >= 0, s["weights"], 0.0))
    a = gate / (1.0 + torch.exp(-gate)) * up * share[:, :, None]
    out = torch.matmul(a.reshape(T, E * F), w2.permute(0, 2, 1).reshape(E * F, D))
    return dict(out=out.to(torch.bfloat16))


def run(s):
    if own:
        return _run_own(s)
    return dict(norm=_norm, norm_bwd=_norm_bwd, route=_route, route_bwd=_route_bwd, moe=_moe)[s["op"]](s)


# ---- the library's calls -----------------------------------------------------------------


def _run_own(s):
    import fp8_dynamic_scaling_amd as f
    op = s["op"]
    if op == "norm":
        kind = f.NORM_LAYER if s["kind"] == "layer" else f.NORM_RMS
        f.fp8_add_norm_quant_row(s["x"], s["res"], s["gamma"], s["beta"], kind, NORM_EPS, f.E4M3_NATIVE, EPS, s["h"],
                                 s["y"], s["q"], s["scale"], s["inv"], mean=s["mean"], rstd=s["rstd"])
        return dict(h=s["h"], y=s["y"], q=s["q"].view(torch.float8_e4m3fn), inv=s["inv"], rstd=s["rstd"],
                    **(dict(mean=s["mean"]) if s["kind"] == "layer" else {}))
    if op == "norm_bwd":
        kind = f.NORM_LAYER if s["kind"] == "layer" else f.NORM_RMS
        if "ws" not in s:
            s["ws"] = torch.empty(f.fp8_add_norm_bwd_ws_bytes(s["rows"], s["cols"], kind), dtype=torch.uint8,
                                  device="cuda")
        f.fp8_add_norm_bwd(s["dy"], s["dh"], s["h"], s["gamma"], s["mean"], s["rstd"], kind, s["dx"], s["dgamma"],
                           s["dbeta"], s["ws"])
        return dict(dx=s["dx"], dgamma=s["dgamma"], **(dict(dbeta=s["dbeta"]) if s["kind"] == "layer" else {}))
    if op in ("route", "route_bwd"):
        gate = dict(softmax=f.GATE_SOFTMAX, softmax_topk=f.GATE_SOFTMAX_TOPK, sigmoid=f.GATE_SIGMOID)[s["gate"]]
        if op == "route_bwd":
            f.fp8_moe_route_bwd(s["logits"], gate, s["ids"], s["weights"], s["dweights"], s["dlogits"])
            return dict(dlogits=s["dlogits"])
        if "ws" not in s:
            s["ws"] = torch.empty(f.fp8_moe_route_ws_bytes(s["tokens"], s["experts"], s["k"]), dtype=torch.uint8,
                                  device="cuda")
        f.fp8_moe_route(s["logits"], gate, s["ids"], s["weights"], s["offsets"], s["order"], s["slot"], s["ws"])
        return {n: s[n] for n in ("ids", "weights", "offsets", "order", "slot")}
    if "ws" not in s:
        s["ws"] = torch.empty(f.fp8_moe_few_ws_bytes(s["tokens"], s["k"], s["F"]), dtype=torch.uint8, device="cuda")
    f.fp8_moe_few(s["x"], s["ids"], s["weights"], s["w13"], s["w13_inv"], s["w2"], s["w2_inv"], f.E4M3_NATIVE,
                  s["out"], s["ws"], packed=s["packed"])
    return dict(out=s["out"])


# ---- the results in 64 bits ----------------------------------------------------------------


def exact(case, seed):
    s = prepare(case, seed)
    op, D64 = case["op"], torch.float64
    if op == "norm":
        layer = case["kind"] == "layer"
        total = s["x"].to(D64) + s["res"].to(D64)
        h = total.to(torch.bfloat16).to(D64)  # the norm is that of the stored residual stream
        n = h.shape[1]
        mean = h.sum(1) / n if layer else torch.zeros(h.shape[0], dtype=D64, device=h.device)
        rstd = torch.rsqrt((h - mean[:, None]).pow(2).sum(1) / n + NORM_EPS)
        y = torch.addcmul(s["beta"].to(D64) if layer else torch.zeros((), dtype=D64, device=h.device),
                          (h - mean[:, None]) * rstd[:, None], s["gamma"].to(D64))
        # the codes are those of the stored bf16 row, whose definition rounds each operation
        # to 32 bits: a product or sum of two 32-bit values taken in 64 and rounded to 32
        t = ((h - mean.float().to(D64)[:, None]).float().to(D64) * rstd.float().to(D64)[:, None]).float().to(D64)
        t = (t * s["gamma"].to(D64)).float()
        if layer:
            t = (t.to(D64) + s["beta"].to(D64)).float()
        t = t.to(torch.bfloat16).to(D64)
        peak = t.abs().max(1).values.clamp(min=EPS)
        return dict(h=total, y=y, q=t * (E4M3_MAX / peak)[:, None], inv=peak / E4M3_MAX, rstd=rstd,
                    **(dict(mean=mean) if layer else {}))
    if op == "norm_bwd":
        layer, n = case["kind"] == "layer", case["cols"]
        h, dy = s["h"].to(D64), s["dy"].to(D64)
        mean = h.sum(1, keepdim=True) / n if layer else 0.0
        sd = ((h - mean).pow(2).sum(1, keepdim=True) / n + NORM_EPS).sqrt()
        xh, up = (h - mean) / sd, dy * s["gamma"].to(D64)
        inner = up - xh * ((up * xh).sum(1, keepdim=True) / n) - (up.sum(1, keepdim=True) / n if layer else 0.0)
        out = dict(dx=inner / sd + s["dh"].to(D64), dgamma=torch.linalg.vecdot(dy, xh, dim=0))
        if layer:
            out["dbeta"] = dy.sum(0)
        return out
    if op in ("route", "route_bwd"):
        l, k = s["logits"].to(D64), case["k"]
        T, E = l.shape
        # the k best by comparison: how many experts come before each one
        ids = torch.full((T, k), -1, dtype=torch.int64, device=l.device)
        left = l.clone()
        for j in range(k):
            best = left.max(1, keepdim=True).values
            first = (left == best).to(torch.int8).argmax(1)
            ids[:, j] = torch.where(best[:, 0] > -math.inf, first, -1)
            left.scatter_(1, first[:, None], -math.inf)
        valid = ids >= 0
        val = torch.gather(l, 1, ids.clamp(min=0)).masked_fill(~valid, -math.inf)
        if case["gate"] == "sigmoid":
            w = torch.sigmoid(val)
        elif case["gate"] == "softmax":
            w = torch.gather(torch.softmax(l, 1), 1, ids.clamp(min=0))
        else:
            w = torch.softmax(val, 1)
        w = w.masked_fill(~valid, 0.0)
        if op == "route":
            return dict(ids=ids, weights=w, offsets=None, order=None, slot=None)
        wl = l.clone().requires_grad_(True)
        live = valid.any(1)
        if not bool(live.any()):
            return dict(dlogits=torch.zeros_like(l))
        rows = wl[live]
        if case["gate"] == "sigmoid":
            score = torch.sigmoid(torch.gather(rows, 1, ids[live].clamp(min=0)))
        elif case["gate"] == "softmax":
            score = torch.gather(torch.softmax(rows, 1), 1, ids[live].clamp(min=0))
        else:
            score = torch.softmax(torch.gather(rows, 1, ids[live].clamp(min=0)).masked_fill(~valid[live], -math.inf), 1)
        (score * s["dweights"].to(D64)[live]).masked_fill(~valid[live], 0.0).sum().backward()
        return dict(dlogits=wl.grad)
    F, x = case["F"], s["x"].to(D64)
    w13, w2 = (_unpack(s["w13"]), _unpack(s["w2"])) if case["packed"] else (s["w13"], s["w2"])
    out = torch.zeros_like(x)
    for e in torch.unique(s["ids"]).tolist():
        if e < 0:
            continue
        t, j = torch.nonzero(s["ids"] == e, as_tuple=True)
        m13 = w13[e].view(torch.float8_e4m3fn).to(D64) * s["w13_inv"][e].to(D64)[:, None]
        m2 = w2[e].view(torch.float8_e4m3fn).to(D64) * s["w2_inv"][e].to(D64)[:, None]
        u = x[t] @ m13.t()
        a = torch.nn.functional.silu(u[:, :F]) * u[:, F:]
        out.index_add_(0, t, (a @ m2.t()) * s["weights"][t, j].to(D64)[:, None])
    return dict(out=out)
