"""Host-side refusals of the gated product and its backward, the AdamW step and the gradients' norm
(CPU only): the C ABI before any device work, and the binding's checks of tensors; and the matrix-core
hazards of the gated kernels' assembly."""
import ctypes
import os
import subprocess

import pytest
import torch

import fp8_dynamic_scaling_amd as f
from fp8_dynamic_scaling_amd import build as hb
from tests.test_mfma_regalloc import mfma_overlaps, mfma_raw_hazards

FAKE = 0x100000  # 16-byte aligned, never dereferenced: validation fails first
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(f.LIB_PATH):
        hb.build()
    return f.load()


def _gated(lib, **kw):
    a = dict(a=FAKE, b=FAKE, fmt=f.E4M3_NATIVE, scaling=f.SCALE_ROW, a_inv=FAKE, b_inv=FAKE, M=4, F=48, K=128,
             act=f.ACT_SILU, packed=0, gu=FAKE, out=FAKE, fast=1, stream=None)
    a.update(kw)
    return lib.fp8_gated_mm(*a.values())


GATED_REFUSALS = [
    (dict(M=-1), f.ERR_INVALID_ARGUMENT), (dict(F=-8), f.ERR_INVALID_ARGUMENT), (dict(K=-16), f.ERR_INVALID_ARGUMENT),
    (dict(act=2), f.ERR_INVALID_ARGUMENT), (dict(act=-1), f.ERR_INVALID_ARGUMENT),
    (dict(a=None), f.ERR_INVALID_ARGUMENT), (dict(b=None), f.ERR_INVALID_ARGUMENT),
    (dict(a_inv=None), f.ERR_INVALID_ARGUMENT), (dict(b_inv=None), f.ERR_INVALID_ARGUMENT),
    (dict(out=None), f.ERR_INVALID_ARGUMENT), (dict(K=136), f.ERR_ALIGNMENT),
    (dict(packed=1, K=64), f.ERR_ALIGNMENT), (dict(packed=1, F=24), f.ERR_ALIGNMENT),
    (dict(a=FAKE + 8), f.ERR_ALIGNMENT), (dict(b=FAKE + 8), f.ERR_ALIGNMENT), (dict(a_inv=FAKE + 2), f.ERR_ALIGNMENT),
    (dict(b_inv=FAKE + 1), f.ERR_ALIGNMENT), (dict(gu=FAKE + 1), f.ERR_ALIGNMENT), (dict(out=FAKE + 1), f.ERR_ALIGNMENT),
    (dict(M=1 << 31), f.ERR_UNSUPPORTED), (dict(F=(1 << 21) + 1), f.ERR_UNSUPPORTED),
    (dict(packed=1, F=1 << 21, K=1024), f.ERR_UNSUPPORTED), (dict(packed=1, F=1 << 15, K=1 << 15), f.ERR_UNSUPPORTED),
]


@pytest.mark.parametrize("kw,want", GATED_REFUSALS + [
    (dict(scaling=f.SCALE_BLOCK128), f.ERR_UNSUPPORTED), (dict(scaling=f.SCALE_MX32), f.ERR_UNSUPPORTED),
    (dict(M=0, a=None, out=None), f.OK), (dict(F=0, b=None, out=None), f.OK),
])
def test_gated_mm_refusals(lib, kw, want):
    assert _gated(lib, **kw) == want


def _grouped(lib, **kw):
    a = dict(a=FAKE, b=FAKE, fmt=f.E4M3_NATIVE, a_inv=FAKE, b_inv=FAKE, offsets=FAKE, E=3, M=4, F=48, K=128,
             act=f.ACT_SILU, packed=0, gu=FAKE, out=FAKE, fast=1, stream=None)
    a.update(kw)
    return lib.fp8_grouped_gated_mm(*a.values())


@pytest.mark.parametrize("kw,want", GATED_REFUSALS + [
    (dict(E=0), f.ERR_INVALID_ARGUMENT), (dict(E=1025), f.ERR_INVALID_ARGUMENT),
    (dict(offsets=None), f.ERR_INVALID_ARGUMENT), (dict(offsets=FAKE + 2), f.ERR_ALIGNMENT),
    (dict(packed=1, M=3), f.ERR_ALIGNMENT), (dict(M=0, a=None, out=None, offsets=None), f.OK),
])
def test_grouped_gated_mm_refusals(lib, kw, want):
    assert _grouped(lib, **kw) == want


def _bwd(lib, **kw):
    a = dict(dh=FAKE, gu=FAKE, M=4, F=48, act=f.ACT_SILU, fmt=f.E5M2_NATIVE, eps=1e-12, dgu=FAKE, q=FAKE, scale=FAKE,
             inv=FAKE, h=FAKE, stream=None)
    a.update(kw)
    return lib.fp8_gated_bwd(*a.values())


@pytest.mark.parametrize("kw,want", [
    (dict(M=-1), f.ERR_INVALID_ARGUMENT), (dict(F=-8), f.ERR_INVALID_ARGUMENT), (dict(act=7), f.ERR_INVALID_ARGUMENT),
    (dict(eps=0.0), f.ERR_INVALID_ARGUMENT), (dict(eps=NAN), f.ERR_INVALID_ARGUMENT),
    (dict(dh=None), f.ERR_INVALID_ARGUMENT), (dict(gu=None), f.ERR_INVALID_ARGUMENT),
    (dict(scale=None), f.ERR_INVALID_ARGUMENT), (dict(q=None), f.ERR_INVALID_ARGUMENT),
    (dict(q=None, scale=None), f.ERR_INVALID_ARGUMENT),  # inv_scale alone
    (dict(dgu=None, q=None, scale=None, inv=None, h=None), f.ERR_INVALID_ARGUMENT),
    (dict(F=44), f.ERR_ALIGNMENT), (dict(F=32776), f.ERR_UNSUPPORTED), (dict(dh=FAKE + 8), f.ERR_ALIGNMENT),
    (dict(gu=FAKE + 8), f.ERR_ALIGNMENT), (dict(dgu=FAKE + 2), f.ERR_ALIGNMENT), (dict(h=FAKE + 8), f.ERR_ALIGNMENT),
    (dict(q=FAKE + 4), f.ERR_ALIGNMENT), (dict(scale=FAKE + 2), f.ERR_ALIGNMENT), (dict(inv=FAKE + 2), f.ERR_ALIGNMENT),
    (dict(M=0, dh=None, gu=None), f.OK),
])
def test_gated_bwd_refusals(lib, kw, want):
    assert _bwd(lib, **kw) == want


def _tensor(**kw):
    t = dict(p=FAKE, g=FAKE, m=FAKE, v=FAKE, ms=0, vs=0, master=0, n=100)
    t.update(kw)
    return tuple(t.values())


def _adamw(lib, tensors=None, **kw):
    rows = [_tensor()] if tensors is None else tensors
    table = (ctypes.c_int64 * max(1, 8 * len(rows)))(*[x for r in rows for x in r])
    a = dict(table=table, count=len(rows), p_type=f.OUT_BF16, g_type=f.OUT_BF16, state=f.STATE_F32, lr=1e-3, b1=0.9,
             b2=0.999, eps=1e-8, wd=0.1, step=1, seed=0, mul=None, step_dev=None, lr_dev=None, stream=None)
    a.update(kw)
    return lib.fp8_adamw(*a.values())


@pytest.mark.parametrize("tensors,kw,want", [
    (None, dict(count=-1), f.ERR_INVALID_ARGUMENT), (None, dict(table=None), f.ERR_INVALID_ARGUMENT),
    (None, dict(p_type=2), f.ERR_INVALID_ARGUMENT), (None, dict(g_type=-1), f.ERR_INVALID_ARGUMENT),
    (None, dict(state=2), f.ERR_INVALID_ARGUMENT), (None, dict(lr=-1.0), f.ERR_INVALID_ARGUMENT),
    (None, dict(lr=NAN), f.ERR_INVALID_ARGUMENT), (None, dict(b1=1.0), f.ERR_INVALID_ARGUMENT),
    (None, dict(b2=-0.1), f.ERR_INVALID_ARGUMENT), (None, dict(eps=INF), f.ERR_INVALID_ARGUMENT),
    (None, dict(wd=-0.1), f.ERR_INVALID_ARGUMENT), (None, dict(step=0), f.ERR_INVALID_ARGUMENT),
    (None, dict(mul=FAKE + 2), f.ERR_ALIGNMENT), (None, dict(step_dev=FAKE + 1), f.ERR_ALIGNMENT),
    (None, dict(lr_dev=FAKE + 2), f.ERR_ALIGNMENT),
    ([_tensor(n=-1)], {}, f.ERR_INVALID_ARGUMENT), ([_tensor(p=0)], {}, f.ERR_INVALID_ARGUMENT),
    ([_tensor(g=0)], {}, f.ERR_INVALID_ARGUMENT), ([_tensor(m=0)], {}, f.ERR_INVALID_ARGUMENT),
    ([_tensor(v=0)], {}, f.ERR_INVALID_ARGUMENT),
    ([_tensor()], dict(state=f.STATE_MX8), f.ERR_INVALID_ARGUMENT),  # no scales
    ([_tensor(ms=FAKE)], dict(state=f.STATE_MX8), f.ERR_INVALID_ARGUMENT),
    ([_tensor(), _tensor(master=FAKE)], {}, f.ERR_INVALID_ARGUMENT),
    ([_tensor(master=FAKE)], dict(p_type=f.OUT_F32), f.ERR_INVALID_ARGUMENT),
    ([_tensor(p=FAKE + 1)], {}, f.ERR_ALIGNMENT), ([_tensor(p=FAKE + 2)], dict(p_type=f.OUT_F32), f.ERR_ALIGNMENT),
    ([_tensor(g=FAKE + 1)], {}, f.ERR_ALIGNMENT), ([_tensor(m=FAKE + 2)], {}, f.ERR_ALIGNMENT),
    ([_tensor(v=FAKE + 2)], {}, f.ERR_ALIGNMENT), ([_tensor(master=FAKE + 2)], {}, f.ERR_ALIGNMENT),
    ([], {}, f.OK), ([_tensor(n=0, p=0, g=0, m=0, v=0)], {}, f.OK),
    ([_tensor(n=0)], dict(step=0, step_dev=FAKE, lr=NAN, lr_dev=FAKE), f.OK),
])
def test_adamw_refusals(lib, tensors, kw, want):
    assert _adamw(lib, tensors, **kw) == want


def _norm(lib, rows=((FAKE, 1 << 20, f.OUT_BF16),), **kw):
    table = (ctypes.c_int64 * max(1, 3 * len(rows)))(*[x for r in rows for x in r])
    a = dict(table=table, count=len(rows), scale=1.0, max_norm=1.0, norm=FAKE, mul=FAKE, step=None, ws=FAKE, ws_bytes=1 << 20,
             stream=None)
    a.update(kw)
    return lib.fp8_grad_norm(*a.values())


@pytest.mark.parametrize("kw,want", [
    (dict(count=-1), f.ERR_INVALID_ARGUMENT), (dict(table=None), f.ERR_INVALID_ARGUMENT),
    (dict(scale=0.0), f.ERR_INVALID_ARGUMENT), (dict(scale=-1.0), f.ERR_INVALID_ARGUMENT),
    (dict(scale=INF), f.ERR_INVALID_ARGUMENT), (dict(max_norm=0.0), f.ERR_INVALID_ARGUMENT),
    (dict(max_norm=NAN), f.ERR_INVALID_ARGUMENT), (dict(rows=((0, 4, 0),)), f.ERR_INVALID_ARGUMENT),
    (dict(rows=((FAKE, -4, 0),)), f.ERR_INVALID_ARGUMENT), (dict(rows=((FAKE, 4, 2),)), f.ERR_INVALID_ARGUMENT),
    (dict(rows=((FAKE + 1, 4, 0),)), f.ERR_ALIGNMENT), (dict(rows=((FAKE + 2, 4, 1),)), f.ERR_ALIGNMENT),
    (dict(norm=None, mul=None), f.ERR_INVALID_ARGUMENT), (dict(norm=FAKE + 2), f.ERR_ALIGNMENT),
    (dict(mul=FAKE + 1), f.ERR_ALIGNMENT), (dict(step=FAKE + 2), f.ERR_ALIGNMENT), (dict(ws=None), f.ERR_WORKSPACE),
    (dict(ws_bytes=7), f.ERR_WORKSPACE), (dict(ws=FAKE + 4), f.ERR_ALIGNMENT),
])
def test_grad_norm_refusals(lib, kw, want):
    assert _norm(lib, **kw) == want


def test_grad_norm_workspace(lib):
    # a partial sum of 8 bytes for each started piece of 2048, from 65 pieces or 129 tensors on
    def need(*sizes):
        table = (ctypes.c_int64 * (3 * len(sizes)))(*[x for n in sizes for x in (FAKE, n, 0)])
        return lib.fp8_grad_norm_ws_bytes(table, len(sizes))

    assert need(1, 0, 2049) == 0
    assert need(64 * 2048, 0) == 0 and need(64 * 2048, 1) == 8 * 65 and need(64 * 2048 + 1) == 8 * 65
    assert need(*[1] * 64) == 0 and need(*[1] * 65) == 8 * 65
    assert lib.fp8_grad_norm_ws_bytes(None, 0) == 0
    assert lib.fp8_grad_norm_ws_bytes(None, 2) == 0


def test_binding_refuses_cpu_tensors():
    x, q = torch.zeros(4, 48, dtype=torch.bfloat16), torch.zeros(4, 128, dtype=torch.uint8)
    b, inv = torch.zeros(96, 128, dtype=torch.uint8), torch.zeros(96)
    with pytest.raises(ValueError, match="on the GPU"):
        f.fp8_gated_mm(q, b, f.E4M3_NATIVE, f.SCALE_ROW, inv, inv, f.ACT_SILU, None, x)
    with pytest.raises(ValueError, match="on the GPU"):
        f.fp8_grouped_gated_mm(q, b, f.E4M3_NATIVE, inv, inv, torch.zeros(2, dtype=torch.int32), f.ACT_SILU, None, x)
    with pytest.raises(ValueError, match="on the GPU"):
        f.fp8_gated_bwd(x, torch.zeros(4, 96, dtype=torch.bfloat16), f.ACT_SILU, f.E5M2_NATIVE, 1e-12, None, None, None)
    with pytest.raises(ValueError, match="on the GPU"):
        f.fp8_adamw([inv], [inv], [inv], [inv], 1e-3, 0.9, 0.999, 1e-8, 0.0, 1)
    with pytest.raises(ValueError, match="one GPU"):
        f.fp8_grad_norm([inv], inv, None, None)
    with pytest.raises(ValueError, match="bfloat16 or float32"):
        f.fp8_adamw([inv.half()], [inv], [inv], [inv], 1e-3, 0.9, 0.999, 1e-8, 0.0, 1)
    with pytest.raises(ValueError, match="need exp_avg_scales"):
        f.fp8_adamw([inv], [inv], [inv.to(torch.uint8)], [inv.to(torch.uint8)], 1e-3, 0.9, 0.999, 1e-8, 0.0, 1)
    f.fp8_adamw([], [], [], [], 1e-3, 0.9, 0.999, 1e-8, 0.0, 1)


def _asm(src, tmp_path):
    out = tmp_path / (src + ".s")
    cmd = [hb.HIPCC] + hb.COMMON + ["--cuda-device-only", "-S", os.path.join(hb.HERE, "csrc", src), "-o", str(out)]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    return out.read_text()


def test_gated_kernels_have_no_mfma_hazard(tmp_path):
    asm = _asm("gemm_gated.hip", tmp_path)
    assert "v_mfma" in asm
    assert not mfma_overlaps(asm)
    assert not mfma_raw_hazards(asm)



def test_layers_refuse():
    from fp8_dynamic_scaling_amd import nn
    with pytest.raises(ValueError, match="act must be"):
        nn.Float8GatedLinear(64, 32, "relu")
    for K, F in ((40, 32), (64, 12), (64, 32776)):
        with pytest.raises(ValueError, match="multiple of 16"):
            nn.Float8GatedLinear(K, F)
    with pytest.raises(ValueError, match="multiple of 16"):
        nn.Float8GatedMLP(64, 24)
    with pytest.raises(RuntimeError, match="ROCm GPU"):
        nn.Float8GatedLinear(64, 32)(torch.zeros(2, 64, dtype=torch.bfloat16))


def _bf16(*shape):
    return torch.nn.Parameter(torch.zeros(shape, dtype=torch.bfloat16))


@pytest.mark.parametrize("kw,match", [
    (dict(state_bits=16), "state_bits"), (dict(lr=-1.0), "lr must"), (dict(lr=torch.zeros(1)), "capturable"),
    (dict(betas=(0.9, 1.0)), "betas"), (dict(betas=(-0.1, 0.9)), "betas"), (dict(eps=-1.0), "negative"),
    (dict(weight_decay=-1.0), "negative"), (dict(max_norm=0.0), "max_norm"), (dict(seed=0), "seed"),
])
def test_optimizer_refuses(kw, match):
    from fp8_dynamic_scaling_amd.optim import AdamW
    with pytest.raises(ValueError, match=match):
        AdamW([_bf16(4, 4)], **kw)


def test_optimizer_refuses_parameters():
    from fp8_dynamic_scaling_amd.optim import AdamW
    with pytest.raises(TypeError, match="bfloat16 or float32"):
        AdamW([torch.nn.Parameter(torch.zeros(4, dtype=torch.float16))])
    with pytest.raises(ValueError, match="contiguous"):
        AdamW([torch.nn.Parameter(torch.zeros(4, 6).t())])
    p = _bf16(4, 4)
    opt = AdamW([p])
    opt.step()  # nothing has a gradient
    with pytest.raises(ValueError, match="max_norm"):
        opt.step(grad_scale=0.5)
    p.grad = torch.zeros_like(p)
    with pytest.raises(ValueError, match="on the GPU"):
        opt.step()


@pytest.mark.parametrize("kw", [{}, dict(max_norm=1.0), dict(capturable=True)])
def test_optimizer_loads_states_as_they_were(kw):
    """Codes, fp32 moments of bf16 parameters and the count of steps survive load_state_dict, which casts states to the
    parameter's type by itself; with the count on the device it is one tensor for all parameters."""
    import copy
    from fp8_dynamic_scaling_amd.optim import AdamW
    for bits in (8, 32):
        a, b = (AdamW([_bf16(5, 7), _bf16(3)], state_bits=bits, master_weights=True, **kw) for _ in range(2))
        for p in a.param_groups[0]["params"]:
            a._new_state(p)
            for k, v in a.state[p].items():
                if torch.is_tensor(v) and k != "step":
                    v.copy_(torch.arange(v.numel()) * (1 if v.dtype == torch.uint8 else 1.0009))
        for p in a.param_groups[0]["params"]:
            if kw:
                a.state[p]["step"].fill_(9)
            else:
                a.state[p]["step"] = 9
        b.load_state_dict(copy.deepcopy(a.state_dict()))
        steps = []
        for p, q in zip(a.param_groups[0]["params"], b.param_groups[0]["params"]):
            assert a.state[p].keys() == b.state[q].keys()
            for k, v in a.state[p].items():
                w = b.state[q][k]
                assert (torch.equal(v, w) and v.dtype == w.dtype) if torch.is_tensor(v) else v == w
            steps.append(b.state[q]["step"])
        assert int(steps[0]) == 9 and (steps[0] is steps[1] if kw else True)


def test_optimizer_copies():
    import copy
    from fp8_dynamic_scaling_amd.optim import AdamW
    a = AdamW([_bf16(5, 7), _bf16(3)], state_bits=8, max_norm=2.0, seed=9)
    for p in a.param_groups[0]["params"]:
        a._new_state(p)
    b = copy.deepcopy(a)
    assert (b.state_bits, b.max_norm, b.seed, b.capturable) == (8, 2.0, 9, False)
    p, q = b.param_groups[0]["params"]
    assert b.state[p]["step"] is b.state[q]["step"] and b.state[p]["exp_avg"].dtype == torch.uint8
    b.step()


def test_optimizer_refuses_capture_without_states(monkeypatch):
    from fp8_dynamic_scaling_amd.optim import AdamW
    monkeypatch.setattr(torch.cuda, "is_initialized", lambda: True)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: True)
    p = _bf16(4)
    p.grad = torch.zeros_like(p)
    with pytest.raises(RuntimeError, match="capturable=True"):
        AdamW([p]).step()
    opt = AdamW([p], capturable=True)
    with pytest.raises(RuntimeError, match="take a step before"):
        opt.step()
    assert "exp_avg" not in opt.state[p]


@pytest.mark.parametrize("bits", [8, 32])
def test_optimizer_loads_its_own_kind_of_state(bits):
    from fp8_dynamic_scaling_amd.optim import AdamW
    make = lambda bits, **kw: AdamW([_bf16(5, 7)], state_bits=bits, **kw)  # noqa: E731
    a, other, kept = make(bits), make(40 - bits), make(bits, master_weights=True)
    a._new_state(a.param_groups[0]["params"][0])
    with pytest.raises(ValueError, match="states of"):
        other.load_state_dict(a.state_dict())
    assert not other.state
    p = kept.param_groups[0]["params"][0]
    with torch.no_grad():
        p.fill_(0.5)
    kept.load_state_dict(a.state_dict())  # saved without fp32 copies: they are made of the parameters
    assert torch.equal(kept.state[p]["master"], torch.full((35,), 0.5))


def test_optimizer_drops_a_refused_group():
    from fp8_dynamic_scaling_amd.optim import AdamW
    opt = AdamW([_bf16(4)])
    with pytest.raises(TypeError, match="bfloat16 or float32"):
        opt.add_param_group(dict(params=[torch.nn.Parameter(torch.zeros(4, dtype=torch.float16))]))
    with pytest.raises(ValueError, match="contiguous"):
        opt.add_param_group(dict(params=[torch.nn.Parameter(torch.zeros(4, 3, dtype=torch.bfloat16).t())]))
    assert len(opt.param_groups) == 1


def test_binding_refuses_shapes():
    bf = dict(dtype=torch.bfloat16)
    x, q = torch.zeros(4, 48, **bf), torch.zeros(4, 128, dtype=torch.uint8)
    b, inv = torch.zeros(96, 128, dtype=torch.uint8), torch.zeros(96)
    mm = lambda b, gu, out: f.fp8_gated_mm(q, b, f.E4M3_NATIVE, f.SCALE_ROW, inv, inv, f.ACT_SILU, gu, out)  # noqa: E731
    with pytest.raises(ValueError, match="codes of"):
        mm(torch.zeros(96, 256, dtype=torch.uint8), None, x)
    with pytest.raises(ValueError, match="gu must be"):
        mm(b, torch.zeros(8, 48, **bf), x)
    with pytest.raises(ValueError, match=r"out must be"):
        mm(b, None, torch.zeros(3, 48, **bf))
    with pytest.raises(ValueError, match="offsets must"):
        f.fp8_grouped_gated_mm(q, b, f.E4M3_NATIVE, inv, inv, None, f.ACT_SILU, None, x)
    with pytest.raises(ValueError, match="gu must be"):
        f.fp8_gated_bwd(x, x, f.ACT_SILU, f.E5M2_NATIVE, 1e-12, None, None, None)
