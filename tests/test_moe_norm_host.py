"""Host-side refusals of the residual norm, the expert router and the few-token expert layer
(CPU only): the C ABI before any device work, and the binding's checks of tensors."""
import os

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


def _norm(lib, **kw):
    a = dict(x=FAKE, res=FAKE, gamma=FAKE, beta=None, rows=4, cols=64, kind=f.NORM_RMS, norm_eps=1e-5,
             fmt=f.E4M3_NATIVE, eps=1e-12, h=FAKE, y=FAKE, q=FAKE, scale=FAKE, inv=FAKE, mean=None, rstd=FAKE,
             stream=None)
    a.update(kw)
    return lib.fp8_add_norm_quant_row(*a.values())


@pytest.mark.parametrize("kw,want", [
    (dict(rows=-1), f.ERR_INVALID_ARGUMENT), (dict(cols=-8), f.ERR_INVALID_ARGUMENT),
    (dict(kind=2), f.ERR_INVALID_ARGUMENT), (dict(beta=FAKE), f.ERR_INVALID_ARGUMENT),
    (dict(mean=FAKE), f.ERR_INVALID_ARGUMENT), (dict(res=None), f.ERR_INVALID_ARGUMENT),
    (dict(x=None), f.ERR_INVALID_ARGUMENT), (dict(gamma=None), f.ERR_INVALID_ARGUMENT),
    (dict(y=None, q=None), f.ERR_INVALID_ARGUMENT), (dict(scale=None), f.ERR_INVALID_ARGUMENT),
    (dict(eps=0.0), f.ERR_INVALID_ARGUMENT), (dict(norm_eps=-1.0), f.ERR_INVALID_ARGUMENT),
    (dict(norm_eps=NAN), f.ERR_INVALID_ARGUMENT), (dict(eps=INF), f.ERR_INVALID_ARGUMENT),
    (dict(cols=68), f.ERR_ALIGNMENT), (dict(cols=16392), f.ERR_UNSUPPORTED),
    (dict(rows=1 << 31), f.ERR_UNSUPPORTED),
    (dict(x=FAKE + 8), f.ERR_ALIGNMENT), (dict(res=FAKE + 2), f.ERR_ALIGNMENT), (dict(h=FAKE + 8), f.ERR_ALIGNMENT),
    (dict(y=FAKE + 8), f.ERR_ALIGNMENT), (dict(q=FAKE + 4), f.ERR_ALIGNMENT), (dict(scale=FAKE + 2), f.ERR_ALIGNMENT),
    (dict(inv=FAKE + 2), f.ERR_ALIGNMENT), (dict(rstd=FAKE + 2), f.ERR_ALIGNMENT),
    (dict(kind=f.NORM_LAYER, mean=FAKE + 2), f.ERR_ALIGNMENT),
    (dict(kind=f.NORM_LAYER, beta=FAKE + 2), f.ERR_ALIGNMENT),
    (dict(rows=0, x=None, y=None, q=None), f.OK),
])
def test_add_norm_refusals(lib, kw, want):
    assert _norm(lib, **kw) == want


def _norm_bwd(lib, **kw):
    a = dict(dy=FAKE, dh=FAKE, h=FAKE, gamma=FAKE, mean=None, rstd=FAKE, rows=4, cols=64, kind=f.NORM_RMS, dx=FAKE,
             dgamma=FAKE, dbeta=None, ws=FAKE, ws_bytes=1 << 30, stream=None)
    a.update(kw)
    return lib.fp8_add_norm_bwd(*a.values())


@pytest.mark.parametrize("kw,want", [
    (dict(rows=-1), f.ERR_INVALID_ARGUMENT), (dict(cols=-8), f.ERR_INVALID_ARGUMENT),
    (dict(kind=7), f.ERR_INVALID_ARGUMENT), (dict(mean=FAKE), f.ERR_INVALID_ARGUMENT),
    (dict(dbeta=FAKE), f.ERR_INVALID_ARGUMENT), (dict(kind=f.NORM_LAYER), f.ERR_INVALID_ARGUMENT),
    (dict(dy=None), f.ERR_INVALID_ARGUMENT), (dict(h=None), f.ERR_INVALID_ARGUMENT),
    (dict(gamma=None), f.ERR_INVALID_ARGUMENT), (dict(rstd=None), f.ERR_INVALID_ARGUMENT),
    (dict(dx=None), f.ERR_INVALID_ARGUMENT), (dict(cols=12), f.ERR_ALIGNMENT), (dict(cols=16392), f.ERR_UNSUPPORTED),
    (dict(dy=FAKE + 8), f.ERR_ALIGNMENT), (dict(dh=FAKE + 8), f.ERR_ALIGNMENT), (dict(h=FAKE + 8), f.ERR_ALIGNMENT),
    (dict(dx=FAKE + 8), f.ERR_ALIGNMENT), (dict(gamma=FAKE + 8), f.ERR_ALIGNMENT),
    (dict(dgamma=FAKE + 1), f.ERR_ALIGNMENT), (dict(rstd=FAKE + 1), f.ERR_ALIGNMENT),
    (dict(ws=None), f.ERR_WORKSPACE), (dict(ws_bytes=8), f.ERR_WORKSPACE), (dict(ws=FAKE + 4), f.ERR_ALIGNMENT),
    (dict(cols=0), f.OK), (dict(rows=0, dgamma=None), f.OK),
])
def test_add_norm_bwd_refusals(lib, kw, want):
    assert _norm_bwd(lib, **kw) == want


def _route(lib, **kw):
    a = dict(logits=FAKE, t=f.OUT_F32, T=100, E=32, k=8, gate=f.GATE_SOFTMAX, ids=FAKE, w=FAKE, offsets=FAKE,
             order=FAKE, slot=FAKE, ws=FAKE, ws_bytes=1 << 30, stream=None)
    a.update(kw)
    return lib.fp8_moe_route(*a.values())


ROUTE = [
    (dict(T=-1), f.ERR_INVALID_ARGUMENT), (dict(E=0), f.ERR_INVALID_ARGUMENT), (dict(k=0), f.ERR_INVALID_ARGUMENT),
    (dict(k=33), f.ERR_INVALID_ARGUMENT), (dict(t=2), f.ERR_INVALID_ARGUMENT), (dict(gate=3), f.ERR_INVALID_ARGUMENT),
    (dict(gate=-1), f.ERR_INVALID_ARGUMENT), (dict(E=1025), f.ERR_UNSUPPORTED),
    (dict(E=64, k=33), f.ERR_UNSUPPORTED), (dict(T=1 << 28), f.ERR_UNSUPPORTED),
    (dict(logits=None), f.ERR_INVALID_ARGUMENT), (dict(ids=None), f.ERR_INVALID_ARGUMENT),
    (dict(w=None), f.ERR_INVALID_ARGUMENT), (dict(logits=FAKE + 2), f.ERR_ALIGNMENT),
    (dict(ids=FAKE + 2), f.ERR_ALIGNMENT), (dict(w=FAKE + 2), f.ERR_ALIGNMENT),
]


@pytest.mark.parametrize("kw,want", ROUTE + [
    (dict(offsets=None), f.ERR_INVALID_ARGUMENT), (dict(order=None), f.ERR_INVALID_ARGUMENT),
    (dict(slot=None), f.ERR_INVALID_ARGUMENT), (dict(offsets=None, order=None), f.ERR_INVALID_ARGUMENT),
    (dict(offsets=FAKE + 2), f.ERR_ALIGNMENT), (dict(order=FAKE + 2), f.ERR_ALIGNMENT),
    (dict(slot=FAKE + 2), f.ERR_ALIGNMENT),
    (dict(ws=None), f.ERR_WORKSPACE), (dict(ws_bytes=8), f.ERR_WORKSPACE), (dict(ws=FAKE + 2), f.ERR_ALIGNMENT),
    (dict(T=0, offsets=None), f.OK),
])
def test_route_refusals(lib, kw, want):
    assert _route(lib, **kw) == want


@pytest.mark.parametrize("kw,want", ROUTE + [(dict(dw=None), f.ERR_INVALID_ARGUMENT),
                                             (dict(dl=None), f.ERR_INVALID_ARGUMENT), (dict(dw=FAKE + 2), f.ERR_ALIGNMENT),
                                             (dict(dl=FAKE + 2), f.ERR_ALIGNMENT), (dict(T=0), f.OK)])
def test_route_bwd_refusals(lib, kw, want):
    a = dict(logits=FAKE, t=f.OUT_F32, T=100, E=32, k=8, gate=f.GATE_SOFTMAX, ids=FAKE, w=FAKE, dw=FAKE, dl=FAKE,
             stream=None)
    a.update(kw)
    assert lib.fp8_moe_route_bwd(*a.values()) == want


@pytest.mark.parametrize("kw,want", [
    (dict(T=-1), f.ERR_INVALID_ARGUMENT), (dict(k=0), f.ERR_INVALID_ARGUMENT), (dict(E=0), f.ERR_INVALID_ARGUMENT),
    (dict(D=-16), f.ERR_INVALID_ARGUMENT), (dict(F=-16), f.ERR_INVALID_ARGUMENT),
    (dict(T=65), f.ERR_UNSUPPORTED), (dict(k=33), f.ERR_UNSUPPORTED), (dict(E=1025), f.ERR_UNSUPPORTED),
    (dict(D=1 << 20), f.ERR_UNSUPPORTED), (dict(F=1 << 20), f.ERR_UNSUPPORTED),
    (dict(D=264), f.ERR_ALIGNMENT), (dict(F=40), f.ERR_ALIGNMENT), (dict(D=272, packed=1), f.ERR_ALIGNMENT),
    (dict(F=80, packed=1), f.ERR_ALIGNMENT),
    *[({n: None}, f.ERR_INVALID_ARGUMENT) for n in ("x", "ids", "w", "w13", "i13", "w2", "i2", "out")],
    *[({n: FAKE + 8}, f.ERR_ALIGNMENT) for n in ("x", "w13", "w2", "out", "ws")],
    *[({n: FAKE + 2}, f.ERR_ALIGNMENT) for n in ("ids", "w", "i13", "i2")],
    (dict(ws=None), f.ERR_WORKSPACE), (dict(ws_bytes=2 * 4 * 2 * 128), f.ERR_WORKSPACE),
    (dict(fmt=f.E5M2_NATIVE), f.ERR_UNSUPPORTED), (dict(fmt=f.E5M2), f.ERR_UNSUPPORTED),
    (dict(T=0), f.OK), (dict(D=0), f.OK),
])
def test_few_refusals(lib, kw, want):
    a = dict(x=FAKE, ids=FAKE, w=FAKE, T=4, k=2, w13=FAKE, i13=FAKE, w2=FAKE, i2=FAKE, fmt=f.E4M3_NATIVE, E=8, D=256,
             F=128, packed=0, out=FAKE, ws=FAKE, ws_bytes=1 << 30, stream=None)
    a.update(kw)
    assert lib.fp8_moe_few(*a.values()) == want


def test_workspace_sizes(lib):
    assert f.fp8_moe_few_ws_bytes(4, 2, 128) > 2 * 4 * 2 * 128
    assert f.fp8_moe_few_ws_bytes(65, 2, 128) == 0
    assert f.fp8_moe_route_ws_bytes(64, 32, 8) == 0 and f.fp8_moe_route_ws_bytes(65, 32, 8) > 0
    assert f.fp8_moe_route_ws_bytes(-1, 32, 8) == 0
    assert f.fp8_add_norm_bwd_ws_bytes(0, 64, f.NORM_RMS) == 0
    one = f.fp8_add_norm_bwd_ws_bytes(4096, 4096, f.NORM_RMS)
    assert one > 0 and f.fp8_add_norm_bwd_ws_bytes(4096, 4096, f.NORM_LAYER) == 2 * one


class _Fake:
    """Stands in for a GPU tensor in the binding's checks (they read only these fields)."""

    def __init__(self, nbytes, dtype, device=0, contiguous=True):
        self.is_cuda, self.nbytes, self.dtype, self._d, self._c = True, nbytes, dtype, device, contiguous

    def get_device(self):
        return self._d

    def is_contiguous(self):
        return self._c


def test_binding_checks():
    b = torch.bfloat16
    assert f._args("fn", ("x", _Fake(64, b), 64, b), ("y", None, None, b), ("z", None, False, b)) == 0
    with pytest.raises(ValueError, match="required"):
        f._args("fn", ("x", None, 64, b))
    with pytest.raises(ValueError, match="needs 64"):
        f._args("fn", ("x", _Fake(62, b), 64, b))
    with pytest.raises(ValueError, match="must be torch.bfloat16"):
        f._args("fn", ("x", _Fake(64, torch.float16), 64, b))
    with pytest.raises(ValueError, match="contiguous"):
        f._args("fn", ("x", _Fake(64, b, contiguous=False), 64, b))
    with pytest.raises(ValueError, match="another GPU"):
        f._args("fn", ("x", _Fake(64, b), 64, b), ("y", _Fake(64, b, device=1), 64, b))
    x = torch.zeros(4, 64, dtype=b)
    with pytest.raises(ValueError, match="on the GPU"):
        f.fp8_add_norm_quant_row(x, x, x[0], None, f.NORM_RMS, 1e-5, f.E4M3_NATIVE, 1e-12, x, x, None, None)
    i = torch.zeros(4, 2, dtype=torch.int32)
    with pytest.raises(ValueError, match=r"\[T\]\[k\]"):
        f.fp8_moe_route(x.float(), f.GATE_SOFTMAX, i[:3], i)
    with pytest.raises(ValueError, match=r"\[E\]\[2F\]"):
        f.fp8_moe_few(x, i, i, None, torch.zeros(3, 5), None, None, f.E4M3_NATIVE, x, None)


def test_few_token_kernels_keep_the_matrix_core_rules(tmp_path):
    """The register rules that tests/test_mfma_regalloc.py checks for the GEMMs."""
    import subprocess
    out = tmp_path / "moe_few.s"
    cmd = [hb.HIPCC] + hb.COMMON + ["--cuda-device-only", "-S", os.path.join(hb.HERE, "csrc", "moe_few.hip"), "-o",
                                    str(out)]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    asm = out.read_text()
    assert "v_mfma" in asm
    assert not mfma_overlaps(asm) and not mfma_raw_hazards(asm)


def test_add_norm_row_limit_holds_for_empty_rows(lib):
    assert _norm(lib, rows=1 << 31, cols=0) == f.ERR_UNSUPPORTED
    assert _norm(lib, rows=1 << 40, cols=0, q=None, scale=None) == f.ERR_UNSUPPORTED


def test_binding_takes_codes_of_any_one_byte_type():
    """As the quantizers and the GEMMs do: codes may be in torch's float8 tensors."""
    class Codes(_Fake):
        def element_size(self):
            return self.dtype.itemsize

    for dtype in (torch.uint8, torch.float8_e4m3fn, torch.float8_e5m2):
        for first in ((), (("x", _Fake(64, torch.bfloat16), 64, torch.bfloat16),)):
            assert f._args("fn", *first, ("q", Codes(64, dtype), 64, 1)) == 0
            with pytest.raises(ValueError, match="needs 65"):
                f._args("fn", *first, ("q", Codes(64, dtype), 65, 1))
    with pytest.raises(ValueError, match=r"1-byte elements \(got torch.bfloat16\)"):
        f._args("fn", ("q", Codes(64, torch.bfloat16), 64, 1))
