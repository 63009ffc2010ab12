"""optim.AdamW on the host (CPU only): states that are loaded, and what a refused call leaves."""
import copy

import pytest
import torch

import fp8_dynamic_scaling_amd as f
from fp8_dynamic_scaling_amd.optim import AdamW
from tests.test_gated_adamw_host import _adamw, lib  # noqa: F401


def _param(*shape, dtype=torch.bfloat16):
    return torch.nn.Parameter(torch.zeros(shape, dtype=dtype))


def _stepped(counts, bits=32, **kw):
    """An optimizer over vectors that have taken `counts` steps."""
    ps = [_param(40 + i) for i in range(len(counts))]
    opt = AdamW(ps, state_bits=bits, **kw)
    for p, n in zip(ps, counts):
        opt._new_state(p)
        opt.state[p]["step"] = n
    return opt


@pytest.mark.parametrize("bits", [8, 32])
@pytest.mark.parametrize("kw", [dict(capturable=True), dict(max_norm=1.0)])
def test_refused_capture_leaves_no_state(monkeypatch, bits, kw):
    p = _param(4)
    p.grad = torch.zeros_like(p)
    opt = AdamW([p], state_bits=bits, **kw)
    with monkeypatch.context() as m:
        m.setattr(torch.cuda, "is_initialized", lambda: True)
        m.setattr(torch.cuda, "is_current_stream_capturing", lambda: True)
        with pytest.raises(RuntimeError, match="take a step before"):
            opt.step()
    assert p not in opt.state
    saved = opt.state_dict()
    assert saved["state"] == {}
    AdamW([_param(4)], state_bits=bits, **kw).load_state_dict(saved)


@pytest.mark.parametrize("bits", [8, 32])
@pytest.mark.parametrize("kw", [{}, dict(max_norm=1.0)])
def test_loads_past_empty_entries(bits, kw):
    """A parameter whose entry holds nothing has no states, as one without an entry."""
    opt = _stepped([3, 3], bits)
    saved = opt.state_dict()
    saved["state"][1] = {}
    new = AdamW([_param(40), _param(41)], state_bits=bits, **kw)
    new.load_state_dict(saved)
    p, q = new.param_groups[0]["params"]
    assert int(new.state[p]["step"]) == 3 and q not in new.state


@pytest.mark.parametrize("kw", [dict(max_norm=1.0), dict(capturable=True)])
def test_refuses_counts_that_differ(kw):
    """With one count on the device two saved ones cannot both go on; without it each keeps its own."""
    saved = _stepped([100, 3]).state_dict()
    shared = AdamW([_param(40), _param(41)], **kw)
    with pytest.raises(ValueError, match="counts of steps"):
        shared.load_state_dict(copy.deepcopy(saved))
    assert not shared.state
    own = AdamW([_param(40), _param(41)])
    own.load_state_dict(saved)
    assert [own.state[p]["step"] for p in own.param_groups[0]["params"]] == [100, 3]


@pytest.mark.parametrize("bits", [8, 32])
def test_refuses_states_of_other_sizes(bits):
    saved = _stepped([1, 1], bits).state_dict()
    for name, n in (("exp_avg", 39), ("exp_avg_sq", 0)) + ((("exp_avg_scale", 1),) if bits == 8 else ()):
        bad = copy.deepcopy(saved)
        bad["state"][0][name] = bad["state"][0][name][:n]
        new = AdamW([_param(40), _param(41)], state_bits=bits)
        with pytest.raises(ValueError, match=name):
            new.load_state_dict(bad)
        assert not new.state
    del saved["state"][1]["exp_avg"]
    with pytest.raises(ValueError, match="exp_avg"):
        AdamW([_param(40), _param(41)], state_bits=bits).load_state_dict(saved)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("kw", [{}, dict(max_norm=1.0), dict(capturable=True)])
def test_loads_torchs_states(dtype, kw):
    """torch.optim.AdamW keeps moments of the parameter's shape and type and an fp32 count."""
    ps = [_param(5, 7, dtype=dtype), _param(3, dtype=dtype)]
    ref = torch.optim.AdamW(ps, lr=1e-2)
    for t in range(3):
        for p in ps:
            p.grad = torch.full_like(p, 0.01 * (t + 1))
        ref.step()
    new = AdamW([_param(5, 7, dtype=dtype), _param(3, dtype=dtype)], **kw)
    new.load_state_dict(ref.state_dict())
    steps = []
    for p, q in zip(ps, new.param_groups[0]["params"]):
        st = new.state[q]
        for k in ("exp_avg", "exp_avg_sq"):
            assert st[k].dtype == torch.float32 and torch.equal(st[k], ref.state[p][k].float().reshape(-1))
        steps.append(st["step"])
    if kw:
        assert steps[0] is steps[1] and steps[0].dtype == torch.int32 and steps[0].tolist() == [3]
    else:
        assert steps == [3, 3] and all(isinstance(s, int) for s in steps)
    assert new.param_groups[0]["lr"] == 1e-2


@pytest.mark.parametrize("other", [dict(amsgrad=True), dict(maximize=True)])
def test_refuses_torchs_variants(other):
    p = _param(4)
    p.grad = torch.ones_like(p)
    ref = torch.optim.AdamW([p], **other)
    ref.step()
    new = AdamW([_param(4)])
    with pytest.raises(ValueError, match=next(iter(other))):
        new.load_state_dict(ref.state_dict())
    assert not new.state


@pytest.mark.parametrize("bad", [dict(lr=-1.0), dict(lr=float("inf")), dict(betas=(0.9, 1.0)), dict(eps=float("nan")), dict(eps=1e-40),
                                 dict(weight_decay=-0.1), dict(lr=torch.ones(1, dtype=torch.float64)), {}])
def test_refused_step_is_not_counted(bad):
    """A value that a scheduler or the user has spoiled (or, at last, parameters that are not on the GPU) is refused
    before the count of steps moves."""
    ps = [_param(4), _param(5)]
    opt = AdamW([dict(params=ps[:1]), dict(params=ps[1:])], capturable=True)
    for p in ps:
        p.grad = torch.ones_like(p)
        opt._new_state(p)
    opt.param_groups[1].update(bad)
    with pytest.raises(ValueError):
        opt.step()
    assert int(opt.state[ps[0]]["step"]) == 0
    assert all((p == 0).all() for p in ps)


@pytest.mark.parametrize("eps,want", [(1e-40, f.ERR_INVALID_ARGUMENT), (2.0 ** -127, f.ERR_INVALID_ARGUMENT),
                                      (1e-50, f.ERR_INVALID_ARGUMENT), (2.0 ** -126, f.OK), (0.0, f.OK)])
def test_epsilon_below_fp32s_normal_numbers(lib, eps, want):  # noqa: F811
    """The reciprocal takes it for zero, so that zero gradients would make NaN of their parameters."""
    assert _adamw(lib, [], eps=eps) == want
    if want != f.OK:
        with pytest.raises(ValueError, match="eps"):
            AdamW([_param(4)], eps=eps)
