"""AdamW over the library's multi-tensor step (fp8_adamw): states in 32 bits or as MXFP8 (8.25 bits a value), fp32
copies of bf16 parameters or stochastic rounding without them, and the clipping of the gradients' norm on the
device (fp8_grad_norm).

A step is one launch for each 48 tensors of a kind. Nothing is read back to the host.
"""
from __future__ import annotations

import math

import torch

from . import fp8_adamw, fp8_grad_norm, fp8_grad_norm_ws_bytes, load


class AdamW(torch.optim.Optimizer):
    """torch.optim.AdamW's update for bf16 and fp32 parameters.

    state_bits: 32, or 8: e4m3 codes of the first moment and of the second's square root with a power of two for
      each 32 elements.
    master_weights: keep an fp32 copy of every bf16 parameter, which is then what is updated.
    stochastic_rounding: round what is held in few bits (8-bit states, bf16 parameters without a copy) up or down
      by chance, right in the mean: to nearest, a step smaller than half the last place is lost. The bits are a hash
      of seed, step and place: a run can be repeated.
    max_norm: clip the gradients of all groups together to this 2-norm (float("inf"): do not clip). The norm is left
      in grad_norm, a tensor of one element. If it is not finite, the step changes nothing and is not counted.
      step(grad_scale=s) multiplies the gradients by s first, to undo a loss scale.
    capturable: count steps on the device, so that step() can be captured into a graph. A captured step keeps the
      rate it was captured with unless lr is an fp32 tensor of one element on the device. The states have to be
      there: one step is taken before.

    With max_norm or capturable all parameters are on one device and share one count of steps. Parameters must be
    contiguous; a gradient that is not is copied.
    """

    def __init__(self, params, lr=1e-3, betas=(0.9, 0.999), eps: float = 1e-8, weight_decay: float = 1e-2, *,
                 state_bits: int = 32, master_weights: bool = False, stochastic_rounding: bool = True, seed: int = 1,
                 max_norm: float | None = None, capturable: bool = False):
        if state_bits not in (8, 32):
            raise ValueError(f"state_bits must be 8 or 32 (got {state_bits})")
        if not isinstance(lr, torch.Tensor) and not lr >= 0:
            raise ValueError(f"lr must not be negative (got {lr})")
        if isinstance(lr, torch.Tensor) and not capturable:
            raise ValueError("lr may be a tensor only with capturable=True")
        if len(betas) != 2 or not all(0 <= b < 1 for b in betas):
            raise ValueError(f"betas must be two numbers in [0, 1) (got {betas})")
        if not eps >= 0 or not weight_decay >= 0:
            raise ValueError("eps and weight_decay must not be negative")
        if 0 < eps < 2.0 ** -126:
            raise ValueError(f"eps must be 0 or a normal fp32 number (got {eps})")
        if max_norm is not None and not max_norm > 0:
            raise ValueError(f"max_norm must be positive (got {max_norm})")
        if not 0 < seed < 1 << 63:
            raise ValueError("seed must be positive")
        self.state_bits, self.master_weights, self.capturable = state_bits, master_weights, capturable
        self.seed, self.max_norm = (seed if stochastic_rounding else 0), max_norm
        self.grad_norm = self._mul = None
        super().__init__(params, dict(lr=lr, betas=tuple(betas), eps=eps, weight_decay=weight_decay))

    def add_param_group(self, group):
        super().add_param_group(group)
        error = None
        for p in self.param_groups[-1]["params"]:
            if p.dtype not in (torch.bfloat16, torch.float32):
                error = TypeError(f"AdamW: parameters must be bfloat16 or float32 (got {p.dtype})")
            elif not p.is_contiguous():
                error = ValueError("AdamW: parameters must be contiguous")
        if error is not None:
            self.param_groups.pop()
            raise error

    def __getstate__(self):  # the base class keeps its own three attributes only
        own = ("state_bits", "master_weights", "capturable", "seed", "max_norm", "grad_norm", "_mul")
        return {**super().__getstate__(), **{k: getattr(self, k) for k in own}}

    @property
    def _counts_on_device(self) -> bool:
        return self.capturable or self.max_norm is not None

    def _new_state(self, p):
        st, dev = self.state[p], p.device
        n = p.numel()
        if self.state_bits == 8:
            for k in ("exp_avg", "exp_avg_sq"):
                st[k] = torch.zeros(n, dtype=torch.uint8, device=dev)
                st[k + "_scale"] = torch.zeros(-(-n // 32), dtype=torch.uint8, device=dev)
        else:
            for k in ("exp_avg", "exp_avg_sq"):
                st[k] = torch.zeros(n, dtype=torch.float32, device=dev)
        if self.master_weights and p.dtype == torch.bfloat16:
            st["master"] = p.detach().float().reshape(-1)
        if self._counts_on_device:
            shared = next((s["step"] for q, s in self.state.items() if "step" in s), None)
            st["step"] = torch.zeros(1, dtype=torch.int32, device=dev) if shared is None else shared
        else:
            st["step"] = 0

    def load_state_dict(self, state_dict):
        """States of this optimizer or, with state_bits=32, of torch.optim.AdamW. What is refused changes nothing."""
        states = state_dict["state"]
        if any(s and ("exp_avg_scale" in s) != (self.state_bits == 8) for s in states.values()):
            raise ValueError(f"AdamW: states of another kind than state_bits={self.state_bits}")
        for variant in ("amsgrad", "maximize"):
            if any(g.get(variant) for g in state_dict["param_groups"]):
                raise ValueError(f"AdamW: the states of a run with {variant} cannot go on without it")
        old = [i for g in state_dict["param_groups"] for i in g["params"]]
        new = [p for g in self.param_groups for p in g["params"]]
        for i, p in zip(old, new):
            if states.get(i):
                self._check_state(states[i], p.numel())
        counts = {int(s["step"]) for s in states.values() if s}
        if self._counts_on_device and len(counts) > 1:
            raise ValueError("AdamW: max_norm and capturable share one count of steps, the saved counts of steps are "
                             f"{sorted(counts)}")
        super().load_state_dict(state_dict)
        # the base class casts states to the parameter's type, which would round moments and spoil codes
        step = None
        for i, p in zip(old, new):
            if not states.get(i):  # no entry, or one that holds nothing
                self.state.pop(p, None)
                continue
            st = self.state[p] = {}
            for k, v in states[i].items():
                if torch.is_tensor(v) and k != "step":
                    v = v.detach().to(p.device, copy=True)
                    # torch.optim.AdamW's moments have the parameter's shape and type
                    if k == "master" or (k in ("exp_avg", "exp_avg_sq") and self.state_bits == 32):
                        v = v.float().reshape(-1)
                st[k] = v
            if self.master_weights and p.dtype == torch.bfloat16 and "master" not in st:
                st["master"] = p.detach().float().reshape(-1)
            st["step"] = int(st["step"])
            if self._counts_on_device:  # one count for all
                if step is None:
                    step = torch.full((1,), st["step"], dtype=torch.int32, device=p.device)
                st["step"] = step

    def _check_state(self, st, n):
        eight = self.state_bits == 8
        sizes = {"exp_avg": n, "exp_avg_sq": n, "step": 1}
        if eight:
            sizes.update(exp_avg_scale=-(-n // 32), exp_avg_sq_scale=-(-n // 32))
        if "master" in st:
            sizes["master"] = n
        for k, want in sizes.items():
            v = st.get(k)
            got = v.numel() if torch.is_tensor(v) else 1 if k == "step" and v is not None else None
            if got != want:
                raise ValueError(f"AdamW: a saved {k} has {got or 'no'} elements where {want} are wanted")
            if eight and k not in ("step", "master") and v.dtype.itemsize != 1:
                raise ValueError(f"AdamW: a saved {k} is {v.dtype} where codes are wanted")

    @staticmethod
    def _check_group(group, dev):
        lr = group["lr"]
        if isinstance(lr, torch.Tensor):
            if lr.device != dev or lr.dtype != torch.float32:
                raise ValueError("AdamW: a tensor lr must be float32 and on the parameters' device")
            lr = 0.0
        if not all(0 <= x < math.inf for x in (lr, group["eps"], group["weight_decay"])):
            raise ValueError("AdamW: lr, eps and weight_decay must be finite and not negative")
        if 0 < group["eps"] < 2.0 ** -126:
            raise ValueError(f"AdamW: eps must be 0 or a normal fp32 number (got {group['eps']})")
        if not all(0 <= b < 1 for b in group["betas"]):
            raise ValueError(f"AdamW: betas must be in [0, 1) (got {group['betas']})")
        if dev.type != "cuda":
            raise ValueError(f"AdamW: parameters must be on the GPU (got {dev})")

    @torch.no_grad()
    def step(self, closure=None, grad_scale: float = 1.0):
        loss = None
        if closure is not None:
            with torch.enable_grad():
                loss = closure()
        load()
        if grad_scale != 1.0 and self.max_norm is None:
            raise ValueError("AdamW: grad_scale needs max_norm (infinity for no clipping)")
        capturing = torch.cuda.is_initialized() and torch.cuda.is_current_stream_capturing()
        if capturing and not self._counts_on_device:
            raise RuntimeError("AdamW: a step is captured only with capturable=True: the graph would keep its number")
        work, grads = {}, []
        for gi, group in enumerate(self.param_groups):
            for p in group["params"]:
                if p.grad is None:
                    continue
                if p.grad.is_sparse:
                    raise RuntimeError("AdamW: sparse gradients are not supported")
                if "exp_avg" not in self.state.get(p, ()):  # reading self.state[p] would make an entry
                    if capturing:  # each replay would begin with states of zero
                        raise RuntimeError("AdamW: take a step before the captured one, which cannot make states")
                    self._new_state(p)
                st, g = self.state[p], p.grad if p.grad.is_contiguous() else p.grad.contiguous()
                grads.append(g)
                t = None if self._counts_on_device else st["step"] + 1
                work.setdefault((gi, p.device, p.dtype, g.dtype, "master" in st, t), []).append((p, g, st))
        if not work:
            return loss
        for gi, dev, *_ in work:  # before the count moves or a part of the parameters
            self._check_group(self.param_groups[gi], dev)
        mul = step_dev = None
        if self._counts_on_device:
            devices = {k[1] for k in work}
            if len(devices) > 1:
                raise RuntimeError("AdamW: max_norm and capturable need all parameters on one device")
            dev = devices.pop()
            step_dev = next(iter(work.values()))[0][2]["step"]
            if self.max_norm is None:
                step_dev.add_(1)
            else:
                need = fp8_grad_norm_ws_bytes(grads)
                if self._mul is None or self._mul.device != dev:
                    self._mul, self.grad_norm = torch.empty(1, device=dev), torch.empty(1, device=dev)
                # a workspace of this step's own: steps on other streams and captured ones do not share it
                ws = torch.empty(max(8, need), dtype=torch.uint8, device=dev)
                mul = self._mul
                fp8_grad_norm(grads, self.grad_norm, mul, ws, grad_scale=grad_scale, max_norm=self.max_norm,
                              step=step_dev)
        for at, ((gi, dev, _, _, master, t), items) in enumerate(work.items()):
            group = self.param_groups[gi]
            lr, (b1, b2) = group["lr"], group["betas"]
            on_dev = isinstance(lr, torch.Tensor)
            col = lambda k: [st[k] for _, _, st in items]  # noqa: E731
            scales = self.state_bits == 8
            # another seed for each call of a step: tensors of two calls have the same places
            seed = (self.seed + at * 0x9E3779B97F4A7C15) % (1 << 64) if self.seed else 0
            fp8_adamw([p for p, _, _ in items], [g for _, g, _ in items], col("exp_avg"), col("exp_avg_sq"),
                      0.0 if on_dev else lr, b1, b2, group["eps"], group["weight_decay"], t or 1,
                      exp_avg_scales=col("exp_avg_scale") if scales else None,
                      exp_avg_sq_scales=col("exp_avg_sq_scale") if scales else None,
                      masters=col("master") if master else None, seed=seed, grad_mul=mul, step_dev=step_dev,
                      lr_dev=lr if on_dev else None)
            if t is not None:
                for _, _, st in items:
                    st["step"] = t
            torch.autograd.graph.increment_version([p for p, _, _ in items])
        return loss
