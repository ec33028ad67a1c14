"""AdamW over many tensors in a few launches, with fp32 or 8-bit moments.

The optimizer of what is trained beside frozen quantized weights: adapters and
norm weights ("bitsandbytes" page: 8-bit optimizer states).  ``state_bits=8``
holds the first moment and the root of the second in e4m3 with an fp32 scale per
256 elements, rounded at random without bias (2.03 bytes of state an element;
fp32 8).  A code reaches down to 4e-6 of its block's largest value: elements
whose gradients stay below that beside their neighbours' take shorter steps than
with fp32 moments, since their root is held at the smallest code.
"""
from __future__ import annotations

from typing import Optional

import torch

from ._ops import AdamWState, nf4_adamw_step


class _Bucket:
    """Parameters of one group, device and pair of dtypes, and their moments."""

    def __init__(self, params, bits: int):
        self.params = params
        self.state = AdamWState([p.numel() for p in params], bits, params[0].device)
        self.steps = [0] * len(params)


class AdamW(torch.optim.Optimizer):
    """AdamW (decoupled weight decay) on bf16 or fp32 parameters, in place.

    A bf16 parameter is rounded to nearest after every step: with a learning
    rate far below its spacing use fp32 parameters.  Gradients may be bf16 or
    fp32 and are made contiguous where they are not.  ``seed`` drives the random
    rounding of 8-bit moments, another draw every step.
    """

    def __init__(self, params, lr: float = 1e-3, betas=(0.9, 0.999), eps: float = 1e-8, weight_decay: float = 0.01,
                 state_bits: int = 32, seed: int = 0):
        if state_bits not in (8, 32):
            raise ValueError(f"state_bits must be 8 or 32 (got {state_bits})")
        if not (lr >= 0 and eps >= 0 and weight_decay >= 0 and 0 <= betas[0] < 1 and 0 <= betas[1] < 1):
            raise ValueError("lr, eps and weight_decay must not be negative and betas lie in [0, 1)")
        super().__init__(params, dict(lr=lr, betas=betas, eps=eps, weight_decay=weight_decay))
        self.state_bits, self.seed, self.calls = state_bits, int(seed), 0
        self._buckets = [{} for _ in self.param_groups]
        for group in self.param_groups:
            self._check(group)

    def __getstate__(self):
        return {**super().__getstate__(), "state_bits": self.state_bits, "seed": self.seed, "calls": self.calls}

    def __setstate__(self, state):
        """A copy or a loaded pickle: its buckets are built anew, with the moments that came with the parameters."""
        super().__setstate__(state)
        self._buckets = [{} for _ in self.param_groups]

    def add_param_group(self, group):
        super().add_param_group(group)
        if hasattr(self, "_buckets"):
            try:
                self._check(self.param_groups[-1])
            except (TypeError, ValueError):
                self.param_groups.pop()
                raise
            self._buckets.append({})

    @staticmethod
    def _check(group):
        for p in group["params"]:
            if p.dtype not in (torch.bfloat16, torch.float32):
                raise TypeError(f"parameters must be bfloat16 or float32 (got {p.dtype})")
            if not p.is_contiguous():
                raise ValueError("parameters must be contiguous")

    def _buckets_of(self, g: int):
        """The group's buckets, by device and dtype; built at the first step (a parameter may move before it)."""
        b = self._buckets[g]
        if not b:
            lists = {}
            for p in self.param_groups[g]["params"]:
                lists.setdefault((p.device, p.dtype), []).append(p)
            for key, ps in lists.items():
                b[key] = _Bucket(ps, self.state_bits)
                for i, p in enumerate(ps):
                    self._expose(b[key], i, p)
        return b.values()

    def _expose(self, bucket: _Bucket, i: int, p):
        """The parameter's share of the flat buffers, as torch keeps optimizer state (for state_dict).

        State that is there already (in a copy of the optimizer) is taken over.
        """
        st = bucket.state
        lo, hi = st.starts[i], st.starts[i] + -(-st.sizes[i] // 256) * 256
        d = {"step": bucket.steps[i], "exp_avg": st.m[lo:hi], "exp_avg_sq": st.v[lo:hi]}
        if st.bits == 8:
            d["exp_avg_scale"], d["exp_avg_sq_scale"] = st.m_scale[lo // 256:hi // 256], st.v_scale[lo // 256:hi // 256]
        if self.state.get(p):
            self._take(bucket, i, d, self.state[p])
        self.state[p] = d

    @staticmethod
    def _take(bucket: _Bucket, i: int, d, src):
        """Copies the state `src` of a parameter into its share `d` of the buffers."""
        for k, t in d.items():
            if k == "step":
                continue
            if src[k].shape != t.shape or src[k].dtype != t.dtype:
                raise ValueError(f"saved {k} is {tuple(src[k].shape)} {src[k].dtype}, expected "
                                 f"{tuple(t.shape)} {t.dtype}")
            t.view(torch.uint8).copy_(src[k].view(torch.uint8))
        bucket.steps[i] = d["step"] = int(src["step"])

    @torch.no_grad()
    def step(self, closure=None, grad_scale: Optional[torch.Tensor] = None):
        """One step; ``grad_scale``: an fp32 device scalar that multiplies every gradient."""
        loss = None
        if closure is not None:
            with torch.enable_grad():
                loss = closure()
        self.calls += 1
        seed = (self.seed + self.calls * 0x9E3779B1) & 0xFFFFFFFF
        for g, group in enumerate(self.param_groups):
            kw = dict(lr=float(group["lr"]), beta1=group["betas"][0], beta2=group["betas"][1], eps=group["eps"],
                      weight_decay=group["weight_decay"], grad_scale=grad_scale)
            for b in self._buckets_of(g):
                # usually one call: every parameter has a gradient of one dtype and the same step count
                runs = {}
                for i, p in enumerate(b.params):
                    if p.grad is not None:
                        runs.setdefault((b.steps[i], p.grad.dtype), []).append(i)
                for (done, _), idx in runs.items():
                    ps = [b.params[i] for i in idx]
                    gs = [p.grad if p.grad.is_contiguous() and p.grad.data_ptr() % 16 == 0 else p.grad.clone(
                        memory_format=torch.contiguous_format) for p in ps]
                    st = b.state if len(idx) == len(b.params) else b.state.subset(idx)
                    nf4_adamw_step(ps, gs, st, step=done + 1, seed=seed, **kw)
                    seed = (seed + 0x51ED2701) & 0xFFFFFFFF
                    for i in idx:
                        b.steps[i] = done + 1
                        self.state[b.params[i]]["step"] = done + 1
        return loss

    def state_dict(self):
        d = super().state_dict()
        d["adamw"] = {"state_bits": self.state_bits, "seed": self.seed, "calls": self.calls}
        return d

    def load_state_dict(self, d):
        """Copies a saved state into this optimizer's buffers (same parameters, same ``state_bits``)."""
        if d.get("adamw", {}).get("state_bits") != self.state_bits:
            raise ValueError(f"the saved state is not one of this optimizer with state_bits={self.state_bits}")
        if len(d["param_groups"]) != len(self.param_groups) or any(
                len(a["params"]) != len(b["params"]) for a, b in zip(d["param_groups"], self.param_groups)):
            raise ValueError("the saved state has other parameter groups")
        self.seed, self.calls = d["adamw"]["seed"], d["adamw"]["calls"]
        for g, saved in enumerate(d["param_groups"]):
            self.param_groups[g].update({k: v for k, v in saved.items() if k != "params"})
            ids = dict(zip(map(id, self.param_groups[g]["params"]), saved["params"]))
            for b in self._buckets_of(g):
                for i, p in enumerate(b.params):
                    src = d["state"].get(ids[id(p)])
                    if src is None:      # saved before its first step
                        for k, t in self.state[p].items():
                            if k != "step":
                                t.view(torch.uint8).zero_()
                        b.steps[i] = self.state[p]["step"] = 0
                        continue
                    self._take(b, i, self.state[p], src)
