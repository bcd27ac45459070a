"""torch.optim front end: MicroAdam over ordinary parameter groups.

Each parameter group is packed into one flat device buffer (fp32, or bfloat16
when the group's parameters are bfloat16), and every parameter's storage is
replaced by a view of that buffer, so the model and the optimizer share the
memory.  At each step the group's gradients are gathered into a flat bfloat16
buffer (torch's round-to-nearest-even conversion) and one libmicroadam handle
runs the whole MicroAdam step on it (page "MicroAdam (Sparse-Gradient Adaptive
Optimization with Quantized Error Feedback)", first paragraph).  The flat order
is the order of the group's parameter list; blocks of B_d ignore tensor
boundaries.  A parameter without a gradient contributes zeros.

Muon, for the matrices of a model, stacks the equally shaped parameters of a
group in one buffer in the same way, so that one call takes all of them; a
model's other parameters go to MicroAdamW.
"""
from __future__ import annotations

import torch

from . import muon as _muon
from .optimizer import MicroAdam as _Handle


class MicroAdamW(torch.optim.Optimizer):
    """MicroAdam with decoupled weight decay.

    density: Top-k fraction (k = floor(density * d), the page's k = d/100 by
    default); m: window rows; block: B_d.  Hyperparameters are per group; lr
    may be changed between steps (param_groups[i]["lr"]).
    """

    def __init__(self, params, lr=1e-4, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.0,
                 density=0.01, m=10, block=16384, seed=42):
        defaults = dict(lr=lr, betas=betas, eps=eps, weight_decay=weight_decay, density=density,
                        m=m, block=block, seed=seed)
        super().__init__(params, defaults)
        for gi, group in enumerate(self.param_groups):
            ps = group["params"]
            if not ps:
                continue
            dev = ps[0].device
            dt = ps[0].dtype
            if dev.type != "cuda":
                raise ValueError("MicroAdamW needs CUDA (HIP) parameters")
            if any(p.device != dev or p.dtype != dt for p in ps):
                raise ValueError("the parameters of one group must share device and dtype")
            if dt not in (torch.float32, torch.bfloat16):
                raise ValueError("parameters must be float32 or bfloat16")
            d = sum(p.numel() for p in ps)
            flat = torch.empty(d, dtype=dt, device=dev)
            off = 0
            for p in ps:
                n = p.numel()
                flat[off:off + n].copy_(p.detach().reshape(-1))
                p.data = flat[off:off + n].view_as(p)
                off += n
            k = int(d * group["density"])
            b1, b2 = group["betas"]
            h = _Handle(d, block=group["block"], k=k, m=group["m"], beta1=b1, beta2=b2, eps=group["eps"],
                        lr=group["lr"], wd=group["weight_decay"], seed=group["seed"] + gi)
            group["_flat"] = flat
            group["_gflat"] = torch.empty(d, dtype=torch.bfloat16, device=dev)
            group["_handle"] = h
            group["_lr_set"] = group["lr"]

    @torch.no_grad()
    def step(self, closure=None):
        loss = None
        if closure is not None:
            with torch.enable_grad():
                loss = closure()
        for group in self.param_groups:
            if "_handle" not in group:
                continue
            h = group["_handle"]
            if group["lr"] != group["_lr_set"]:
                h.set_lr(group["lr"])
                group["_lr_set"] = group["lr"]
            gflat = group["_gflat"]
            off = 0
            for p in group["params"]:
                n = p.numel()
                if p.grad is None:
                    gflat[off:off + n].zero_()
                else:
                    gflat[off:off + n].copy_(p.grad.reshape(-1))
                off += n
            flat = group["_flat"]
            h.step(flat if flat.dtype == torch.float32 else flat.view(torch.int16), gflat.view(torch.int16))
        return loss

    def state_dict(self):
        sd = super().state_dict()
        sd["microadam"] = [g["_handle"].export_state() if "_handle" in g else None for g in self.param_groups]
        for g in sd["param_groups"]:
            for key in ("_flat", "_gflat", "_handle", "_lr_set"):
                g.pop(key, None)
        return sd

    def load_state_dict(self, state_dict):
        saved = state_dict.get("microadam", [])
        groups = [dict(g) for g in state_dict["param_groups"]]
        keep = [{k: g[k] for k in ("_flat", "_gflat", "_handle", "_lr_set") if k in g} for g in self.param_groups]
        super().load_state_dict({"state": state_dict["state"], "param_groups": groups})
        for g, extra, st in zip(self.param_groups, keep, saved):
            g.update(extra)
            if st is not None:
                g["_handle"].import_state(st)


class Muon(torch.optim.Optimizer):
    """Muon: momentum whose update is orthogonalized by Newton-Schulz products,
    with decoupled weight decay (ma_muon_step, ma_muon8_step).

    params: matrices [rows, cols], or stacks of them [n, rows, cols] that are
    orthogonalized one by one; float32 or bfloat16, on one device.  momentum_bits:
    32, or 8 for a momentum of 1 + 4/256 bytes per parameter.  scale: factor of
    the update, "rms" for 0.2 sqrt(max(rows, cols)) (one learning rate then
    serves this and MicroAdamW).  lr, weight_decay, momentum, nesterov and scale
    may be changed between steps.  A parameter without a gradient is left alone,
    its momentum too; its neighbours in a buffer then go in smaller batches, which
    can change their results by roundings.  Gradients are rounded to bfloat16, as
    MicroAdamW rounds them, into a buffer of 2 bytes per parameter that is kept
    beside the momentum, with a copy for each parameter.  The parameters are moved
    into one buffer for each shape and type here: a model is moved or converted
    before this, not after (step refuses then).
    """

    def __init__(self, params, lr=1e-3, momentum=0.95, weight_decay=0.0, nesterov=True, scale="rms", steps=5,
                 coefficients=_muon.COEFFICIENTS, eps=1e-7, momentum_bits=32):
        defaults = dict(lr=lr, momentum=momentum, weight_decay=weight_decay, nesterov=nesterov, scale=scale, steps=steps,
                        coefficients=coefficients, eps=eps, momentum_bits=momentum_bits)
        super().__init__(params, defaults)

    def add_param_group(self, param_group):
        super().add_param_group(param_group)
        group = self.param_groups[-1]
        try:
            group["_stacks"] = _stacks(group)
        except BaseException:   # memory that runs out too
            self.param_groups.pop()
            raise

    @torch.no_grad()
    def step(self, closure=None):
        loss = None
        if closure is not None:
            with torch.enable_grad():
                loss = closure()
        for st in (st for group in self.param_groups for st in group["_stacks"]):
            if any(p.data_ptr() != at for p, at in zip(st["of"], st["at"])):
                raise RuntimeError("a parameter was moved or converted after it was given to Muon, which keeps "
                                   "equally shaped ones in one buffer: make the optimizer afterwards")
        for group in self.param_groups:
            for st in group["_stacks"]:
                rows, cols = st["params"].shape[-2:]
                scale = _muon.rms_scale(rows, cols) if group["scale"] == "rms" else float(group["scale"])
                kw = dict(lr=group["lr"], beta=group["momentum"], wd=group["weight_decay"], nesterov=group["nesterov"],
                          scale=scale, steps=group["steps"], coefficients=group["coefficients"], eps=group["eps"])
                # runs of parameters that have gradients: all of them, as a rule
                n, at = len(st["of"]), 0
                while at < n:
                    end = at
                    while end < n and st["of"][end].grad is not None:
                        st["grads"][end].copy_(st["of"][end].grad)
                        end += 1
                    if end > at:
                        p, g = st["params"][at:end], st["grads"][at:end]
                        if "codes" in st:
                            _muon.muon8_step(p, g, st["codes"][at:end], st["scales"][at:end], **kw)
                        else:
                            _muon.muon_step(p, g, st["momentum"][at:end], **kw)
                        _muon.changed(*st["of"][at:end])
                    at = end + 1
        return loss

    def state_dict(self):
        """The usual dictionary, and under "muon" every stack's momentum (codes and
        scales in 8 bits) as it is."""
        sd = super().state_dict()
        sd["muon"] = [[{k: st[k].clone() for k in ("momentum", "codes", "scales") if k in st} for st in g["_stacks"]]
                      for g in self.param_groups]
        for g in sd["param_groups"]:
            g.pop("_stacks", None)
        return sd

    def load_state_dict(self, state_dict):
        saved = state_dict["muon"]
        stacks = [g["_stacks"] for g in self.param_groups]
        same = len(saved) == len(stacks) and all(
            len(a) == len(b) and all(x.keys() == {k for k in ("momentum", "codes", "scales") if k in y}
                                     and all(x[k].shape == y[k].shape and x[k].dtype == y[k].dtype for k in x)
                                     for x, y in zip(a, b)) for a, b in zip(saved, stacks))
        if not same:
            raise ValueError("the saved momentum is that of other parameters or of another momentum_bits")
        super().load_state_dict({"state": state_dict["state"], "param_groups": [dict(g) for g in state_dict["param_groups"]]})
        for g, mine, theirs in zip(self.param_groups, stacks, saved):
            g["_stacks"] = mine
            for st, new in zip(mine, theirs):
                for k, v in new.items():
                    st[k].copy_(v)


def _stacks(group):
    """The group's parameters in one buffer for each shape and type, in the order
    of the list, with their bf16 gradients and momentum beside them."""
    if group["momentum_bits"] not in (8, 32):
        raise ValueError("momentum_bits must be 32 or 8")
    if len(set(map(id, group["params"]))) < len(group["params"]):
        raise ValueError("a parameter appears twice in a group")
    by = {}
    for p in group["params"]:
        if p.dim() not in (2, 3):
            raise ValueError("Muon takes matrices [rows, cols] or stacks of them [n, rows, cols]")
        if p.device.type != "cuda":
            raise ValueError("Muon needs CUDA (HIP) parameters")
        if p.dtype not in (torch.float32, torch.bfloat16):
            raise ValueError("parameters must be float32 or bfloat16")
        if p.device != group["params"][0].device:
            raise ValueError("the parameters of one group must share a device")
        by.setdefault((tuple(p.shape), p.dtype), []).append(p)
    out = []
    for (shape, dtype), ps in by.items():
        flat = torch.empty((len(ps), *shape), dtype=dtype, device=ps[0].device)
        for i, p in enumerate(ps):
            flat[i].copy_(p.detach())
            p.data = flat[i]
        st = {"of": ps, "at": [p.data_ptr() for p in ps], "params": flat,
              "grads": torch.zeros(flat.shape, dtype=torch.bfloat16, device=flat.device)}
        if group["momentum_bits"] == 8:
            st["codes"] = torch.zeros(flat.shape, dtype=torch.int8, device=flat.device)
            st["scales"] = torch.zeros(_muon.scales_shape(flat.shape), device=flat.device)
        else:
            st["momentum"] = torch.zeros(flat.shape, dtype=torch.float32, device=flat.device)
        out.append(st)
    return out
