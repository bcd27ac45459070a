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
model's other parameters go to MicroAdamW or AdamW.

AdamW takes parameters of any shape where they lie, all of a group in one call, with
dense moments in 32 or 8 bits, and can clip by the norm of all gradients.
"""
from __future__ import annotations

from itertools import zip_longest

import torch

from . import adamw as _adamw
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


class AdamW(torch.optim.Optimizer):
    """AdamW over parameters where they lie, each group in one call (ma_adamw_many_step,
    ma_adamw8_many_step), optionally clipped by the norm of all gradients
    (ma_grad_norm) without waiting for it.

    params: float32 or bfloat16, dense, on one device.  state_bits: 32, or 8 for moments
    of 2 + 8/256 bytes per parameter.  master_weights: 32-bit copies of the bfloat16
    parameters, which take the steps in their place; they are made here, of the
    weights that the parameters have now.  max_norm: clips the gradients of all groups
    together to this norm; `grad_norm` is then the last step's, as a tensor on the
    GPU (a captured step's is the one that its capture left there), and a step whose
    norm is not finite changes nothing and is not counted.

    lr, betas, eps and weight_decay may be changed between steps; lr may be a
    float32 tensor of one element on the GPU, which a captured step reads at
    every replay.  A parameter without a gradient is left alone, its moments and its
    count of steps too.  Counts are kept on the GPU, one for all parameters that
    have had gradients at the same steps; these go in one call for each group.  A
    captured step goes on with the parameters and counts it was captured with; the
    parameters that share a count there have gradients together from then on, in
    other steps too, or none (RuntimeError); where several sets of them do, a step is
    taken with each before the first capture.  A step that is refused changes nothing in
    any group and is not counted.
    Gradients are float32 or bfloat16 as they are; others, and ones that lie unlike
    their parameter, are copied first.
    """

    def __init__(self, params, lr=1e-3, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.0, state_bits=32, master_weights=False,
                 max_norm=None):
        if max_norm is not None and not max_norm > 0:
            raise ValueError("max_norm must be positive")
        self.max_norm, self.grad_norm = max_norm, None
        # A count for each history of gradients, the first _histories of _counts; a group's _slots say
        # which one a parameter goes by.  A history is at least one parameter's, so that there is room
        # for all of them from the start: a captured step holds their addresses.
        self._counts, self._histories, self._begun = [], 0, False
        # The histories that a captured step goes by.
        self._captured = set()
        super().__init__(params, dict(lr=lr, betas=betas, eps=eps, weight_decay=weight_decay, state_bits=state_bits,
                                      master_weights=master_weights))

    def add_param_group(self, param_group):
        super().add_param_group(param_group)
        group = self.param_groups[-1]
        try:
            _numbers(group)
            group["_moments"] = _moments(group, next((g for g in self.param_groups if g["params"]), group))
            group["_layout"] = _adamw.layout(group["params"])
            group["_slots"] = [self._histories if self._begun else 0] * len(group["params"])
            if group["params"]:
                self._counts += torch.zeros(len(group["params"]), dtype=torch.int64, device=group["params"][0].device).split(1)
                self._histories = group["_slots"][0] + 1
        except BaseException:   # memory that runs out too
            self.param_groups.pop()
            raise

    @torch.no_grad()
    def step(self, closure=None, scale=None):
        """scale: a factor of all gradients instead of max_norm's, a float32 tensor of one
        element on the GPU (adamw.grad_norm's of more gradients than these); where it is
        NaN the step changes nothing and is not counted."""
        loss = None
        if closure is not None:
            with torch.enable_grad():
                loss = closure()
        if scale is not None and self.max_norm is not None:
            raise ValueError("a step takes scale or max_norm, not both")
        if scale is not None and not (torch.is_tensor(scale) and scale.dtype == torch.float32 and scale.numel() == 1 and scale.is_cuda):
            raise ValueError("scale must be a float32 tensor of one element on the GPU")
        for group in self.param_groups:
            if _adamw.layout(group["params"]) != group["_layout"]:
                raise RuntimeError("a parameter was moved, converted or laid out anew after it was given to AdamW, whose moments "
                                   "lie like it: make the optimizer afterwards")
            _numbers(group)
        grads = [[p.grad for p in group["params"]] for group in self.param_groups]
        none = [_adamw.missing(group["params"], gs) for group, gs in zip(self.param_groups, grads)]
        for i, (group, gs) in enumerate(zip(self.param_groups, grads)):
            if none[i] < 0:
                gs[:] = [None if g is None else _like(g, p) for g, p in zip(gs, group["params"])]
                none[i] = sum(g is None for g in gs)
        if sum(none) == sum(map(len, grads)):
            return loss
        slots = [0] if self._histories == 1 and not any(none) else self._part(grads)
        self._begun = True
        counts = [self._counts[s] for s in slots]
        norm = None
        if self.max_norm is not None:
            out = torch.empty(2, dtype=torch.float32, device=counts[0].device)
            norm, scale = out.unbind()
        # All calls are looked at before the first one is made and the step is counted: a step is
        # taken by all groups or refused.
        calls = []
        for group, gs in zip(self.param_groups, grads):
            st, (b1, b2) = group["_moments"], group["betas"]
            for slot, count in zip(slots, counts):
                some = gs if len(slots) == 1 else [g if s == slot else None for s, g in zip(group["_slots"], gs)]
                if all(g is None for g in some):
                    continue
                state = (st["cm"], st["cv"], st["sm"], st["sr"]) if "cm" in st else (st["m"], st["v"])
                calls.append(_adamw.step_call(group["params"], some, state, count, group["lr"], b1, b2, group["eps"], group["weight_decay"],
                                              scale, st.get("master"), apart=True))
        if norm is not None:
            # the norm's call counts the step where there is one count to raise
            _adamw.norm_into(out, [g for gs in grads for g in gs], self.max_norm, counts[0] if len(slots) == 1 else None)
            self.grad_norm = norm
        if norm is None or len(slots) > 1:
            taken = 1 if scale is None else (scale == scale).reshape(1)
            for count in counts:
                count.add_(taken)
        for call in calls:
            call()
        if torch.cuda.is_current_stream_capturing():
            self._captured.update(slots)
        return loss

    def _part(self, grads):
        """The histories of the parameters with gradients; those without one that shared such a history
        part from it here."""
        has, new = set(), {}
        for group, gs in zip(self.param_groups, grads):
            has.update(s for s, g in zip(group["_slots"], gs) if g is not None)
        parting = [(group["_slots"], i) for group, gs in zip(self.param_groups, grads)
                   for i, (s, g) in enumerate(zip(group["_slots"], gs)) if g is None and s in has]
        if any(slots[i] in self._captured for slots, i in parting):
            # its replays take them all, by one count
            raise RuntimeError("only some of the parameters that a captured step takes together have gradients: take a step with "
                               "each such set before the first capture or, without that captured step, go on with a new AdamW "
                               "that is loaded with this one's state_dict()")
        if parting and self._begun and torch.cuda.is_current_stream_capturing():
            # every replay would copy the count anew
            raise RuntimeError("other parameters have gradients than in the steps before: take a step with these before capturing one")
        for slots, i in parting:
            s = slots[i]
            if s not in new:
                new[s], self._histories = self._histories, self._histories + 1
                if self._begun:
                    self._counts[new[s]].copy_(self._counts[s])
            slots[i] = new[s]
        return sorted(has)

    def __getstate__(self):
        """What copy.deepcopy and pickle take: the counts too, as one tensor."""
        return {**super().__getstate__(), "max_norm": self.max_norm, "grad_norm": self.grad_norm, "_histories": self._histories,
                "_begun": self._begun, "_counts": torch.cat(self._counts) if self._counts else None}

    def __copy__(self):
        raise TypeError("a shallow copy of AdamW would step the same moments by counts of its own: use copy.deepcopy")

    def __setstate__(self, state):
        if "_counts" in state:   # (not where torch loads a state dictionary)
            counts = state["_counts"]
            state = {**state, "_counts": [] if counts is None else list(counts.split(1)), "_captured": set()}
        super().__setstate__(state)
        for g in self.param_groups:
            # unpickled onto another device, moments and all
            if "_moments" in g and all(g["_moments"].get(k) == v for k, v in _kinds(g["params"]).items()):
                g["_layout"] = _adamw.layout(g["params"])

    def state_dict(self):
        """The usual dictionary, and under "adamw" the counts and every group's moments as they are."""
        sd = super().state_dict()
        sd["adamw"] = dict(counts=[int(c) for c in self._counts[:self._histories]],
                           slots=[list(g["_slots"]) for g in self.param_groups],
                           groups=[{k: v.clone() if torch.is_tensor(v) else v for k, v in g["_moments"].items()}
                                   for g in self.param_groups])
        for g in sd["param_groups"]:
            g.pop("_moments", None)
            g.pop("_layout", None)
            g.pop("_slots", None)
        return sd

    def load_state_dict(self, state_dict):
        """Moments, copies, counts and an lr that is a tensor are written where this optimizer's lie, so
        that a captured step goes on with them."""
        saved, mine = state_dict["adamw"], [(g["_moments"], g["_layout"]) for g in self.param_groups]
        same = len(saved["groups"]) == len(mine) and all(
            a.keys() | {"types"} == b.keys() | {"types"} and [tuple(map(tuple, x)) for x in a["layout"]] == b["layout"]
            for a, (b, _) in zip(saved["groups"], mine))
        if not same:
            raise ValueError("the saved moments are those of other parameters, layouts, state_bits or master_weights")
        # Moments are the same in either type, but a copy is kept of bfloat16 parameters only.  (States were
        # saved without types at first; then they are taken to be those of the parameters now.)
        for a, (b, _) in zip(saved["groups"], mine):
            if "master" in b and any(y == "bfloat16" != x for x, y in zip(a.get("types", b["types"]), b["types"])):
                raise ValueError("a bfloat16 parameter was float32 when its state was saved, without a 32-bit copy: load into "
                                 "parameters of the types that were saved")
        if self._captured and [list(x) for x in saved["slots"]] != [g["_slots"] for g in self.param_groups]:
            raise RuntimeError("the saved parameters had gradients together that a captured step does not take together: load "
                               "into a new AdamW")
        rates, shared = [g["lr"] for g in self.param_groups], {}
        for lr, g in zip(rates, state_dict["param_groups"]):
            if torch.is_tensor(lr) and shared.setdefault(id(lr), float(g["lr"])) != float(g["lr"]):
                raise ValueError("groups share one tensor for lr, and other rates were saved for them")
        super().load_state_dict({"state": state_dict["state"], "param_groups": [dict(g) for g in state_dict["param_groups"]]})
        for g, lr in zip(self.param_groups, rates):
            if torch.is_tensor(lr):
                lr.fill_(float(g["lr"]))
                g["lr"] = lr
            elif torch.is_tensor(g["lr"]) and g["params"]:
                g["lr"] = g["lr"].to(g["params"][0].device)
        for g, (st, layout), new, slots in zip(self.param_groups, mine, saved["groups"], saved["slots"]):
            g["_moments"], g["_layout"], g["_slots"] = st, layout, list(slots)
            for k, v in new.items():
                if torch.is_tensor(v):
                    st[k].copy_(v)
        self._histories = len(saved["counts"])
        self._begun = self._histories > 1 or any(saved["counts"])
        for count, n in zip_longest(self._counts, saved["counts"], fillvalue=0):
            count.fill_(n)


def _numbers(group):
    """ValueError for a group's numbers that the steps refuse."""
    (b1, b2), lr = group["betas"], group["lr"]
    _adamw.check_numbers(0.0 if torch.is_tensor(lr) else lr, b1, b2, group["eps"], group["weight_decay"])


def _like(g, p):
    """The gradient in a type and layout that the step takes."""
    if g.is_sparse:
        raise ValueError("AdamW does not take sparse gradients")
    if _adamw.missing([p], [g]) == 0:
        return g
    dtype = g.dtype if g.dtype in (torch.float32, torch.bfloat16) else torch.float32
    return torch.empty_like(p, dtype=dtype, memory_format=torch.preserve_format).copy_(g)


def _kinds(ps):
    """What a group's state says of its parameters."""
    return {"layout": [(tuple(p.shape), p.stride()) for p in ps], "types": [str(p.dtype).replace("torch.", "") for p in ps]}


def _moments(group, first):
    """A group's moments, and the 32-bit copies of its bfloat16 parameters."""
    ps = group["params"]
    if group["state_bits"] not in (8, 32):
        raise ValueError("state_bits must be 32 or 8")
    if len(set(map(id, ps))) < len(ps):
        raise ValueError("a parameter appears twice in a group")
    for p in ps:
        if p.device.type != "cuda":
            raise ValueError("AdamW needs CUDA (HIP) parameters")
        if p.dtype not in (torch.float32, torch.bfloat16):
            raise ValueError("parameters must be float32 or bfloat16")
        if p.device != (first["params"] or ps)[0].device:
            raise ValueError("the parameters must share a device")
    st = _kinds(ps)
    if not ps:
        return st
    size, device = _adamw.state_size(ps), ps[0].device
    _adamw.require_dense(ps)
    zeros = lambda n, dtype=torch.float32: torch.zeros(n, dtype=dtype, device=device)  # noqa: E731
    if group["state_bits"] == 8:
        st.update(cm=zeros(size, torch.int8), cv=zeros(size, torch.uint8), sm=zeros(size // _adamw.BLOCK), sr=zeros(size // _adamw.BLOCK))
    else:
        st.update(m=zeros(size), v=zeros(size))
    if group["master_weights"] and any(p.dtype == torch.bfloat16 for p in ps):
        st["master"] = zeros(size)
        for view, p in zip(_adamw.views(st["master"], ps), ps):
            if p.dtype == torch.bfloat16:
                view.copy_(p.detach())
    return st
