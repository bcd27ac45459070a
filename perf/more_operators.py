"""The AdamW operators over many tensors on their own: the norm of all gradients
with the factor that clips them, the AdamW step with its moments in 32 bits
(with or without a 32-bit copy of 16-bit parameters), and the step with its
moments in 8 bits.

Each case is one call on a whole list of tensors.  `run` computes it tensor by
tensor in elementary torch operations (32 bits; 64 for the norm's sum and where a
code of the 8-bit moments is decided) or, with `own`, through this framework's
calls.
"""
import math

import torch

own = False

BETA1, BETA2, EPS = 0.9, 0.999, 1e-8
BLOCK = 256          # elements of a tensor that share the scales of their 8-bit moments
TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16}


def _case(name, op, gtype, layers=0, hidden=0, matrices=True, ffn=0, gated=False, rank=0, vectors=0, heads=0, vocab=0,
          packed=False, **more):
    """A list of tensors: `heads` matrices [vocab, hidden], then in each of `layers` layers, if
    rank > 0, four pairs of adapters [rank, hidden], [hidden, rank], else, with matrices,
    four [hidden, hidden] and, if ffn > 0, [ffn, hidden] (two if gated), [hidden, ffn];
    and `vectors` vectors [hidden].  packed: one behind the other in one buffer, at any element."""
    return dict(name=name, op=op, gtype=gtype, layers=layers, hidden=hidden, matrices=matrices, ffn=ffn, gated=gated, rank=rank,
                vectors=vectors, heads=heads, vocab=vocab, packed=packed, **more)


def listed():
    return [
        # gains and biases of a BERT-Base-sized model: what a call on many small tensors costs
        _case("norm 120 vectors of 768 fp32", "norm", "fp32", layers=12, hidden=768, matrices=False, vectors=10, max_norm=1.0),
        # gradients that lie in one buffer one behind the other, sides that are no multiple of anything
        _case("norm packed odd bf16", "norm", "bf16", layers=6, hidden=1001, ffn=1537, vectors=5, packed=True, max_norm=0.5),
        # every matrix of four LLaMA-2-7B-sized layers
        _case("norm 4 layers of 4096 bf16", "norm", "bf16", layers=4, hidden=4096, ffn=11008, gated=True, max_norm=1.0),
        # the vectors that stay with AdamW where the matrices have another optimizer
        _case("adamw 120 vectors of 768 fp32", "adamw", "fp32", layers=12, hidden=768, matrices=False, vectors=10,
              ptype="fp32", copy=False, clip=True, on_device=False, t=1000, lr=1e-4, wd=0.0),
        # low-rank adapters (rank 16) of q, k, v and o of 24 layers
        _case("adamw adapters 192 of 16x2048 fp32", "adamw", "bf16", layers=24, hidden=2048, rank=16,
              ptype="fp32", copy=False, clip=False, on_device=False, t=20, lr=2e-4, wd=0.0),
        # embedding and attention of a BERT-Base-sized model, clipped, count and rate on the GPU as a captured step has them
        _case("adamw embedding and 48 of 768x768 fp32", "adamw", "bf16", layers=12, hidden=768, vectors=6, heads=1, vocab=30522,
              ptype="fp32", copy=False, clip=True, on_device=True, t=300, lr=5e-5, wd=0.01),
        # odd tensors one behind the other in bf16, first step
        _case("adamw packed odd bf16", "adamw", "bf16", layers=8, hidden=777, ffn=1535, vectors=3, heads=1, vocab=5003, packed=True,
              ptype="bf16", copy=False, clip=True, on_device=False, t=1, lr=1e-3, wd=0.1),
        # two LLaMA-2-7B-sized layers in bf16 with a 32-bit copy: how such a model is pre-trained
        _case("adamw 2 layers of 4096 bf16 with copy", "adamw", "bf16", layers=2, hidden=4096, ffn=11008, gated=True, vectors=2,
              ptype="bf16", copy=True, clip=True, on_device=False, t=5000, lr=3e-4, wd=0.1),
        # the vectors of an OPT-1.3B-sized model
        _case("adamw8 240 vectors of 2048 bf16", "adamw8", "bf16", layers=24, hidden=2048, matrices=False, vectors=10,
              ptype="bf16", copy=False, clip=False, on_device=False, t=100, lr=1e-3, wd=0.0),
        # odd tensors one behind the other, fp32 gradients: short last blocks everywhere
        _case("adamw8 packed odd fp32", "adamw8", "fp32", layers=5, hidden=1001, ffn=515, vectors=4, packed=True,
              ptype="fp32", copy=False, clip=True, on_device=True, t=7, lr=1e-4, wd=0.01),
        # two OPT-1.3B-sized layers, bf16 parameters with a 32-bit copy
        _case("adamw8 2 layers of 2048 bf16 with copy", "adamw8", "bf16", layers=2, hidden=2048, ffn=8192, vectors=10,
              ptype="bf16", copy=True, clip=True, on_device=False, t=2000, lr=1e-4, wd=0.1),
        # embedding and head of a LLaMA-2-7B-sized model, the part that a matrix optimizer leaves to AdamW
        _case("adamw8 2 of 32000x4096 bf16", "adamw8", "bf16", hidden=4096, heads=2, vocab=32000,
              ptype="bf16", copy=False, clip=True, on_device=False, t=1000, lr=3e-4, wd=0.1),
    ]


def draw(rng):
    most = max(work(c)["bytes"] for c in listed())
    log = lambda lo, hi: int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))  # noqa: E731
    while True:
        kind = rng.choice(["matrices", "matrices", "adapters", "vectors"])
        case = _case("", rng.choice(["norm", "adamw", "adamw8"]), rng.choice(["fp32", "bf16"]), layers=log(1, 32),
                     hidden=log(1, 6000), matrices=kind == "matrices", ffn=rng.choice([0, log(1, 16000)]), gated=rng.random() < 0.5,
                     rank=log(1, 64) if kind == "adapters" else 0, vectors=rng.randint(kind == "vectors", 10),
                     heads=rng.randint(0, 2), vocab=log(1, 50000), packed=rng.random() < 0.5)
        del case["name"]
        if case["op"] == "norm":
            case["max_norm"] = rng.choice([0.25, 1.0, 1e3])
        else:
            case["ptype"] = rng.choice(["fp32", "bf16"])
            case["copy"] = case["ptype"] == "bf16" and rng.random() < 0.5
            case.update(clip=rng.random() < 0.5, on_device=rng.random() < 0.3, t=rng.choice([1, 2, log(3, 100000)]),
                        lr=1e-4 * log(1, 30), wd=rng.choice([0.0, 0.01, 0.1]))
        if work(case)["bytes"] <= most and _elements(case) <= 850_000_000:
            return case


def _shapes(case):
    h, out = case["hidden"], [(case["vocab"], case["hidden"])] * case["heads"]
    for _ in range(case["layers"]):
        if case["rank"]:
            out += [(case["rank"], h), (h, case["rank"])] * 4
        elif case["matrices"]:
            out += [(h, h)] * 4
            if case["ffn"]:
                out += [(case["ffn"], h)] * (2 if case["gated"] else 1) + [(h, case["ffn"])]
        out += [(h,)] * case["vectors"]
    return out


def _elements(case):
    return sum(math.prod(d) for d in _shapes(case))


def _starts(case, align):
    """Where each tensor begins in a buffer, and the buffer's length."""
    at, out = 0, []
    for shape in _shapes(case):
        out.append(at)
        at += -(-math.prod(shape) // align) * align
    return out, at


def _student(n, g):
    """Student-t with three degrees of freedom: the tails of a gradient's entries."""
    z = torch.randn(n, device="cuda", generator=g)
    chi = sum(torch.randn(n, device="cuda", generator=g).square() for _ in range(3))
    return z / (chi / 3).sqrt()


def _codes(x, top, steps):
    """Codes c >= 0 of x >= 0 (64 bits, [blocks, BLOCK]), each block's top standing for
    `steps`: c^2 / steps^2 of the top is the nearest such value to x, the larger one of two."""
    y = torch.where(top > 0, x * (steps * steps / torch.where(top > 0, top, 1.0)), 0.0)
    return (0.5 + (y - 0.25).clamp(min=0).sqrt()).floor().clamp(max=steps)


def _quantized(m, v):
    """The 8-bit form of moments in 64 bits ([blocks, BLOCK]): int8 codes of m, uint8
    codes of sqrt(v), and their fp32 scales."""
    r = v.sqrt()
    sm, sr = m.abs().amax(-1).float(), r.amax(-1).float()
    cm = _codes(m.abs(), sm.double()[:, None], 127) * m.sign()
    cv = torch.maximum(_codes(r, sr.double()[:, None], 255), (v > 0).double())
    return cm.to(torch.int8), cv.to(torch.uint8), sm, sr


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    shapes = _shapes(case)
    s = dict(case)
    align = 1 if case["packed"] else BLOCK
    starts, total = _starts(case, align)

    def views(flat):
        return [flat[a:a + math.prod(d)].view(d) for a, d in zip(starts, shapes)]

    grads = torch.zeros(total, dtype=TYPES[case["gtype"]], device="cuda")
    s["grads"] = views(grads)
    at, size = _starts(case, BLOCK)
    adamw = case["op"] != "norm"
    if adamw:
        params = torch.zeros(total, dtype=TYPES[case["ptype"]], device="cuda")
        s["flat"], s["params"] = params, views(params)
        m, v = torch.zeros(size, device="cuda"), torch.zeros(size, device="cuda")
        s["master"] = torch.zeros(size, device="cuda") if case["copy"] else None
    scales = torch.rand(len(shapes), generator=torch.Generator().manual_seed(seed)).mul(2).sub(4).tolist()
    for i, shape in enumerate(shapes):
        n, sigma = math.prod(shape), 10.0 ** scales[i]
        new = sigma * _student(n, g)
        seen = None
        if i < case["heads"]:   # rows of tokens that did not occur this time, and of some that never did
            row = torch.rand(shape[0], 1, device="cuda", generator=g)
            new = (new.view(shape) * (row < 0.5)).view(-1)
            seen = row < 0.75
        s["grads"][i].view(-1).copy_(new)
        if not adamw:
            continue
        p = 0.02 * torch.randn(n, device="cuda", generator=g)
        s["params"][i].view(-1).copy_(p)
        if case["copy"]:
            s["master"][at[i]:at[i] + n] = p
        if case["t"] > 1:       # what earlier steps left: decayed sums of gradients like this one and of their squares
            mo = sigma * math.sqrt(3 * (1 - BETA1) / (1 + BETA1)) * torch.randn(n, device="cuda", generator=g)
            vo = sigma ** 2 * 3 * (1 - BETA2 ** (case["t"] - 1)) * torch.rand(n, device="cuda", generator=g).add(0.25)
            if seen is not None:
                mo, vo = ((x.view(shape) * seen).view(-1) for x in (mo, vo))
            m[at[i]:at[i] + n], v[at[i]:at[i] + n] = mo, vo
    if not adamw:
        return s
    if case["op"] == "adamw":
        s["m"], s["v"] = m, v
    else:
        s["cm"], s["cv"] = torch.empty(size, dtype=torch.int8, device="cuda"), torch.empty(size, dtype=torch.uint8, device="cuda")
        s["sm"], s["sr"] = torch.empty(size // BLOCK, device="cuda"), torch.empty(size // BLOCK, device="cuda")
        for k in range(0, size // BLOCK, 1 << 18):
            b = slice(k, k + (1 << 18))
            e = slice(k * BLOCK, (k + (1 << 18)) * BLOCK)
            cm, cv, s["sm"][b], s["sr"][b] = _quantized(m[e].double().view(-1, BLOCK), v[e].double().view(-1, BLOCK))
            s["cm"][e], s["cv"][e] = cm.view(-1), cv.view(-1)
    s["t"] = torch.tensor([case["t"]], device="cuda") if case["on_device"] else case["t"]
    s["lr"] = torch.tensor([case["lr"]], device="cuda") if case["on_device"] else case["lr"]
    # what clipping by the norm of all gradients gives
    s["scale"] = torch.tensor([0.37 + 1e-3 * (seed % 97)], device="cuda") if case["clip"] else None
    s["at"] = at
    return s


def _plain_norm(s):
    total = sum(g.double().square().sum() for g in s["grads"])
    norm = total.sqrt()
    scale = torch.where(norm.isfinite(), (s["max_norm"] / (norm + 1e-6)).clamp(max=1.0), math.nan)
    return {"norm": norm.float(), "scale": scale.float()}


def _moved(s, p, m, v, c1, c2):
    """p after the step with moments m, v, in 32 bits."""
    u = (m * c1) / ((v.sqrt() * c2) + EPS)
    return p - s["lr"] * (u + s["wd"] * p)


def _plain(s):
    if s["op"] == "norm":
        return _plain_norm(s)
    if torch.is_tensor(s["t"]):
        c1, c2 = (1 / (1 - b ** s["t"].double()) for b in (BETA1, BETA2))
        c1, c2 = c1.float(), c2.sqrt().float()
    else:
        c1, c2 = 1 / (1 - BETA1 ** s["t"]), 1 / math.sqrt(1 - BETA2 ** s["t"])
    eight = s["op"] == "adamw8"
    for p, g, a in zip(s["params"], s["grads"], s["at"]):
        n = p.numel()
        if eight:
            nb = -(-n // BLOCK)
            e, b = slice(a, a + nb * BLOCK), slice(a // BLOCK, a // BLOCK + nb)
            x = torch.nn.functional.pad(g.reshape(-1).double(), (0, nb * BLOCK - n)).view(nb, BLOCK)
            if s["scale"] is not None:
                x = x * s["scale"].double()
            cm, cv = s["cm"][e].view(nb, BLOCK).double(), s["cv"][e].view(nb, BLOCK).double()
            mo = cm * cm.abs() * (s["sm"][b].double() / 127 ** 2)[:, None]
            ro = cv * cv * (s["sr"][b].double() / 255 ** 2)[:, None]
            m = BETA1 * mo + (1 - BETA1) * x
            v = BETA2 * ro * ro + (1 - BETA2) * x * x
            cm, cv, s["sm"][b], s["sr"][b] = _quantized(m, v)
            s["cm"][e], s["cv"][e] = cm.view(-1), cv.view(-1)
            m, v = (t.view(-1)[:n].float().view(p.shape) for t in (m, v))
        else:
            m, v = s["m"][a:a + n].view(p.shape), s["v"][a:a + n].view(p.shape)
            x = g.float()
            if s["scale"] is not None:
                x = x * s["scale"]
            m.mul_(BETA1).add_(x * (1 - BETA1))
            v.mul_(BETA2).add_(x.square() * (1 - BETA2))
        if s["master"] is not None:
            w = s["master"][a:a + n].view(p.shape)
            w.copy_(_moved(s, w, m, v, c1, c2))
            p.copy_(w)
        else:
            p.copy_(_moved(s, p.float(), m, v, c1, c2))
    out = {"params": s["flat"], "master": s["master"]}
    if not eight:
        return dict(out, m=s["m"], v=s["v"])
    cm, cv = s["cm"].view(-1, BLOCK).float(), s["cv"].view(-1, BLOCK).double()
    m = (cm * cm.abs()).double() * (s["sm"].double() / 127 ** 2)[:, None]
    v = (cv * cv * (s["sr"].double() / 255 ** 2)[:, None]).square()
    return dict(out, m=m.float().view(-1), v=v.float().view(-1), sm=s["sm"], sr=s["sr"])


def _own(s):
    from memory_compressed_adaptive_amd import adamw
    if s["op"] == "norm":
        norm, scale = adamw.grad_norm(s["grads"], s["max_norm"])
        return {"norm": norm, "scale": scale}
    kw = dict(lr=s["lr"], beta1=BETA1, beta2=BETA2, eps=EPS, wd=s["wd"], scale=s["scale"], master=s["master"])
    out = {"params": s["flat"], "master": s["master"]}
    if s["op"] == "adamw":
        adamw.adamw_step(s["params"], s["grads"], s["m"], s["v"], s["t"], **kw)
        return dict(out, m=s["m"], v=s["v"])
    adamw.adamw8_step(s["params"], s["grads"], s["cm"], s["cv"], s["sm"], s["sr"], s["t"], **kw)
    m, v = adamw.adamw8_values(s["cm"], s["cv"], s["sm"], s["sr"])
    return dict(out, m=m, v=v, sm=s["sm"], sr=s["sr"])


def run(state):
    return _own(state) if own else _plain(state)


def work(case):
    n = _elements(case)
    size = {"fp32": 4, "bf16": 2}
    if case["op"] == "norm":
        return {"bytes": n * size[case["gtype"]], "flops": 2 * n}
    each = size[case["gtype"]] + size[case["ptype"]] + (8 if case["copy"] else size[case["ptype"]])
    if case["op"] == "adamw":
        each += 16                        # both moments, read and written
    else:
        each += 4 + 16 / BLOCK + 8        # their codes and scales, and the values that they stand for
    return {"bytes": each * n, "flops": 14 * n}


def exact(case, seed):
    """The definitions in 64 bits, all tensors of a list at once where they lie."""
    s = prepare(case, seed)
    if case["op"] == "norm":
        norm = math.sqrt(math.fsum(float(torch.linalg.vector_norm(g.double())) ** 2 for g in s["grads"]))
        return {"norm": norm, "scale": min(1.0, case["max_norm"] / (norm + 1e-6))}
    t, lr = case["t"], case["lr"]
    if case["on_device"]:
        lr = float(s["lr"].double())
    factor = 1.0 if s["scale"] is None else float(s["scale"].double())
    out = {"params": torch.zeros(s["flat"].shape, dtype=torch.float64, device="cuda")}
    size = _starts(case, BLOCK)[1]
    for k in ["m", "v"] + ["master"] * case["copy"]:
        out[k] = torch.zeros(size, dtype=torch.float64, device="cuda")
    if case["op"] == "adamw8":
        out["sm"], out["sr"] = torch.zeros_like(s["sm"]).double(), torch.zeros_like(s["sr"]).double()
    base = s["flat"].data_ptr()
    for p, g, a in zip(s["params"], s["grads"], s["at"]):
        n = p.numel()
        x = g.reshape(-1).double() * factor
        if case["op"] == "adamw":
            old_m, old_v = s["m"][a:a + n].double(), s["v"][a:a + n].double()
        else:
            block = (torch.arange(n, device="cuda") + a) // BLOCK
            c, q = s["cm"][a:a + n].double(), s["cv"][a:a + n].double()
            old_m = torch.sign(c) * (c / 127) ** 2 * s["sm"].double()[block]
            old_v = ((q / 255) ** 2 * s["sr"].double()[block]) ** 2
        m = old_m + (1 - BETA1) * (x - old_m)
        v = old_v * BETA2 + x ** 2 * (1 - BETA2)
        old = s["master"][a:a + n].double() if case["copy"] else p.reshape(-1).double()
        new = old * (1 - lr * case["wd"]) - lr * (m / (1 - BETA1 ** t)) / (torch.sqrt(v / (1 - BETA2 ** t)) + EPS)
        first = (p.data_ptr() - base) // p.element_size()
        out["params"][first:first + n] = new
        if case["copy"]:
            out["master"][a:a + n] = new
        if case["op"] == "adamw":
            out["m"][a:a + n], out["v"][a:a + n] = m, v
            continue
        for key, top, x, steps in (("m", "sm", m, 127), ("v", "sr", v.sqrt(), 255)):
            peak = torch.zeros(out[top].numel(), dtype=torch.float64, device="cuda").scatter_reduce_(0, block, x.abs(), "amax").float().double()
            mine = slice(a // BLOCK, a // BLOCK + -(-n // BLOCK))
            out[top][mine] = peak[mine]
            unit = peak[block] / steps ** 2
            k = torch.floor(torch.sqrt(torch.where(unit > 0, x.abs() / unit, 0.0))).clamp(max=steps)
            up = torch.minimum(k + 1, torch.full_like(k, steps))
            near = torch.where(x.abs() - k * k * unit < up * up * unit - x.abs(), k, up)   # the nearer of two neighbours
            if key == "v":
                near = torch.where(x > 0, near.clamp(min=1), near)
            value = near * near * unit
            out[key][a:a + n] = value ** 2 if key == "v" else value * x.sign()
    return out
