"""torch_optim.AdamW: its steps are those of the operators on the same lists, alone and
beside Muon and MicroAdamW, clipped and not, captured and not, and its state round-trips."""
import copy
import math
import pickle

import pytest
import torch

from gpu_harness import say
from memory_compressed_adaptive_amd import adamw
from memory_compressed_adaptive_amd.torch_optim import AdamW, MicroAdamW, Muon

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


SHAPES = [(40, 70), (1,), (300,), (3, 20, 90), (513,)]


def _params(seed, dtypes=(F32,)):
    g = torch.Generator().manual_seed(seed)
    return [torch.nn.Parameter((0.02 * torch.randn(s, generator=g)).to(dtypes[i % len(dtypes)]).cuda()) for i, s in enumerate(SHAPES)]


def _grads(seed):
    g = torch.Generator().manual_seed(seed)
    return [1e-3 * torch.randn(s, generator=g).cuda() for s in SHAPES]


class Own:
    """The operators on a list of their own."""

    def __init__(self, ps, bits, copies):
        self.ps, n = [p.detach().clone() for p in ps], adamw.state_size(ps)
        self.master = None
        if copies and any(p.dtype == BF16 for p in ps):
            self.master = torch.zeros(n, device="cuda")
            for v, p in zip(adamw.views(self.master, self.ps), self.ps):
                v.copy_(p)
        if bits == 32:
            self.fn, self.state = adamw.adamw_step, [torch.zeros(n, device="cuda") for _ in range(2)]
        else:
            self.fn = adamw.adamw8_step
            self.state = [torch.zeros(n, dtype=d, device="cuda") for d in (torch.int8, torch.uint8)]
            self.state += [torch.zeros(n // 256, device="cuda") for _ in range(2)]

    def step(self, gs, t, **kw):
        self.fn(self.ps, gs, *self.state, t, master=self.master, **kw)

    def same(self, ps):
        return all(torch.equal(a, b) for a, b in zip(self.ps, ps))


@pytest.mark.parametrize("dtypes,copies", [((F32,), False), ((BF16,), False), ((BF16, F32), True)])
@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("max_norm", [None, 1e-2])
def test_steps_are_the_operators(dtypes, copies, bits, max_norm):
    ps = _params(1, dtypes)
    own = [Own(ps[:2], bits, copies), Own(ps[2:], bits, copies)]
    opt = AdamW([{"params": ps[:2]}, {"params": ps[2:], "weight_decay": 0.0}], lr=0.01, betas=(0.8, 0.99), weight_decay=0.1,
                state_bits=bits, master_weights=copies, max_norm=max_norm)
    lr, counts = 0.01, [0] * len(ps)
    for t in range(1, 6):
        gs = [g.to(p.dtype) for g, p in zip(_grads(10 + t), ps)]
        for i, (p, g) in enumerate(zip(ps, gs)):
            p.grad = None if (t, i) in ((2, 0), (3, 3)) else g
        if t == 4:
            lr = 0.003
            for group in opt.param_groups:
                group["lr"] = lr
        say(f"[torch adamw] step {t} {dtypes} bits={bits} max_norm={max_norm}")
        opt.step()
        scale = None
        if max_norm is not None:
            norm, scale = adamw.grad_norm([p.grad for p in ps], max_norm)
            assert float(norm) == float(opt.grad_norm) and float(scale) < 1
        counts = [k + (p.grad is not None) for k, p in zip(counts, ps)]
        for k in sorted(set(counts)):
            some = [p.grad if c == k else None for c, p in zip(counts, ps)]
            count = torch.tensor([k], device="cuda")
            own[0].step(some[:2], count, lr=lr, beta1=0.8, beta2=0.99, wd=0.1, scale=scale)
            own[1].step(some[2:], count, lr=lr, beta1=0.8, beta2=0.99, wd=0.0, scale=scale)
        assert own[0].same(ps[:2]) and own[1].same(ps[2:]), t


def test_32_bits_are_torchs_adamw():
    """Both differ from the formula by roundings: a few parts in 10^7 of lr a step, and of the parameter."""
    ps, qs = _params(2), _params(2)
    a, b = AdamW(ps, lr=1e-2, weight_decay=0.1), torch.optim.AdamW(qs, lr=1e-2, weight_decay=0.1)
    for t in range(20):
        for p, q, g in zip(ps, qs, _grads(40 + t)):
            p.grad, q.grad = g, g.clone()
        a.step(), b.step()
        for p, q in zip(ps, qs):
            assert bool(((p - q).abs() <= (t + 1) * (1e-2 * 40 * 2.0 ** -24 + 4 * 2.0 ** -24 * q.abs())).all()), t


def test_parameters_that_join_later_are_torchs_adamw():
    """The first step of a parameter is corrected as a first step, whenever it comes."""
    ps, qs = _params(12), _params(12)
    a, b = AdamW([{"params": ps[:2]}, {"params": ps[2:]}], lr=1e-2), torch.optim.AdamW(qs, lr=1e-2, weight_decay=0.0)
    for t in range(12):
        for i, (p, q, g) in enumerate(zip(ps, qs, _grads(60 + t))):
            p.grad, q.grad = (None, None) if t < 3 * i or (i == 0 and t % 5 == 4) else (g, g.clone())
        a.step(), b.step()
        for p, q in zip(ps, qs):
            assert bool(((p - q).abs() <= (t + 1) * (1e-2 * 40 * 2.0 ** -24 + 4 * 2.0 ** -24 * q.abs())).all()), t
    assert sorted(a.state_dict()["adamw"]["counts"]) == sorted({int(b.state[q].get("step", 0)) for q in qs})


def test_a_captured_step_of_some_parameters():
    ps, qs = _params(13), _params(13)
    a, b = AdamW(ps, lr=1e-2, max_norm=1.0), AdamW(qs, lr=1e-2, max_norm=1.0)

    def grads(t, but=None):
        for i, (p, q, g) in enumerate(zip(ps, qs, _grads(70 + t))):
            if i == but:
                p.grad = q.grad = None
            elif p.grad is None:
                p.grad, q.grad = g, g.clone()
            else:
                p.grad.copy_(g), q.grad.copy_(g)

    grads(0), a.step(), b.step()
    grads(1, but=1)
    a.step(), b.step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a.step()
    for t in range(2, 5):
        grads(t, but=1)
        graph.replay()
        b.step()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(ps, qs)), t
    grads(5), a.step(), b.step()
    assert all(torch.equal(p, q) for p, q in zip(ps, qs))
    assert a.state_dict()["adamw"]["counts"] == b.state_dict()["adamw"]["counts"] == [6, 2]


@pytest.mark.parametrize("value", [math.inf, math.nan])
@pytest.mark.parametrize("how", ["max_norm", "scale"])
def test_a_step_that_is_not_finite_is_not_taken(value, how):
    ps, qs = _params(3), _params(3)
    kw = dict(max_norm=1.0) if how == "max_norm" else {}
    a, b = AdamW(ps, lr=1e-2, **kw), AdamW(qs, lr=1e-2, **kw)
    for t in range(3):
        for p, q, g in zip(ps, qs, _grads(50 + t)):
            p.grad, q.grad = g, g.clone()
        if t == 1:
            ps[2].grad[7] = value
            before = [p.detach().clone() for p in ps]
        step = (lambda o, xs: o.step()) if how == "max_norm" else \
            (lambda o, xs: o.step(scale=adamw.grad_norm([x.grad for x in xs], 1.0)[1]))
        step(a, ps)
        if t == 1:
            assert all(torch.equal(p, x) for p, x in zip(ps, before))
        else:
            step(b, qs)
    assert all(torch.equal(p, q) for p, q in zip(ps, qs)) and a.state_dict()["adamw"]["counts"] == [2]


@pytest.mark.parametrize("bits,copies", [(32, False), (32, True), (8, True)])
def test_state_dict_resume(bits, copies, tmp_path):
    def run(split):
        ps = _params(5, (BF16, F32))
        opt = AdamW(ps, lr=0.01, state_bits=bits, master_weights=copies, max_norm=1e-2)
        for t in range(6):
            if t == split:
                torch.save(opt.state_dict(), tmp_path / "state")
                sd = torch.load(tmp_path / "state", weights_only=True)
                ps2 = _params(6, (BF16, F32))
                for a, b in zip(ps2, ps):
                    a.data.copy_(b.data)
                opt = AdamW(ps2, lr=0.5, state_bits=bits, master_weights=copies, max_norm=1e-2)
                opt.load_state_dict(sd)
                assert opt.param_groups[0]["lr"] == 0.01
                ps = ps2
            for p, g in zip(ps, _grads(20 + t)):
                p.grad = g.to(p.dtype)
            opt.step()
        return ps

    for a, b in zip(run(3), run(-1)):
        assert torch.equal(a, b)


def test_load_refuses_other_moments():
    a = AdamW(_params(1, (BF16,)))
    for kw, ps in ((dict(state_bits=8), _params(1, (BF16,))), (dict(master_weights=True), _params(1, (BF16,))), ({}, _params(1)[:2])):
        with pytest.raises(ValueError, match="saved moments"):
            AdamW(ps, **kw).load_state_dict(a.state_dict())
    turned = [torch.nn.Parameter(p.detach().t().clone(memory_format=torch.contiguous_format).t()) if p.dim() == 2 else p for p in _params(1, (BF16,))]
    with pytest.raises(ValueError, match="saved moments"):
        AdamW(turned).load_state_dict(a.state_dict())


def test_step_refuses_parameters_that_were_converted():
    ps = _params(9)
    opt = AdamW(ps)
    for p, g in zip(ps, _grads(9)):
        p.grad = g
    before = ps[1].detach().clone()
    ps[0].data = ps[0].data.t().contiguous().t()
    with pytest.raises(RuntimeError, match="laid out anew"):
        opt.step()
    assert torch.equal(ps[1].detach(), before)
    ps[0].data = ps[0].data.contiguous().clone()   # elsewhere, but lying the same: taken
    opt.step()
    assert not torch.equal(ps[1].detach(), before)


def test_gradients_of_other_layouts():
    w = torch.nn.Parameter(torch.randn(30, 20, device="cuda").t())
    q = torch.nn.Parameter(w.detach().contiguous())
    a, b = AdamW([w]), AdamW([q])
    for g in (torch.randn(20, 30, device="cuda"), torch.randn(30, 20, device="cuda").t(), torch.ones(20, 1, device="cuda").expand(20, 30)):
        w.grad, q.grad = g, g
        a.step(), b.step()
        assert torch.equal(w, q)


@pytest.mark.parametrize("bits", [32, 8])
def test_a_captured_step_replays_as_eager_ones(bits):
    ps, qs = _params(7, (BF16, F32)), _params(7, (BF16, F32))
    lr = [torch.full((1,), 0.01, device="cuda") for _ in range(2)]
    for p, q, g in zip(ps, qs, _grads(7)):
        p.grad, q.grad = g.to(p.dtype), g.to(p.dtype)
    kw = dict(weight_decay=0.1, state_bits=bits, master_weights=True, max_norm=1e-2)
    captured, eager = AdamW(ps, lr=lr[0], **kw), AdamW(qs, lr=lr[1], **kw)
    adamw.grad_norm([p.grad for p in ps])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured.step()
    for t in range(5):
        for p, q, g in zip(ps, qs, _grads(30 + t)):
            p.grad.copy_(g)
            q.grad.copy_(g)
        for x in lr:
            x.fill_(0.01 / (t + 1))
        graph.replay()
        eager.step()
        torch.cuda.synchronize()
        assert float(captured.grad_norm) == float(eager.grad_norm)
        assert all(torch.equal(p, q) for p, q in zip(ps, qs)), t


def test_a_model_trained_by_three_optimizers():
    """Matrices to Muon, the embedding to AdamW in 8 bits, vectors to MicroAdamW, all clipped by
    one norm, as a user sets them up; AdamW's update is checked against the operators."""
    torch.manual_seed(0)
    emb = torch.nn.Embedding(300, 48).cuda()
    model = torch.nn.Sequential(torch.nn.Linear(48, 96), torch.nn.Tanh(), torch.nn.Linear(96, 8)).cuda()
    matrices = [p for p in model.parameters() if p.dim() == 2]
    vectors = [p for p in model.parameters() if p.dim() == 1]
    every = [emb.weight, *matrices, *vectors]
    ad = AdamW([emb.weight], lr=1e-2, state_bits=8)
    opts = [Muon(matrices, lr=1e-2), MicroAdamW(vectors, lr=1e-3, density=0.05, m=4, block=64)]
    own = Own([emb.weight], 8, False)
    x, y = torch.randint(0, 150, (64,), device="cuda"), torch.randn(64, 8, device="cuda")
    unseen = emb.weight[150:].detach().clone()
    for t in range(1, 5):
        for p in every:
            p.grad = None
        torch.nn.functional.mse_loss(model(emb(x)), y).backward()
        norm, scale = adamw.grad_norm([p.grad for p in every], 0.05)
        assert float(scale) < 1
        own.step([emb.weight.grad], torch.tensor([t], device="cuda"), lr=1e-2, scale=scale)
        ad.step(scale=scale)
        for p in matrices + vectors:
            p.grad.mul_(scale)
        for o in opts:
            o.step()
        assert own.same([emb.weight]) and all(bool(p.isfinite().all()) for p in every)
    assert torch.equal(emb.weight[150:].detach(), unseen)


def test_added_group_and_refusals():
    ps = _params(1)
    opt = AdamW(ps[:2])
    opt.add_param_group({"params": ps[2:], "lr": 0.02, "state_bits": 8})
    for p, g in zip(ps, _grads(1)):
        p.grad = g
    before = [p.detach().clone() for p in ps]
    opt.step()
    assert all(not torch.equal(p, q) for p, q in zip(ps, before))
    with pytest.raises(ValueError, match="float32 or bfloat16"):
        opt.add_param_group({"params": [torch.nn.Parameter(torch.zeros(4, 4, dtype=torch.float16, device="cuda"))]})
    with pytest.raises(ValueError, match="dense"):
        opt.add_param_group({"params": [torch.nn.Parameter(torch.zeros(4, 4, device="cuda")[:, ::2])]})
    assert len(opt.param_groups) == 2
    with pytest.raises(ValueError, match="not both"):
        AdamW(_params(1), max_norm=1.0).step(scale=torch.ones(1, device="cuda"))
    for scale in (0.5, torch.ones(1), torch.ones(2, device="cuda"), torch.ones(1, device="cuda", dtype=torch.float64)):
        with pytest.raises(ValueError, match="scale"):
            opt.step(scale=scale)
    assert opt.state_dict()["adamw"]["counts"] == [1]
    opt.step()
    loss = opt.step(lambda: torch.tensor(3.0))
    assert float(loss) == 3.0


def test_a_kept_graph_is_not_used_with_new_parameters():
    torch.manual_seed(0)
    w, still = (torch.nn.Parameter(torch.randn(40, 40, device="cuda")) for _ in range(2))
    x = torch.randn(8, 40, device="cuda", requires_grad=True)
    opt = AdamW([w, still])
    first, second = (x @ w).sum(), (x @ still).sum()
    first.backward(retain_graph=True)
    opt.step()
    second.backward(retain_graph=True)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        first.backward()
    still.grad = None
    (x @ w).sum().backward()


@pytest.mark.parametrize("bits,max_norm", [(32, None), (32, 1e-2), (8, None), (8, 1e-2)])
def test_a_refused_step_changes_nothing(bits, max_norm):
    """Put right and taken again it is the step that it would have been."""
    ps, qs = _params(15), _params(15)
    kw = dict(lr=1e-2, state_bits=bits, max_norm=max_norm)
    a, b = (AdamW([{"params": x[:2]}, {"params": x[2:]}], **kw) for x in (ps, qs))
    bad = [dict(eps=0.0), dict(betas=(0.9, 1.0)), dict(weight_decay=-0.1), dict(lr=torch.ones(1)), dict(lr=math.nan),
           dict(lr=torch.ones(1, dtype=torch.float64, device="cuda")), dict(lr=torch.ones(2, device="cuda"))]

    def everything():
        return [x.clone() for x in ps] + [v.clone() for g in a.param_groups for v in g["_moments"].values() if torch.is_tensor(v)]

    for t, wrong in enumerate(bad):
        for p, q, g in zip(ps, qs, _grads(80 + t)):
            p.grad, q.grad = g, g.clone()
        before, counts = everything(), a.state_dict()["adamw"]["counts"]
        group = a.param_groups[1]
        kept = {k: group[k] for k in wrong}
        group.update(wrong)
        with pytest.raises(ValueError):
            a.step()
        assert all(torch.equal(x, y) for x, y in zip(before, everything())) and a.state_dict()["adamw"]["counts"] == counts
        group.update(kept)
        own, ps[4].data = ps[4].data, ps[3].data.view(-1)[7:520]
        with pytest.raises(ValueError, match="overlap"):
            a.step()
        ps[4].data = own
        with pytest.raises(ValueError):
            a.step(scale=torch.ones(1)) if max_norm is None else a.step(scale=torch.ones(1, device="cuda"))
        assert all(torch.equal(x, y) for x, y in zip(before, everything())) and a.state_dict()["adamw"]["counts"] == counts
        a.step(), b.step()
        assert all(torch.equal(p, q) for p, q in zip(ps, qs)), t
    where = ps[0].data
    ps[0].data = where.cpu()
    with pytest.raises(RuntimeError, match="moved"):
        a.step()
    ps[0].data = where
    assert a.state_dict()["adamw"]["counts"] == [len(bad)]


@pytest.mark.parametrize("how", ["deepcopy", "pickle"])
@pytest.mark.parametrize("bits,copies", [(32, False), (8, True)])
def test_a_copy_goes_on_as_the_original(how, bits, copies):
    ps = _params(16, (BF16, F32))
    ps[0] = torch.nn.Parameter(ps[0].detach().t().contiguous().t())      # a dense layout of its own
    a = AdamW([{"params": ps[:2]}, {"params": ps[2:]}], lr=1e-2, state_bits=bits, master_weights=copies, max_norm=1e-2)

    def step(opt, t, but=None):
        flat = [p for g in opt.param_groups for p in g["params"]]
        for i, (p, g) in enumerate(zip(flat, _grads(90 + t))):
            p.grad = None if i == but else g.to(p.dtype)
        opt.step()
        return flat

    step(a, 0), step(a, 1, but=3)
    b = copy.deepcopy(a) if how == "deepcopy" else pickle.loads(pickle.dumps(a))
    norm = float(a.grad_norm)
    assert float(b.grad_norm) == norm
    for t in range(2, 5):
        xs, ys = step(a, t), step(b, t)
        assert all(torch.equal(x, y) and x.data_ptr() != y.data_ptr() for x, y in zip(xs, ys)), t
        assert float(a.grad_norm) == float(b.grad_norm) != norm
    before = [x.clone() for x in ys]
    step(a, 5)
    assert all(torch.equal(x, y) for x, y in zip(before, ys))
    assert a.state_dict()["adamw"]["counts"] == [6, 5] and b.state_dict()["adamw"]["counts"] == [5, 4]


@pytest.mark.parametrize("bits", [32, 8])
def test_load_with_copies_goes_by_the_types_saved(bits):
    """A parameter of 32 bits has no copy that a 16-bit one could go on from."""
    def make(seed, dtypes):
        return AdamW(_params(seed, dtypes), lr=1e-2, state_bits=bits, master_weights=True)

    a = make(17, (BF16, F32))
    for p, g in zip(a.param_groups[0]["params"], _grads(17)):
        p.grad = g.to(p.dtype)
    a.step()
    with pytest.raises(ValueError, match="32-bit copy"):
        make(18, (BF16,)).load_state_dict(a.state_dict())
    b = make(18, (BF16, F32))
    b.load_state_dict(a.state_dict())
    for x, y in zip(a.param_groups[0]["params"], b.param_groups[0]["params"]):
        y.data.copy_(x.data)
        y.grad = x.grad.clone()
    a.step(), b.step()
    assert all(torch.equal(x, y) for x, y in zip(a.param_groups[0]["params"], b.param_groups[0]["params"]))


def test_a_captured_step_goes_on_after_a_load(tmp_path):
    """Moments, counts and the rate are read where they were when the step was captured."""
    ps, qs = _params(19, (BF16, F32)), _params(19, (BF16, F32))
    kw = dict(weight_decay=0.1, state_bits=8, master_weights=True, max_norm=1e-2)
    rate = torch.full((1,), 0.01, device="cuda")
    captured, eager = AdamW(ps, lr=rate, **kw), AdamW(qs, lr=0.01, **kw)
    for p, q, g in zip(ps, qs, _grads(19)):
        p.grad, q.grad = g.to(p.dtype), g.to(p.dtype)
    captured.step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured.step()
    for t in range(3):
        graph.replay()
        eager.step()
        torch.cuda.synchronize()
    eager.param_groups[0]["lr"] = 2.0 ** -7
    for saved in (0, 1):
        torch.save((eager.state_dict(), [q.detach() for q in qs]), tmp_path / "state")
        sd, values = torch.load(tmp_path / "state", weights_only=True, map_location="cpu")
        captured.load_state_dict(sd)
        for p, x in zip(ps, values):
            p.data.copy_(x)
        assert captured.param_groups[0]["lr"] is rate and float(rate) == 2.0 ** -7
        for t in range(3):
            for p, q, g in zip(ps, qs, _grads(120 + 3 * saved + t)):
                p.grad.copy_(g)
                q.grad.copy_(g)
            graph.replay()
            eager.step()
            torch.cuda.synchronize()
            assert all(torch.equal(p, q) for p, q in zip(ps, qs)), (saved, t)
        captured.step(), eager.step()
        assert all(torch.equal(p, q) for p, q in zip(ps, qs))
    other = AdamW(_params(20, (BF16, F32)), **kw)     # a number before: the saved tensor, on the parameters' device
    torch.save(captured.state_dict(), tmp_path / "state")
    other.load_state_dict(torch.load(tmp_path / "state", weights_only=True, map_location="cpu"))
    assert other.param_groups[0]["lr"].is_cuda
    for p, x in zip(other.param_groups[0]["params"], ps):
        p.data.copy_(x.data)
        p.grad = x.grad.clone()
    other.step(), captured.step()
    assert all(torch.equal(p, q) for p, q in zip(ps, other.param_groups[0]["params"]))


def test_a_captured_steps_parameters_have_gradients_together():
    ps, qs = _params(21), _params(21)
    a, b = AdamW(ps, lr=1e-2), AdamW(qs, lr=1e-2)
    for p, q, g in zip(ps, qs, _grads(21)):
        p.grad, q.grad = g, g.clone()
    a.step(), b.step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a.step()
    held, ps[2].grad = ps[2].grad, None
    with pytest.raises(RuntimeError, match="captured"):
        a.step()
    ps[2].grad = held
    for t in range(3):
        graph.replay()
        b.step()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(ps, qs)), t
        a.step(), b.step()
        assert all(torch.equal(p, q) for p, q in zip(ps, qs)), t
    assert a.state_dict()["adamw"]["counts"] == b.state_dict()["adamw"]["counts"] == [7]


def test_two_captured_steps_of_different_parameters():
    """Taken with each set before the first capture, the steps replay in any order beside eager ones."""
    ps, qs = _params(22), _params(22)
    a, b = AdamW(ps, lr=1e-2, max_norm=1e-2), AdamW(qs, lr=1e-2, max_norm=1e-2)
    held = [(torch.empty_like(p), torch.empty_like(p)) for p in ps]
    sets = {"all": range(5), "some": (0, 3), "one": (3,)}

    def grads(t, name):
        for i, (p, q, g) in enumerate(zip(ps, qs, _grads(140 + t))):
            held[i][0].copy_(g), held[i][1].copy_(g)
            p.grad, q.grad = held[i] if i in sets[name] else (None, None)

    for t, name in enumerate(sets):
        grads(t, name), a.step(), b.step()
    torch.cuda.synchronize()
    graphs = {}
    for name in ("all", "some"):
        grads(3, name)
        graphs[name] = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graphs[name]):
            a.step()
    for t, name in enumerate(("some", "all", "one", "some", "some", "one", "all"), 4):
        grads(t, name)
        graphs[name].replay() if name in graphs else a.step()
        b.step()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(ps, qs)), (t, name)
    counts = lambda o: [o.state_dict()["adamw"]["counts"][s] for s in o.param_groups[0]["_slots"]]  # noqa: E731
    assert counts(a) == counts(b) == [7, 3, 3, 10, 3]
