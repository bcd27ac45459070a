"""The AdamW operators over many tensors against their formulas in 64 bits, within
bounds derived from each rounding (tests/adamw_reference.py)."""
import ctypes as C
import math

import pytest
import torch

import adamw_reference as R
from gpu_harness import say
from memory_compressed_adaptive_amd import _lib as L
from memory_compressed_adaptive_amd import adamw

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


# around a thread's run, a block, a workgroup's chunk and several of them; an empty one
SHAPES = [(1,), (7,), (8,), (9,), (255,), (0,), (256,), (257,), (3, 85), (2047,), (2048,), (2049,), (31, 67), (5, 4099), ()]


def _place(shapes, dtype, offset):
    """Zeros of these shapes, `offset` elements behind an aligned start (None: allocated apart)."""
    out = []
    for s in shapes:
        n = math.prod(s)
        buf = torch.zeros(n + (offset or 0), dtype=dtype, device="cuda")
        out.append(buf[(offset or 0):].view(s))
    return out


class Case:
    """A list with its states on the GPU and, in 64 bits, on the CPU."""

    def __init__(self, seed, shapes=SHAPES, ptypes=(F32,), gtypes=(F32,), offset=None, bits=32, copy=False, spread=2.0):
        self.g = torch.Generator().manual_seed(seed)
        self.shapes, self.gtypes, self.offset, self.bits, self.spread = shapes, gtypes, offset, bits, spread
        kinds = [ptypes[i % len(ptypes)] for i in range(len(shapes))]
        self.params = [_place([s], k, offset)[0] for s, k in zip(shapes, kinds)]
        values = [0.02 * torch.randn(s, generator=self.g, dtype=torch.float64) for s in shapes]
        for p, x in zip(self.params, values):
            p.copy_(x)
        self.at, size = adamw.starts(self.params), adamw.state_size(self.params)
        self.fill = 1.0 if bits == 32 else 3   # between the tensors: not touched
        self.master = torch.full((size,), float(self.fill), device="cuda") if copy else None
        if bits == 32:
            self.state = [torch.full((size,), self.fill, device="cuda") for _ in range(2)]
        else:
            self.state = [torch.full((size,), self.fill, dtype=d, device="cuda") for d in (torch.int8, torch.uint8)]
            self.state += [torch.zeros(size // 256, device="cuda") for _ in range(2)]
        self.inside = torch.zeros(size, dtype=torch.bool)
        for i, p in enumerate(self.params):
            s = slice(self.at[i], self.at[i] + p.numel())
            self.inside[s] = True
            for x in self.state[:2]:
                x[s] = 0
            if copy:
                # a copy with the bits that bf16 leaves out
                self.master[s] = (values[i].view(-1).float().cuda() if kinds[i] == BF16 else 7.0)
        self.near = math.inf

    def grads(self, zeros=0.1):
        """Gradients of very different sizes in one block, some of them zero."""
        out = []
        for i, s in enumerate(self.shapes):
            x = torch.randn(s, generator=self.g, dtype=torch.float64) * 10.0 ** (-2 - self.spread * torch.rand(s, generator=self.g, dtype=torch.float64))
            x = x * (torch.rand(s, generator=self.g) >= zeros)
            kind = self.gtypes[(i // 2) % len(self.gtypes)]
            out.append(_place([s], kind, self.offset)[0].copy_(x))
        return out

    def snapshot(self):
        return [x.cpu() for x in self.state], None if self.master is None else self.master.cpu(), [p.detach().cpu() for p in self.params]

    def run(self, grads, t, **kw):
        fn = adamw.adamw_step if self.bits == 32 else adamw.adamw8_step
        fn(self.params, grads, *self.state, t, master=self.master, **kw)

    def check(self, before, grads, t, lr, wd, scale=1.0, beta1=0.9, beta2=0.999, eps=1e-8):
        """The step that led from `before` to now."""
        state0, master0, params0 = before
        state1, master1, params1 = self.snapshot()
        for x0, x1 in zip(state0[:2], state1[:2]):
            assert torch.equal(x0[~self.inside], x1[~self.inside]), "between the tensors"
        for i, (p0, p1) in enumerate(zip(params0, params1)):
            n = p0.numel()
            if not n:
                continue
            e = slice(self.at[i], self.at[i] + n)
            b = slice(self.at[i] // 256, self.at[i] // 256 + -(-n // 256))
            if grads[i] is None:
                assert torch.equal(p0, p1) and all(torch.equal(x0[e], x1[e]) for x0, x1 in zip(state0[:2], state1[:2]))
                continue
            copied = self.master is not None and p0.dtype == BF16
            p = (master0[e] if copied else p0.reshape(-1)).double()
            g = grads[i].cpu().double().reshape(-1)
            if self.bits == 32:
                m, v = (x[e].double() for x in state0)
            else:
                m, v = R.decode(state0[0][e], state0[1][e], state0[2][b], state0[3][b])
            q, m1, v1, upd = R.step(p, g, m, v, t, lr, wd, scale, beta1, beta2, eps)
            # 32 bits: root, its factor, sum with eps, eps, the other factor, its product, division (each half a
            # step).  8 bits: an estimated root and reciprocal instead, within the 16 half steps that
            # their documented errors come to.
            em, ev, ep = R.step_tolerance(p, g * scale, m, v, m1, v1, upd, q, lr, wd, beta1, beta2, eps, t, 7.5 if self.bits == 32 else 17)
            got = (master1[e] if copied else p1.reshape(-1)).double()
            if p0.dtype == BF16:
                if copied:
                    assert torch.equal(p1.reshape(-1), master1[e].bfloat16()), "the copy's rounding"
                else:
                    ep = ep + 2.0 ** -8 * (q.abs() + ep)
            assert bool(((got - q).abs() <= ep).all()), (i, float(((got - q).abs() / ep).max()))
            if self.master is not None and not copied:
                assert torch.equal(master0[e], master1[e])
            if self.bits == 32:
                assert bool(((state1[0][e].double() - m1).abs() <= em).all()), (i, "m")
                assert bool(((state1[1][e].double() - v1).abs() <= ev).all()), (i, "v")
            else:
                sm, sr = state1[2][b], state1[3][b]
                for what, have, top in zip(("sm", "sr"), (sm, sr), R.tops(m1, v1)):
                    assert bool(R.is_rounded(have, top).all()), (i, what)
                cm, cv, near = R.encode(m1, v1, sm, sr)
                self.near = min(self.near, near)
                for what, want, have in (("cm", cm, state1[0][e]), ("cv", cv, state1[1][e])):
                    assert torch.equal(want, have), (i, what, int((want != have).sum()), near)


TYPES = [((F32,), (F32,)), ((F32,), (BF16,)), ((BF16,), (F32,)), ((BF16,), (BF16,)), ((F32, BF16, BF16), (BF16, F32))]


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("offset", [None, 1])
@pytest.mark.parametrize("ptypes,gtypes", TYPES)
def test_steps(bits, offset, ptypes, gtypes):
    c = Case(11, ptypes=ptypes, gtypes=gtypes, offset=offset, bits=bits)
    for t in range(1, 5):
        g, before = c.grads(), c.snapshot()
        kw = dict(lr=1e-3, wd=0.1 if t % 2 else 0.0)
        say(f"[adamw many] bits={bits} offset={offset} {ptypes} {gtypes} step {t}")
        c.run(g, t, **kw)
        c.check(before, g, t, **kw)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("ptypes,gtypes", TYPES[2:])
def test_steps_with_copies(bits, ptypes, gtypes):
    c = Case(12, ptypes=ptypes, gtypes=gtypes, bits=bits, copy=True)
    for t in range(1, 4):
        g, before = c.grads(), c.snapshot()
        say(f"[adamw many] copies, bits={bits} {ptypes} {gtypes} step {t}")
        c.run(g, t, lr=3e-4, wd=0.1)
        c.check(before, g, t, 3e-4, 0.1)


@pytest.mark.parametrize("bits", [32, 8])
def test_arguments_on_the_gpu(bits):
    """Count, rate and the gradients' factor as tensors, and other betas and eps."""
    c = Case(13, bits=bits, gtypes=(BF16, F32))
    lr, scale, t = (torch.zeros(1, device="cuda"), torch.zeros(1, device="cuda"), torch.zeros(1, dtype=torch.int64, device="cuda"))
    for step, (rate, factor, beta1, beta2, eps) in enumerate([(1e-2, 0.25, 0.9, 0.999, 1e-8), (3e-3, 1.0, 0.0, 0.95, 1e-6),
                                                              (1e-4, 3e-3, 0.95, 0.0, 1e-12), (1e-3, 0.7, 0.8, 0.9999, 1e-3)]):
        count = (1, 2, 3, 123456789)[step]
        lr.fill_(rate), scale.fill_(factor), t.fill_(count)
        g, before = c.grads(), c.snapshot()
        say(f"[adamw many] on the GPU, bits={bits} step {step}")
        c.run(g, t, lr=lr, wd=0.05, scale=scale, beta1=beta1, beta2=beta2, eps=eps)
        c.check(before, g, count, float(lr), 0.05, float(scale), beta1, beta2, eps)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("t,scale", [(0, 0.5), (-4, 0.5), (3, math.nan)])
def test_steps_that_change_nothing(bits, t, scale):
    c = Case(14, bits=bits, ptypes=(F32, BF16), copy=True)
    c.run(c.grads(), 1, lr=1e-3)
    before = c.snapshot()
    c.run(c.grads(), torch.tensor([t], device="cuda"), lr=1e-3, wd=0.1, scale=torch.tensor([scale], device="cuda"))
    after = c.snapshot()
    assert all(torch.equal(a, b) for a, b in zip(before[0] + before[2] + [before[1]], after[0] + after[2] + [after[1]]))


@pytest.mark.parametrize("bits", [32, 8])
def test_missing_gradients_and_long_lists(bits):
    """More tensors than a launch takes, of all types, every fifth without a gradient."""
    g = torch.Generator().manual_seed(5)
    shapes = [(int(n),) for n in torch.randint(0, 700, (487,), generator=g)]
    c = Case(15, shapes=shapes, ptypes=(BF16, F32, F32), gtypes=(BF16, F32), bits=bits, copy=True)
    for t in (1, 2):
        gs, before = c.grads(), c.snapshot()
        for i in range(t, len(gs), 5):
            gs[i] = None
        say(f"[adamw many] long list, bits={bits} step {t}")
        c.run(gs, t, lr=1e-3, wd=0.01)
        c.check(before, gs, t, 1e-3, 0.01)


@pytest.mark.parametrize("bits", [32, 8])
def test_one_long_tensor_and_every_workgroup(bits):
    """More chunks than workgroups, with an odd end."""
    c = Case(16, shapes=[(2048 * 2048 * 2 + 2049,), (5,)], ptypes=(BF16,), gtypes=(BF16,), bits=bits)
    g, before = c.grads(), c.snapshot()
    c.run(g, 1, lr=1e-3)
    c.check(before, g, 1, 1e-3, 0.0)


@pytest.mark.parametrize("bits", [32, 8])
def test_permuted_parameters(bits):
    """Dense parameters in any order of their dimensions, with gradients that lie like them."""
    shapes = [(6, 50, 9)]
    c = Case(17, shapes=shapes, bits=bits)
    base, g = c.params[0], c.grads()[0]
    before = c.snapshot()
    fn = adamw.adamw_step if bits == 32 else adamw.adamw8_step
    fn([base.permute(2, 0, 1)], [g.permute(2, 0, 1)], *c.state, 1, lr=1e-3)
    c.check(before, [g], 1, 1e-3, 0.0)
    with pytest.raises(ValueError, match="strides"):
        fn([base.permute(2, 0, 1)], [g.permute(2, 0, 1).contiguous()], *c.state, 2)
    with pytest.raises(ValueError, match="dense"):
        fn([base[:, :, ::2]], [g[:, :, ::2]], *c.state, 2)


def _moves(p, g):
    """Whether a step takes this pair: with m = v = 0 each element moves by lr against its gradient's sign."""
    q, size = p.clone(), adamw.state_size([p])
    m, v = (torch.zeros(size, device="cuda") for _ in range(2))
    try:
        adamw.adamw_step([p], [g], m, v, 1, lr=1.0)
    except ValueError:
        return False
    # m^ = g and v^ = g^2, so the move is |g| / (|g| + eps) = 1 - eps / (|g| + eps) of lr = 1; a sum in fp32
    # and the update's 8 roundings are off by 2^-24 each, of at most |q| + 2
    assert bool(((p - (q - g.sign())).abs() <= 1e-8 / g.abs() + 2.0 ** -20 * (q.abs() + 2)).all())
    return True


def test_layouts():
    """Every dense layout is taken where the gradient has it too; others are refused."""
    f = lambda *s: torch.randn(*s, device="cuda")  # noqa: E731
    assert _moves(f(4, 6, 5).permute(2, 0, 1), f(4, 6, 5).permute(2, 0, 1))
    assert _moves(f(2, 3, 4, 5).to(memory_format=torch.channels_last), f(2, 3, 4, 5).to(memory_format=torch.channels_last))
    assert _moves(f(4, 6)[1], f(6)) and _moves(f(4, 6)[:1, :1], f(1, 1)) and _moves(f(6, 1), f(1, 6).t()) and _moves(f(3, 1, 4), f(3, 4)[:, None])
    assert _moves(f(1, 6, 1).expand(1, 6, 1), f(1, 6, 1))
    assert not _moves(f(4, 6), f(6, 4).t()) and not _moves(f(6, 4).t(), f(4, 6)) and not _moves(f(4, 6), f(6, 4)) and not _moves(f(24), f(4, 6))
    assert not _moves(f(4, 6), f(4, 1).expand(4, 6)) and not _moves(f(4, 6)[:, ::2], f(4, 6)[:, ::2]) and not _moves(f(4, 1).expand(4, 6), f(4, 6))
    assert not _moves(f(4, 6), f(4, 6).to_sparse()) and not _moves(f(4, 6), torch._neg_view(f(4, 6)))
    with pytest.raises(ValueError):
        adamw.grad_norm([f(4, 6)[:, 1]])
    with pytest.raises(ValueError):
        adamw.grad_norm([f(4, 1).expand(4, 6)])
    want = f(3, 4, 5)
    norm, _ = adamw.grad_norm(iter([want.permute(1, 2, 0), want[0, 0]]))
    assert float(norm) == pytest.approx(float((want.double().square().sum() + want[0, 0].double().square().sum()).sqrt()), rel=1e-7)


@pytest.mark.parametrize("bits", [32, 8])
def test_the_same_bits_in_other_lists_and_calls(bits):
    """How tensors are put together in lists changes no bit."""
    a, b = Case(18, bits=bits, gtypes=(BF16,)), Case(18, bits=bits, gtypes=(BF16,))
    fn = adamw.adamw_step if bits == 32 else adamw.adamw8_step
    for t in (1, 2, 3):
        g = a.grads()
        a.run(g, t, lr=1e-3, wd=0.1)
        for i, p in enumerate(b.params):
            e = slice(b.at[i], b.at[i] + -(-p.numel() // 256) * 256)
            s = slice(e.start // 256, e.stop // 256)
            fn([p], [g[i]], *(x[e] for x in b.state[:2]), *(x[s] for x in b.state[2:]), t, lr=1e-3, wd=0.1)
    assert all(torch.equal(x, y) for x, y in zip(a.params + a.state, b.params + b.state))


SPECIAL = [0.0, -0.0, 1e-30, -1e-38, 1e-42, 3e-23, 1e10, -1e18, 1.0, 1e-8]


@pytest.mark.parametrize("bits", [32, 8])
def test_extreme_gradients(bits):
    """Zeros, subnormal and huge values, alone in a block and together."""
    shapes = [(300,)] * len(SPECIAL) + [(300,)]
    c = Case(19, shapes=shapes, bits=bits)
    for t in (1, 2):
        g = [torch.full(s, x, device="cuda") for s, x in zip(shapes, SPECIAL)]
        g.append(torch.tensor(SPECIAL * 30, device="cuda"))
        before = c.snapshot()
        say(f"[adamw many] extremes, bits={bits} step {t}")
        c.run(g, t, lr=1e-3)
        c.check(before, g, t, 1e-3, 0.0)


def test_8_bit_moments_that_fade():
    """Blocks whose gradients stop: m fades to subnormal numbers and to zero within a thousand
    steps while v hardly does, which crosses every way of forming codes."""
    shapes = [(700,), (256,), (1,)]
    c = Case(23, shapes=shapes, bits=8)
    c.run(c.grads(), 1, lr=1e-3)
    zero = [torch.zeros(s, device="cuda") for s in shapes]
    checked = {2, 3, 50, 300, 500, 620, 640, 660, 680, 780, 800, 830, 870, 900, 930, 950, 970, 990, 1010}
    for t in range(2, 1012):
        before = c.snapshot() if t in checked else None
        c.run(zero, t, lr=1e-3, wd=0.01)
        if t in checked:
            c.check(before, zero, t, 1e-3, 0.01)
    assert not bool(c.state[0][c.inside.cuda()].any()) and bool((c.state[3] > 0).all())


@pytest.mark.parametrize("exponent", [-140, -100, -95, -90, -75, -70, -65, -60, -45, 20, 29, 31, 32, 33, 45, 62, 64, 66])
def test_8_bit_moments_of_any_size(exponent):
    """Gradients around a power of two, where the ways of forming codes meet."""
    shapes = [(1000,), (40,)]
    c = Case(24, shapes=shapes, bits=8)
    for t in (1, 2, 3):
        g = [(x.double().cpu() * 2.0 ** exponent * 300).float().cuda() for x in c.grads()]
        before = c.snapshot()
        c.run(g, t, lr=1e-3, wd=0.1)
        c.check(before, g, t, 1e-3, 0.1)


@pytest.mark.parametrize("value", [math.inf, -math.inf, math.nan])
def test_values_that_are_not_finite(value):
    """32 bits: the element alone is lost.  8 bits: its block of 256 reads as NaN from
    the next step on, the blocks beside it are what they would be without."""
    a, b = (Case(20, shapes=[(1000,)]) for _ in range(2))
    ga, gb = a.grads()[0], b.grads()[0]
    ga[300] = value
    a.run([ga], 1, lr=1e-3), b.run([gb], 1, lr=1e-3)
    keep = torch.arange(1000) != 300
    for x, y in zip([a.params[0], a.state[0][:1000], a.state[1][:1000]], [b.params[0], b.state[0][:1000], b.state[1][:1000]]):
        assert torch.equal(x.cpu()[keep], y.cpu()[keep]) and not math.isfinite(float(x[300]))
    a, b = (Case(20, shapes=[(1000,)], bits=8) for _ in range(2))
    a.run([ga], 1, lr=1e-3), b.run([gb], 1, lr=1e-3)
    # the block's scale of sqrt(v), which the update's estimate of the root goes by, lacks the lost
    # element: others in it are off by a few half steps of their update at most
    pa, pb = a.params[0].cpu(), b.params[0].cpu()
    block = torch.arange(1000) // 256 == 1
    assert torch.equal(pa[~block], pb[~block]) and not math.isfinite(float(pa[300]))
    assert bool(((pa - pb).abs()[block & keep] <= 1e-3 * 40 * R.U + R.U * pb.abs()[block & keep] * 2).all())
    m, v = (x.cpu()[:1000] for x in adamw.adamw8_values(*a.state))
    assert bool(m[block].isnan().all() and v[block].isnan().all()) and bool(m[~block].isfinite().all() and v[~block].isfinite().all())
    for x, y in zip(a.state[:2], b.state[:2]):
        assert not bool(x.cpu()[:1000][block].any()) and torch.equal(x.cpu()[:1000][~block], y.cpu()[:1000][~block])
    a.run([gb], 2, lr=1e-3)
    assert bool(a.params[0].cpu()[block].isnan().all()) and bool(a.params[0].cpu()[~block].isfinite().all())


def test_values_of_all_codes():
    cm = torch.arange(-128, 128, dtype=torch.int64).to(torch.int8).repeat(3).cuda()
    cv = torch.arange(256, dtype=torch.int64).to(torch.uint8).repeat(3).cuda()
    sm, sr = torch.tensor([0.37, 3e38, 0.0], device="cuda"), torch.tensor([2.1e-3, 1e-20, 0.0], device="cuda")
    m, v = (x.cpu().double() for x in adamw.adamw8_values(cm, cv, sm, sr))
    want_m, want_v = R.decode(cm.cpu(), cv.cpu(), sm.cpu(), sr.cpu())
    inside = want_m.abs() <= torch.finfo(F32).max
    assert bool(((m - want_m).abs()[inside] <= 1.001 * R.U * want_m.abs()[inside] + R.TINY).all())
    assert bool(((v - want_v).abs() <= 1.001 * R.U * want_v.abs() + R.TINY).all())


# ------------------------------------------------------------------- the norm


def _want(grads):
    return math.sqrt(math.fsum(float(g.cpu().double().square().sum()) for g in grads if g is not None))


@pytest.mark.parametrize("offset", [None, 1])
@pytest.mark.parametrize("gtypes", [(F32,), (BF16,), (BF16, F32)])
@pytest.mark.parametrize("max_norm", [math.inf, 1e-3, 1e6])
def test_norm(offset, gtypes, max_norm):
    c = Case(30, shapes=SHAPES + [(100, 1001), (9000,)], gtypes=gtypes, offset=offset)
    g = c.grads()
    say(f"[norm] {offset} {gtypes} {max_norm}")
    norm, scale = adamw.grad_norm(g, max_norm)
    want = _want(g)
    assert abs(float(norm) - want) <= 1.001 * R.U * want
    factor = min(1.0, max_norm / (want + 1e-6))
    assert abs(float(scale) - factor) <= 1.001 * R.U * factor
    again = adamw.grad_norm(g, max_norm)
    assert torch.equal(norm, again[0]) and torch.equal(scale, again[1])


def test_norm_of_long_lists_and_none():
    g = torch.Generator().manual_seed(6)
    gs = [torch.randn(int(n), generator=g).cuda() if n % 7 else None for n in torch.randint(0, 500, (1000,), generator=g)]
    out = torch.empty(2, device="cuda")
    t = torch.tensor([41], device="cuda")
    norm, _ = adamw.grad_norm(gs, 2.0, t=t, out=out)
    want = _want(gs)
    assert abs(float(norm) - want) <= 1.001 * R.U * want and float(out[0]) == float(norm) and int(t) == 42
    norm, scale = adamw.grad_norm([None], out=out)
    assert float(norm) == 0.0 and float(scale) == 1.0


@pytest.mark.parametrize("shapes", [
    [(2048,)] * 64, [(2048,)] * 65, [(2049,)] * 32, [(2049,)] * 33, [(64 * 2048,)], [(64 * 2048 + 1,)],   # one launch, or two
    [(3,)] * 60 + [(0,)] * 200, [(1,)] * 250, [(1,)] * 251, [(5,)] * 501,                                 # one table, two, three
    [(8192 * 3,), (8191,), (8193,)], [(8192 * 513,)], [(511,), (512,), (513,), (1536,), (2047,)]])
@pytest.mark.parametrize("gtypes", [(F32,), (BF16, F32)])
def test_norms_of_all_lengths(shapes, gtypes):
    c = Case(32, shapes=shapes, gtypes=gtypes, offset=3)
    g = c.grads(zeros=0.0)
    say(f"[norm] {len(shapes)} tensors of {shapes[0]}")
    norm, _ = adamw.grad_norm(g)
    want = _want(g)
    assert abs(float(norm) - want) <= 1.001 * R.U * want


def test_norm_of_one_long_tensor():
    g = torch.randn(40_000_003, device="cuda", generator=torch.Generator("cuda").manual_seed(2)).bfloat16()
    norm, _ = adamw.grad_norm([g])
    want = float(g.double().square().sum().sqrt())
    assert abs(float(norm) - want) <= 1.001 * R.U * want


@pytest.mark.parametrize("value", [1e30, 1e-30, 3e38, 1e-45])
def test_norms_of_extreme_gradients(value):
    g = [torch.full((3,), value, device="cuda"), torch.zeros(1000, device="cuda")]
    norm, scale = adamw.grad_norm(g, 1.0)
    want = math.sqrt(3) * float(g[0][0])
    assert float(norm) == pytest.approx(want, rel=1e-7, abs=1e-45) if want < 3.4e38 else float(norm) == math.inf
    assert float(scale) == pytest.approx(min(1.0, 1.0 / (want + 1e-6)), rel=1e-7, abs=1e-45)


@pytest.mark.parametrize("value", [math.inf, -math.inf, math.nan])
def test_a_norm_that_is_not_finite_stops_the_step(value):
    c = Case(31, gtypes=(BF16, F32), bits=8)
    g, t = c.grads(), torch.tensor([1], device="cuda")
    g[7].view(-1)[100] = value
    norm, scale = adamw.grad_norm(g, 1.0, t=t)
    assert not math.isfinite(float(norm)) and math.isnan(float(scale)) and int(t) == 1
    before = c.snapshot()
    c.run(g, t, lr=1e-3, scale=scale)
    after = c.snapshot()
    assert all(torch.equal(a, b) for a, b in zip(before[0] + before[2], after[0] + after[2]))


# ------------------------------------------------ together, graphs, streams, sizes


@pytest.mark.parametrize("bits", [32, 8])
def test_clipped_steps_together(bits):
    """Norm, factor and step as a training loop calls them, with gradients above and below max_norm."""
    c = Case(40, ptypes=(F32, BF16), gtypes=(F32, BF16), bits=bits, copy=True)
    t = torch.zeros(1, dtype=torch.int64, device="cuda")
    for step in range(1, 5):
        g, before = c.grads(), c.snapshot()
        if step % 2:
            for x in g:
                x.mul_(1000)
        norm, scale = adamw.grad_norm(g, 1.0, t=t)
        c.run(g, t, lr=1e-3, wd=0.1, scale=scale)
        want = _want(g)
        assert (float(scale) < 1) == (want > 1) and int(t) == step
        c.check(before, g, step, 1e-3, 0.1, float(scale))


@pytest.mark.parametrize("bits", [32, 8])
def test_a_captured_step(bits):
    """Replayed steps with new gradients, counts and rates are the eager ones, bit for
    bit, with eager work and synchronizations between them."""
    shapes = SHAPES + [(100,)] * 130
    a, b = (Case(41, shapes=shapes, ptypes=(BF16, F32), gtypes=(F32,), bits=bits, copy=True) for _ in range(2))
    static = a.grads()
    ta, tb = (torch.zeros(1, dtype=torch.int64, device="cuda") for _ in range(2))
    lr = torch.full((1,), 1e-3, device="cuda")

    def step(c, g, t):
        norm, scale = adamw.grad_norm(g, 0.5, t=t)
        c.run(g, t, lr=lr, wd=0.1, scale=scale)
        return norm

    graph = torch.cuda.CUDAGraph()
    warm = torch.cuda.Stream()
    with torch.cuda.stream(warm):
        adamw.grad_norm(static)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        norm = step(a, static, ta)
    for i in range(5):
        g = b.grads()
        for x, y in zip(static, g):
            x.copy_(y)
        lr.fill_(1e-3 / (i + 1))
        graph.replay()
        if i % 2:
            torch.cuda.synchronize()
        other = step(b, g, tb)
        torch.cuda.synchronize()
        say(f"[adamw many] replay {i} bits={bits}")
        assert float(norm) == float(other) and int(ta) == int(tb) == i + 1
        for x, y in zip(a.params + a.state + [a.master], b.params + b.state + [b.master]):
            assert torch.equal(x, y)


def test_two_captured_norms_at_once():
    """Each graph has a workspace of its own."""
    sets = [[torch.randn(3_000_000, device="cuda", generator=torch.Generator("cuda").manual_seed(s))] for s in (1, 2)]
    adamw.grad_norm(sets[0])
    torch.cuda.synchronize()
    graphs, outs = [], []
    for s in sets:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(adamw.grad_norm(s)[0])
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(10):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for o, s in zip(outs, sets):
            assert float(o) == float(adamw.grad_norm(s)[0])


@pytest.mark.parametrize("bits", [32, 8])
def test_another_stream(bits):
    a, b = Case(42, bits=bits), Case(42, bits=bits)
    s = torch.cuda.Stream()
    for t in (1, 2):
        g = a.grads()
        a.run(g, t, lr=1e-3)
        torch.cuda.synchronize()
        _, scale = adamw.grad_norm(g, math.inf, stream=s)
        b.run(g, t, lr=1e-3, stream=s)
        s.synchronize()
        assert float(scale) == 1.0
    if bits == 8:
        m, _ = adamw.adamw8_values(*b.state, stream=s)
        s.synchronize()
        assert torch.equal(m, adamw.adamw8_values(*a.state)[0])
    assert all(torch.equal(x, y) for x, y in zip(a.params + a.state, b.params + b.state))


@pytest.mark.parametrize("bits", [32, 8])
def test_two_lists_at_once(bits):
    """Steps and norms of two lists on two streams, under way together, are those one after the other."""
    shapes = [(300_000,), (7,), (65_537,)] + [(100,)] * 150
    a, b = ([Case(44 + k, shapes=shapes, ptypes=(BF16, F32), gtypes=(F32,), bits=bits, copy=True) for k in range(2)] for _ in range(2))
    gs = [[c.grads() for _ in range(4)] for c in a]
    streams, ts = [torch.cuda.Stream() for _ in a], [torch.zeros(1, dtype=torch.int64, device="cuda") for _ in a + b]
    torch.cuda.synchronize()
    norms = [[], []]
    for i in range(4):
        for k, (c, s) in enumerate(zip(a, streams)):
            norm, scale = adamw.grad_norm(gs[k][i], 0.1, t=ts[k], stream=s)
            c.run(gs[k][i], ts[k], lr=1e-3, wd=0.1, scale=scale, stream=s)
            norms[k].append((norm, scale))
    torch.cuda.synchronize()
    for k, c in enumerate(b):
        for i in range(4):
            norm, scale = adamw.grad_norm(gs[k][i], 0.1, t=ts[2 + k])
            c.run(gs[k][i], ts[2 + k], lr=1e-3, wd=0.1, scale=scale)
            assert float(norm) == float(norms[k][i][0]) and float(scale) == float(norms[k][i][1])
        for x, y in zip(a[k].params + a[k].state + [a[k].master], c.params + c.state + [c.master]):
            assert torch.equal(x, y)


def test_autograd_is_told():
    w = torch.nn.Parameter(torch.ones(4, device="cuda"))
    y = (w * w).sum()
    m, v = torch.zeros(256, device="cuda"), torch.zeros(256, device="cuda")
    adamw.adamw_step([w], [torch.ones(4, device="cuda")], m, v, 1)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()


def test_inference_tensors_and_generators():
    with torch.inference_mode():
        p, g = torch.zeros(10, device="cuda"), torch.ones(10, device="cuda")
        m, v = torch.zeros(256, device="cuda"), torch.zeros(256, device="cuda")
        adamw.adamw_step((x for x in [p]), (x for x in [g]), m, v, 1)
        assert bool((p < 0).all())


@pytest.mark.parametrize("bits", [32, 8])
def test_a_tensor_given_twice_and_gradients_shared(bits):
    c = Case(43, shapes=[(300,), (300,)], bits=bits)
    g = c.grads()[0]
    before = c.snapshot()
    c.run([g, g], 1, lr=1e-3)
    c.check(before, [g, g], 1, 1e-3, 0.0)
    c.params[1] = c.params[0]
    with pytest.raises(L.MicroAdamError, match="overlap"):
        c.run([g, g], 2)
    c.params[0], c.params[1] = c.params[0][:299], c.params[0][1:]
    with pytest.raises(L.MicroAdamError, match="overlap"):
        c.run([g[:299], g[1:]], 2)


def test_refusals_with_tensors():
    p, g = [torch.zeros(300, device="cuda")], [torch.ones(300, device="cuda")]
    s = [torch.zeros(512, device="cuda") for _ in range(2)]
    bad = [
        dict(grads=[g[0][:-1]]), dict(grads=[g[0].half()]), dict(grads=[g[0].cpu()]), dict(m=s[0][:256]), dict(m=s[0].double()),
        dict(v=s[1].view(2, 256).t()), dict(master=s[0][:256]), dict(t=torch.ones(1, device="cuda")), dict(t=torch.ones(1, dtype=torch.int64)),
        dict(t=torch.ones(2, dtype=torch.int64, device="cuda")), dict(lr=torch.ones(1, device="cuda", dtype=torch.float64)),
        dict(scale=torch.ones(2, device="cuda")), dict(scale=torch.ones(1))]
    for kw in bad:
        kw = {**dict(params=p, grads=g, m=s[0], v=s[1], t=1), **kw}
        with pytest.raises(ValueError):
            adamw.adamw_step(**kw)
    for kw in (dict(params=p + p, grads=g + g, m=torch.zeros(1024, device="cuda"), v=torch.zeros(1024, device="cuda")), dict(t=0),
               dict(lr=math.nan), dict(beta1=1.0)):
        kw = {**dict(params=p, grads=g, m=s[0], v=s[1], t=1), **kw}
        with pytest.raises(L.MicroAdamError):
            adamw.adamw_step(**kw)
    assert not any(bool(x.any()) for x in p + s)
    with pytest.raises(ValueError):
        adamw.grad_norm([g[0][::2]])
    with pytest.raises(L.MicroAdamError):
        adamw.grad_norm(g, 0.0)
    codes = [torch.zeros(512, dtype=d, device="cuda") for d in (torch.int8, torch.uint8)]
    scales = [torch.zeros(2, device="cuda") for _ in range(2)]
    for i in range(4):
        state = codes + scales
        state[i] = state[i][:1]
        with pytest.raises(ValueError):
            adamw.adamw8_step(p, g, *state, 1)
        if i:
            with pytest.raises(ValueError):
                adamw.adamw8_values(*state)


@pytest.mark.parametrize("bits", [32, 8])
def test_offsets_past_32_bits(bits):
    """A tensor of 2^31 + 2^21 + 3 elements (byte offsets past 2^32, elements past 2^31) and
    one behind it: the ends are as if they were lists of their own."""
    n, tail = 2 ** 31 + 2 ** 21 + 3, 2 ** 21 + 3
    gen = torch.Generator("cuda").manual_seed(9)
    p = torch.zeros(n, dtype=BF16, device="cuda")
    g = torch.zeros(n, dtype=BF16, device="cuda")
    p[-tail:] = (0.02 * torch.randn(tail, device="cuda", generator=gen)).bfloat16()
    g[-tail:] = (1e-3 * torch.randn(tail, device="cuda", generator=gen)).bfloat16()
    p2, g2 = p[-1000:].clone(), g[-1000:].clone()
    size = adamw.state_size([p, p2])
    dtypes = [(torch.float32, 1)] * 2 if bits == 32 else [(torch.int8, 1), (torch.uint8, 1), (torch.float32, 256), (torch.float32, 256)]
    state = [torch.zeros(size // k, dtype=d, device="cuda") for d, k in dtypes]
    q, q2, end = p[-tail:].clone(), p2.clone(), adamw.state_size([p[-tail:], p2])
    small = [torch.zeros(end // k, dtype=d, device="cuda") for d, k in dtypes]
    fn = adamw.adamw_step if bits == 32 else adamw.adamw8_step
    say(f"[adamw many] {n} elements, bits={bits}")
    fn([p, p2], [g, g2], *state, 1, lr=1e-3)
    fn([q, q2], [g[-tail:], g2], *small, 1, lr=1e-3)
    assert torch.equal(p[-tail:], q) and torch.equal(p2, q2) and not bool(p[:-tail].any())
    for (_, k), x, y in zip(dtypes, state, small):
        assert torch.equal(x[-(end // k):], y)
    norm, _ = adamw.grad_norm([g])
    want = float(g[-tail:].double().square().sum().sqrt())
    assert abs(float(norm) - want) <= 1.001 * R.U * want


def test_more_chunks_than_a_grid_takes():
    """17 parameters of 2^30 elements and some (35 GB of bf16, 36 GB of moments) with one gradient:
    past 2^32 threads of a launch.  The ends are as if they were lists of their own."""
    if torch.cuda.mem_get_info()[0] < 100e9:
        pytest.skip("too little memory")
    gen = torch.Generator("cuda").manual_seed(10)
    n, tail = 2 ** 30 + 1000, 5096
    g = torch.zeros(n, dtype=BF16, device="cuda")
    g[-tail:] = (1e-3 * torch.randn(tail, device="cuda", generator=gen)).bfloat16()
    ps = [torch.zeros(n, dtype=BF16, device="cuda") for _ in range(17)]
    for p in ps:
        p[-tail:] = (0.02 * torch.randn(tail, device="cuda", generator=gen)).bfloat16()
    qs = [p[-tail:].clone() for p in ps]
    state, small = ([torch.zeros(adamw.state_size(x) // k, dtype=d, device="cuda")
                     for d, k in ((torch.int8, 1), (torch.uint8, 1), (torch.float32, 256), (torch.float32, 256))] for x in (ps, qs))
    assert (n - tail) % 256 == 0 and state[0].numel() > 2 ** 34
    say("[adamw many] 17 of 2^30 elements")
    adamw.adamw8_step(ps, [g] * 17, *state, 1, lr=1e-3)
    adamw.adamw8_step(qs, [g[-tail:]] * 17, *small, 1, lr=1e-3)
    for i, (p, q, a, b) in enumerate(zip(ps, qs, adamw.starts(ps), adamw.starts(qs))):
        assert torch.equal(p[-tail:], q), i
        a += n - tail
        e = -(-tail // 256) * 256
        for x, y, k in zip(state, small, (1, 1, 256, 256)):
            assert torch.equal(x[a // k:(a + e) // k], y[b // k:(b + e) // k]), i
    assert not any(bool(p[:-tail].any()) for p in (ps[0], ps[15], ps[16]))


def test_the_c_call_takes_the_null_stream():
    p, g = torch.zeros(10, device="cuda"), torch.ones(10, device="cuda")
    m, v = torch.zeros(256, device="cuda"), torch.zeros(256, device="cuda")
    torch.cuda.synchronize()
    rows = (L.Tensor * 1)(L.Tensor(p.data_ptr(), g.data_ptr(), 10, 0, 0, 0))
    a = L.AdamwArgs(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, wd=0.0, t=1)
    L.check(L.lib().ma_adamw_many_step(1, rows, C.byref(a), None, m.data_ptr(), v.data_ptr(), 256, None))
    torch.cuda.synchronize()
    assert torch.allclose(p, torch.full_like(p, -1e-3), rtol=1e-5) and not bool(m[10:].any())


@pytest.mark.parametrize("n", [1000, 1024, 2048])
def test_norm_of_gradients_that_an_iterator_makes(n):
    """Nobody else holds the 32-bit copies, which are as large as the call's workspace."""
    torch.manual_seed(5)
    g = [torch.randn(n, device="cuda").to(BF16) for _ in range(300)]
    want = math.sqrt(sum(float(x.double().square().sum()) for x in g))
    for _ in range(3):
        norm, scale = adamw.grad_norm((x.float() for x in g), 1.0)
        # one rounding each, beside those in 64 bits
        assert float(norm) == pytest.approx(want, rel=1.01 * 2.0 ** -24)
        assert float(scale) == pytest.approx(1 / (want + 1e-6), rel=1.01 * 2.0 ** -24)


def test_codes_next_to_a_border():
    """Enough elements that some lie nearer to a border between two codes than the kernel's 32-bit
    estimates can tell (6e-7 of the code, so twice that of the value), and are decided in 64 bits; none
    so near that 64 bits cannot tell."""
    c = Case(50, shapes=[(1 << 18,)], bits=8)
    for t in range(1, 4):
        g, before = c.grads(), c.snapshot()
        c.run(g, t, lr=1e-3)
        c.check(before, g, t, 1e-3, 0.0)
    assert 1e-13 < c.near < 6e-7
