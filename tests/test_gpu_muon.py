"""GPU tests of the Muon operators (orthogonalize, muon_step, muon8_step,
momentum8_values) against their formulas in 64 bits.  Tolerances are the bounds
that tests/muon_reference.py derives from the kernels' roundings."""
import math

import numpy as np
import pytest
import torch

import muon_reference as R
from gpu_harness import say
from memory_compressed_adaptive_amd import muon

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _matrix(shape, seed, dtype=torch.float32, size=1e-3):
    g = torch.Generator().manual_seed(seed)
    return (size * torch.randn(shape, generator=g)).to(dtype)


def _check_orthogonal(what, got, u, **kw):
    """got (bf16) against the formula on u, one matrix: the roundings' bound plus
    the result's own rounding to bf16."""
    want, err = R.orthogonalized(u, **kw)
    got = got.detach().cpu()
    assert got.dtype == torch.bfloat16 and got.shape == want.shape
    off = (got.double() - want).norm().item()
    tol = err + R.BF16 * (want.norm().item() + err)
    say(f"[muon] {what}: off {off / want.norm().item():.2e}, allowed {tol / want.norm().item():.2e}")
    assert off <= tol, what


SIZES = [(1, 1), (1, 7), (7, 1), (2, 300), (33, 65), (64, 64), (65, 64), (63, 129), (130, 70), (100, 1000), (517, 260),
         (256, 256), (300, 300), (128, 2048), (700, 390), (512, 512), (600, 770), (1024, 1024), (1030, 1290), (1300, 1025),
         (40, 9000), (130, 5000), (9001, 150), (600, 8200)]


@pytest.mark.parametrize("steps", [1, 2, 5])
@pytest.mark.parametrize("rows,cols", SIZES)
def test_orthogonalize_sizes(rows, cols, steps):
    dtype = torch.bfloat16 if (rows + steps) % 2 else torch.float32
    u = _matrix((rows, cols), 1000 * rows + cols, dtype)
    say(f"[muon] orthogonalize {rows}x{cols} {dtype} steps={steps}")
    got = muon.orthogonalize(u.cuda(), steps=steps)
    _check_orthogonal(f"{rows}x{cols} steps={steps}", got, u, steps=steps)


@pytest.mark.parametrize("rows,cols", [(2500, 8), (3900, 5), (2300, 4), (2600, 2), (4500, 8)])
def test_orthogonalize_long_and_very_narrow(rows, cols):
    """A wave of the load kernel goes over 32 or 64 rows of these at once, and the
    matrices are too long for one workgroup's LDS."""
    u = _matrix((rows, cols), rows + cols)
    _check_orthogonal(f"{rows}x{cols}", muon.orthogonalize(u.cuda()), u)


@pytest.mark.parametrize("rows,cols,batch", [(64, 64, 5), (40, 200, 3), (200, 40, 70), (260, 300, 3), (300, 20, 300), (1024, 1020, 15)])
def test_orthogonalize_batch(rows, cols, batch):
    u = _matrix((batch, rows, cols), rows, torch.bfloat16)
    u *= torch.logspace(-6, 6, batch).bfloat16()[:, None, None]   # each matrix has its own norm
    got = muon.orthogonalize(u.cuda())
    for b in {0, 1, batch // 2, batch - 1}:
        _check_orthogonal(f"batch {b} of {batch} {rows}x{cols}", got[b], u[b])
    # a matrix's result does not depend on the batch it is in
    one = muon.orthogonalize(u[batch - 1].cuda())
    assert torch.equal(one, got[batch - 1])


def test_orthogonalize_more_matrices_than_one_launch_takes():
    """2^21 of them go into one launch."""
    batch = (1 << 21) + 3
    u = _matrix((1, 2, 3), 6, torch.bfloat16).cuda().repeat(batch, 1, 1)
    u[-1] *= -1
    got = muon.orthogonalize(u)
    want = muon.orthogonalize(u[0])
    _check_orthogonal("2x3", want, u[0])
    assert bool((got[:-1] == want).all()) and torch.equal(got[-1], -want)


def test_orthogonalize_leading_dimensions_and_zero_sizes():
    u = _matrix((2, 3, 20, 50), 5)
    got = muon.orthogonalize(u.cuda())
    assert got.shape == u.shape
    _check_orthogonal("2x3 of 20x50", got[1, 2], u[1, 2])
    for shape in ((0, 4, 4), (3, 0, 4), (3, 4, 0)):
        assert muon.orthogonalize(torch.zeros(shape, device="cuda")).shape == shape


def test_orthogonalize_strided_input_and_output():
    big = _matrix((3, 90, 140), 8, torch.bfloat16).cuda()
    x = big[:, 5:75, 3:104]                       # 70 x 101, rows of 140, odd start
    _check_orthogonal("a view", muon.orthogonalize(x)[1], x[1])
    hold = torch.full((3, 80, 120), 7.0, dtype=torch.bfloat16, device="cuda")
    out = hold[:, 4:74, 9:110]
    muon.orthogonalize(x, out=out)
    assert torch.equal(out, muon.orthogonalize(x))
    hold[:, 4:74, 9:110] = 7.0
    assert bool((hold == 7.0).all()), "values around the output were changed"
    # one matrix read for the whole batch
    same = muon.orthogonalize(x[:1].expand(4, -1, -1))
    assert all(torch.equal(same[b], same[0]) for b in range(4))
    # in place
    y = x.contiguous()
    muon.orthogonalize(y, out=y)
    assert torch.equal(y, muon.orthogonalize(x.contiguous()))


@pytest.mark.parametrize("rows,heads,cols", [(96, 5, 20), (300, 3, 130), (700, 2, 72)])
def test_heads_that_are_column_blocks_of_one_matrix(rows, heads, cols):
    """Results and parameters written where the matrices' rows lie side by side."""
    whole = _matrix((rows, heads * cols + 8), 17, torch.bfloat16).cuda()
    x = whole[:, 4:4 + heads * cols].view(rows, heads, cols).transpose(0, 1)
    hold = torch.full_like(whole, 7.0)
    out = hold[:, 4:4 + heads * cols].view(rows, heads, cols).transpose(0, 1)
    muon.orthogonalize(x, out=out)
    assert torch.equal(out, muon.orthogonalize(x.contiguous()))
    assert bool((hold[:, :4] == 7.0).all()) and bool((hold[:, 4 + heads * cols:] == 7.0).all())
    m = torch.zeros(x.shape, device="cuda")
    p, m2 = out.contiguous(), torch.zeros_like(m)
    muon.muon_step(out, x, m, lr=0.1, wd=0.1)
    muon.muon_step(p, x.contiguous(), m2, lr=0.1, wd=0.1)
    assert torch.equal(out, p) and torch.equal(m, m2)
    assert bool((hold[:, :4] == 7.0).all()) and bool((hold[:, 4 + heads * cols:] == 7.0).all())
    codes, scales = torch.zeros_like(m, dtype=torch.int8), torch.zeros(muon.scales_shape(m.shape), device="cuda")
    codes2, scales2 = codes.clone(), scales.clone()
    muon.muon8_step(out, x, codes, scales, lr=0.1, wd=0.1)
    muon.muon8_step(p, x.contiguous(), codes2, scales2, lr=0.1, wd=0.1)
    assert torch.equal(out, p) and torch.equal(codes, codes2) and torch.equal(scales, scales2)


@pytest.mark.parametrize("size", [1e-30, 1e-19, 1e19, 3e36])
def test_orthogonalize_any_magnitude(size):
    u = _matrix((70, 90), 11) * size * 1e3
    _check_orthogonal(f"entries about {size}", muon.orthogonalize(u.cuda(), eps=1e-37), u, eps=1e-37)


def test_orthogonalize_small_norm_is_divided_by_eps():
    u = _matrix((40, 60), 12, size=1e-6)
    _check_orthogonal("eps above the norm", muon.orthogonalize(u.cuda(), eps=0.25), u, eps=float(np.float32(0.25)))


@pytest.mark.parametrize("rows,cols", [(64, 64), (300, 200)])
def test_orthogonalize_zero_and_non_finite_matrices(rows, cols):
    u = _matrix((5, rows, cols), 13)
    u[0] = 0
    u[1, 3, 4] = float("nan")
    u[2, rows - 1, cols - 1] = float("inf")
    u[3, 0, 0] = -float("inf")
    got = muon.orthogonalize(u.cuda()).cpu()
    assert bool((got[0] == 0).all())
    assert all(bool(got[b].isnan().all()) for b in (1, 2, 3))
    _check_orthogonal("beside them", got[4], u[4])


def test_orthogonalize_sparse_matrix():
    # one entry holds the whole norm; rank one; one row; a diagonal
    u = torch.zeros(4, 96, 160)
    u[0, 95, 159] = -3.0
    u[1] = torch.linspace(-1, 1, 96)[:, None] * torch.linspace(0.5, 1, 160)
    u[2, 40] = _matrix((160,), 3)
    u[3, torch.arange(96), torch.arange(96)] = torch.linspace(0.1, 1, 96)
    got = muon.orthogonalize(u.cuda())
    for b in range(4):
        _check_orthogonal(f"sparse {b}", got[b], u[b], worst=True)


@pytest.mark.parametrize("steps", [2, 3, 4, 6, 7])
@pytest.mark.parametrize("rows,cols", [(16, 900), (60, 700), (140, 4100), (2600, 520)])
def test_orthogonalize_pairs_of_steps(rows, cols, steps):
    u = _matrix((rows, cols), 15 * steps)
    _check_orthogonal(f"{rows}x{cols} steps={steps}", muon.orthogonalize(u.cuda(), steps=steps), u, steps=steps)


def test_orthogonalize_coefficients_for_each_step():
    ks = ((4.0, -6.9, 2.9), (3.4445, -4.7750, 2.0315), (1.875, -1.25, 0.375))
    for shape in ((90, 130), (40, 600), (150, 4000)):
        u = _matrix(shape, 14)
        _check_orthogonal("three triples", muon.orthogonalize(u.cuda(), steps=3, coefficients=ks), u, steps=3, coefficients=ks)
    _check_orthogonal("cubic", muon.orthogonalize(u.cuda(), steps=12, coefficients=(1.5, -0.5, 0.0)), u, steps=12,
                      coefficients=(1.5, -0.5, 0.0))


def _muon_reference(p, g, m, lr, beta, wd, nesterov, scale):
    """One step in 64 bits: (params, momentum, U, bound on the orthogonalized U's error)."""
    m = beta * m + (1 - beta) * g
    u = beta * m + (1 - beta) * g if nesterov else m
    x, err = R.orthogonalized(u)
    return p * (1 - lr * wd) - lr * scale * x, m, err


@pytest.mark.parametrize("rows,cols,dtype,nesterov,wd", [
    (64, 64, torch.float32, True, 0.0), (100, 333, torch.float32, False, 0.1), (333, 100, torch.float32, True, 0.1),
    (257, 515, torch.bfloat16, True, 0.1), (515, 64, torch.bfloat16, False, 0.0), (1, 40, torch.float32, True, 0.1),
    (16, 700, torch.float32, True, 0.0)])
@pytest.mark.parametrize("bits", [32, 8])
def test_muon_steps(rows, cols, dtype, nesterov, wd, bits):
    """Three steps; each is checked from the state that the kernels left."""
    batch, lr, beta, scale = 2, 0.5, 0.9, 1.5
    p = _matrix((batch, rows, cols), 21, dtype, 0.02).cuda()
    mom = torch.zeros(batch, rows, cols, device="cuda")
    codes = torch.zeros(batch, rows, cols, dtype=torch.int8, device="cuda")
    scales = torch.zeros(muon.scales_shape(codes.shape), device="cuda")
    for t in range(3):
        g = _matrix((batch, rows, cols), 22 + t, torch.bfloat16)
        say(f"[muon] step {t}: {rows}x{cols} {dtype} bits={bits}")
        before = p.cpu().double()
        old = mom.cpu().double() if bits == 32 else R.values(codes.cpu(), scales.cpu())
        kw = dict(lr=lr, beta=beta, wd=wd, nesterov=nesterov, scale=scale)
        if bits == 32:
            muon.muon_step(p, g.cuda(), mom, **kw)
        else:
            muon.muon8_step(p, g.cuda(), codes, scales, **kw)
        for b in range(batch):
            want, m, err = _muon_reference(before[b], g[b].double(), old[b], lr, beta, wd, nesterov, scale)
            if bits == 32:
                # two products and a sum, each rounded to fp32 (beta too)
                tol = 3 * R.FP32 * (beta * old[b].abs() + (1 - beta) * g[b].double().abs()) + R.FP32 * m.abs()
                assert bool(((mom[b].cpu().double() - m).abs() <= tol).all())
            else:
                qc, qs = R.quantized(m)
                assert torch.equal(scales[b].cpu(), qs)
                assert torch.equal(codes[b].cpu(), qc)
            off = (p[b].cpu().double() - want).norm().item()
            # U in fp32 is off by 2^-22 at most, far below the products' roundings
            tol = lr * scale * err * (1 + 2 ** -6)
            tol += (R.BF16 if dtype == torch.bfloat16 else 4 * R.FP32) * (want.norm().item() + tol)
            assert off <= tol, (off, tol)


@pytest.mark.parametrize("steps", [1, 2, 3, 5])
@pytest.mark.parametrize("rows,cols", [(300, 2400), (2400, 300), (440, 6000), (6000, 440), (130, 5000)])
def test_muon_step_on_wide_matrices_of_few_steps(rows, cols, steps):
    """fp32 parameters show the products' roundings, those of the last product's
    diagonal too: nothing of them is hidden by a result in bf16."""
    p = _matrix((rows, cols), 45, size=0.02)
    g = _matrix((rows, cols), 46, torch.bfloat16)
    want, err = R.orthogonalized(g, steps=steps)
    got, m = p.cuda(), torch.zeros(rows, cols, device="cuda")
    muon.muon_step(got, g.cuda(), m, lr=0.5, wd=0.1, beta=0.0, nesterov=False, scale=2.0, steps=steps)
    want = p.double() * 0.95 - want
    off, tol = (got.cpu().double() - want).norm().item(), err + 4 * R.FP32 * (want.norm().item() + err)
    say(f"[muon] {rows}x{cols} steps={steps}: off {off:.2e}, allowed {tol:.2e}")
    assert off <= tol


def test_muon8_non_finite_block_and_short_block():
    rows, cols = 3, 600                               # blocks of 256, 256 and 88
    g = _matrix((rows, cols), 31, torch.bfloat16)
    g[1, 300] = float("inf")
    g[2, 520:] = 0
    codes = torch.zeros(rows, cols, dtype=torch.int8, device="cuda")
    scales = torch.zeros(rows, 3, device="cuda")
    p = torch.zeros(rows, cols, device="cuda")
    muon.muon8_step(p, g.cuda(), codes, scales, beta=0.9)
    qc, qs = R.quantized(0.09999999999999998 * g.double())
    assert torch.equal(codes.cpu(), qc)
    assert torch.equal(scales.cpu().nan_to_num(-1.0), qs.nan_to_num(-1.0)) and bool(scales[1, 1].isnan())
    assert bool(p.isnan().all())                      # the matrix is one product
    v = muon.momentum8_values(codes, scales).cpu()
    assert bool(v[1, 256:512].isnan().all()) and int(v.isnan().sum()) == 256
    fine = ~v.isnan()
    assert torch.equal(v[fine], (codes.cpu().float() * qs.repeat_interleave(256, 1)[:, :cols])[fine])


@pytest.mark.parametrize("cols", [256, 2560])
def test_muon8_a_value_between_two_codes_takes_the_even_one(cols):
    """With beta = 1/2 a block of scale 2 d keeps its largest code, 127, and has
    the scale d afterwards; m = (k + 1/2) d is exactly between two codes.  The
    sum, the scale and the quotient are exact, so the codes must be equal.  (For
    d = 49, k = 1 the product with 1/d in 64 bits falls short of 3/2.)"""
    scale = [49, 161, 97, 113, 1.75, 161 * 2.0 ** -12, 125, 0.921875]
    codes, want, g = (torch.zeros(len(scale), cols, dtype=t) for t in (torch.int8, torch.int8, torch.bfloat16))
    for r, d in enumerate(scale):
        codes[r, ::256], want[r, ::256] = 127, 127
        at = 1
        for k in range(-127, 127):
            # m = code d + g / 2
            for code in range(-127, 128):
                e = (2 * k + 1 - 2 * code) * d
                if code != 0 and abs(e) <= 128 * d and float(torch.tensor(e).bfloat16()) == e:
                    codes[r, at], g[r, at], want[r, at] = code, e, 2 * round((2 * k + 1) / 4)   # the even neighbour
                    at += 1
                    break
            else:
                continue
            if at == 256:
                break
        assert at > 100
    scales = 2 * torch.tensor(scale).repeat_interleave(cols // 256).reshape(len(scale), -1)
    m = 0.5 * R.values(codes, scales) + 0.5 * g.double()
    qc, qs = R.quantized(m)
    assert torch.equal(qc, want) and torch.equal(qs, scales / 2)
    p, codes, scales = torch.zeros(want.shape, device="cuda"), codes.cuda(), scales.cuda()
    muon.muon8_step(p, g.cuda(), codes, scales, beta=0.5)
    assert torch.equal(scales.cpu(), qs)
    assert torch.equal(codes.cpu(), qc)


@pytest.mark.parametrize("shape", [(5,), (1, 1), (3, 255), (2, 7, 512), (300, 1001)])
def test_momentum8_values(shape):
    g = torch.Generator().manual_seed(3)
    codes = torch.randint(-127, 128, shape, generator=g, dtype=torch.int8).cuda()
    scales = torch.rand(muon.scales_shape(shape), generator=g).cuda()
    want = codes.float() * scales.repeat_interleave(256, -1)[..., : shape[-1]]
    assert torch.equal(muon.momentum8_values(codes, scales), want)
    assert muon.momentum8_values(codes[:0], scales[:0]).numel() == 0


def test_muon_step_writes_only_its_parameters():
    hold = _matrix((2, 50, 90), 41).cuda()
    p, keep = hold[:, 3:40, 5:80], hold.clone()
    g = _matrix((2, 60, 100), 42, torch.bfloat16).cuda()[:, 10:47, 11:86]
    m = torch.zeros(2, 37, 75, device="cuda")
    p2, m2 = p.contiguous(), torch.zeros_like(m)
    muon.muon_step(p, g, m, lr=0.1, wd=0.1)
    muon.muon_step(p2, g.contiguous(), m2, lr=0.1, wd=0.1)
    assert torch.equal(p, p2) and torch.equal(m, m2)
    hold[:, 3:40, 5:80] = keep[:, 3:40, 5:80]
    assert torch.equal(hold, keep)


def test_autograd_sees_what_a_call_wrote():
    x = torch.ones(20, 20, device="cuda", requires_grad=True)
    g = _matrix((20, 20), 43, torch.bfloat16).cuda()
    p, m = torch.ones(20, 20, device="cuda"), torch.zeros(20, 20, device="cuda")
    codes, scales = torch.zeros(20, 20, dtype=torch.int8, device="cuda"), torch.zeros(20, 1, device="cuda")
    out, values = torch.ones(20, 20, dtype=torch.bfloat16, device="cuda"), torch.ones(20, 20, device="cuda")
    for t, call in ((p, lambda: muon.muon_step(p, g, m)), (m, lambda: muon.muon_step(p, g, m)),
                    (p, lambda: muon.muon8_step(p, g, codes, scales)), (scales, lambda: muon.muon8_step(p, g, codes, scales)),
                    (out, lambda: muon.orthogonalize(g, out=out)), (values, lambda: muon.momentum8_values(codes, scales, out=values))):
        y = (x * t).sum()
        before = codes._version
        call()
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            y.backward()
    assert before > 0
    # read only: as it was
    y = (x * g).sum()
    muon.muon_step(p, g, m)
    muon.orthogonalize(g)
    y.backward()
    with torch.inference_mode():
        q = torch.ones(20, 20, device="cuda")
        muon.muon_step(q, g, m)


def test_muon_captured_graphs_replay_as_eager_steps():
    """Two captured graphs (32- and 8-bit) replayed in turn with eager work
    between, each replay against an eager step from the same state."""
    shape = (2, 130, 200)
    g = _matrix(shape, 51, torch.bfloat16).cuda()
    p = [_matrix(shape, 52, size=0.02).cuda() for _ in range(2)]
    mom = torch.zeros(shape, device="cuda")
    codes, scales = torch.zeros(shape, dtype=torch.int8, device="cuda"), torch.zeros(muon.scales_shape(shape), device="cuda")
    q = [t.clone() for t in p]
    mom2, codes2, scales2 = mom.clone(), codes.clone(), scales.clone()
    graphs = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()]
    with torch.cuda.graph(graphs[0]):
        muon.muon_step(p[0], g, mom, lr=0.1)
    with torch.cuda.graph(graphs[1]):
        muon.muon8_step(p[1], g, codes, scales, lr=0.1)
    for t in range(4):
        g.copy_(_matrix(shape, 60 + t, torch.bfloat16))
        graphs[0].replay()
        graphs[1].replay()
        muon.muon_step(q[0], g, mom2, lr=0.1)
        muon.muon8_step(q[1], g, codes2, scales2, lr=0.1)
        torch.cuda.synchronize()
        assert torch.equal(p[0], q[0]) and torch.equal(mom, mom2)
        assert torch.equal(p[1], q[1]) and torch.equal(codes, codes2) and torch.equal(scales, scales2)


@pytest.mark.parametrize("shape", [(3, 40, 200), (2, 700, 390), (1, 200, 5000)])
def test_orthogonalize_captured_and_replayed(shape):
    """One workgroup to a matrix; launches of a tall batch; pairs of steps with
    the long sums in parts."""
    x = _matrix(shape, 53, torch.bfloat16).cuda()
    out = torch.zeros_like(x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        muon.orthogonalize(x, out=out)
    for t in range(4):
        x.copy_(_matrix(shape, 54 + t, torch.bfloat16))
        want = muon.orthogonalize(x)
        graph.replay()
        other = muon.orthogonalize(x.float())     # eager work beside the replay
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(other, want)


def test_muon_on_another_stream():
    x = [_matrix((200, 300), 71 + k, torch.bfloat16).cuda() for k in range(4)]
    want = [muon.orthogonalize(t) for t in x]
    streams = [torch.cuda.Stream() for _ in range(4)]
    torch.cuda.synchronize()
    got = [torch.empty_like(t) for t in x]
    for _ in range(3):
        for k in range(4):
            muon.orthogonalize(x[k], out=got[k], stream=streams[k])
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_muon_results_are_allocated_on_the_stream_that_writes_them():
    """Memory that the current stream has given back may still be in use there:
    a result written by another stream must not lie in it."""
    x = _matrix((200, 300), 75, torch.bfloat16).cuda()
    codes, scales = torch.ones(200, 300, dtype=torch.int8, device="cuda"), torch.ones(200, 2, device="cuda")
    want = muon.orthogonalize(x), muon.momentum8_values(codes, scales)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for call, ref in ((lambda: muon.orthogonalize(x, stream=side), want[0]),
                      (lambda: muon.momentum8_values(codes, scales, stream=side), want[1])):
        free = torch.empty_like(ref)
        at = free.data_ptr()
        del free
        got = call()
        assert got.data_ptr() != at
        torch.cuda.synchronize()
        assert torch.equal(got, ref)


def test_muon_same_inputs_give_the_same_bits():
    u = _matrix((3, 390, 520), 81).cuda()
    first = muon.orthogonalize(u)
    for _ in range(3):
        assert torch.equal(muon.orthogonalize(u), first)


def test_muon_offsets_past_32_bits():
    """The longest side with more than 2^31 elements.  The formula is taken on the
    short side in 64 bits, X = U F(U^T U), and compared on rows at both ends and
    in between.  Tolerance: five steps of three roundings of 2^-11, each grown at
    most fivefold (s f'(s) / f(s) of a step's f on 0..1.2), and the result's 2^-8;
    an offset that lost its upper bits would be off by the whole value."""
    rows, cols = 1 << 21, 1040
    gen = torch.Generator(device="cuda").manual_seed(91)
    u = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda")
    a = torch.zeros(cols, cols, dtype=torch.float64, device="cuda")
    for part in u.split(1 << 17):
        part.normal_(generator=gen)
        wide = part.double()
        a += wide.T.contiguous() @ wide
    say("[muon] 2^21 x 1040: inputs made")
    got = muon.orthogonalize(u)
    norm = a.trace().sqrt()
    a = (a / norm ** 2).cpu()
    f = torch.eye(cols, dtype=torch.float64)
    for _ in range(5):
        ka, kb, kc = muon.COEFFICIENTS
        p = ka * torch.eye(cols, dtype=torch.float64) + kb * a + kc * a @ a
        f, a = p @ f, p @ a @ p
    f /= norm.cpu()
    tol = 15 * 5 * 2.0 ** -11 + R.BF16
    for at in (0, 1 << 20, (1 << 31) // cols, rows - 64):
        want = u[at:at + 64].cpu().double() @ f
        off = (got[at:at + 64].cpu().double() - want).norm() / want.norm()
        say(f"[muon] rows {at}..: off {off:.2e}, allowed {tol:.2e}")
        assert off <= tol
    # a step from nothing, with the whole gradient as its momentum, gives the same
    params = torch.zeros_like(u)
    codes = torch.zeros(rows, cols, dtype=torch.int8, device="cuda")
    scales = torch.zeros(muon.scales_shape(codes.shape), device="cuda")
    muon.muon8_step(params, u, codes, scales, lr=1.0, beta=0.0, nesterov=False, scale=-1.0)
    for x, y in zip(params.split(1 << 17), got.split(1 << 17)):
        assert torch.equal(x, y)
    for at in (0, (1 << 31) // cols, rows - 8):
        qc, qs = R.quantized(u[at:at + 8].cpu().double())
        assert torch.equal(codes[at:at + 8].cpu(), qc) and torch.equal(scales[at:at + 8].cpu(), qs)
    values = muon.momentum8_values(codes, scales)
    want = codes[-8:].float() * scales[-8:].repeat_interleave(256, 1)[:, :cols]
    assert torch.equal(values[-8:], want)


def test_muon_refusals_on_the_gpu():
    p = torch.zeros(4, 6, device="cuda")
    g = torch.zeros(4, 6, dtype=torch.bfloat16, device="cuda")
    m = torch.zeros(4, 6, device="cuda")
    with pytest.raises(ValueError):
        muon.muon_step(p.T, g.T, m.T)                 # last dimension not contiguous
    with pytest.raises(ValueError):
        muon.muon_step(p, g.float(), m)
    with pytest.raises(ValueError):
        muon.muon_step(p, g, m[:, :3])
    with pytest.raises(ValueError):
        muon.muon_step(p.half(), g, m)
    with pytest.raises(ValueError):
        muon.muon8_step(p, g, m.to(torch.int8), torch.zeros(4, 2, device="cuda"))
    with pytest.raises(ValueError):
        muon.orthogonalize(p, out=torch.zeros(4, 6, device="cuda"))
    with pytest.raises(ValueError):
        muon.orthogonalize(p, steps=2, coefficients=((1.5, -0.5, 0.0),))
    for bad in (dict(beta=1.0), dict(wd=-1.0), dict(lr=math.nan), dict(eps=0.0), dict(steps=65),
                dict(coefficients=(9.0, 0.0, 0.0)), dict(coefficients=(math.nan, 0.0, 0.0))):
        with pytest.raises(muon._L.MicroAdamError) as e:
            muon.muon_step(p, g, m, **bad)
        assert e.value.code == muon._L.MA_EINVAL
    shared = torch.zeros(6, device="cuda").expand(4, 6)
    with pytest.raises(muon._L.MicroAdamError):
        muon.muon_step(shared, g, m)                  # rows of the parameters overlap
    assert not p.any() and not m.any()
