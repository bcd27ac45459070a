"""GPU tests of the Muon calls on batches that between them use every kernel for
products (tests/muon_cases.py), with parameters, momentum and decay that are not
zero, against the formulas in 64 bits."""
import pytest
import torch

import muon_cases as M
import muon_reference as R
from gpu_harness import say
from memory_compressed_adaptive_amd import muon

pytestmark = pytest.mark.gpu

LR, BETA, WD, SCALE = 0.5, 0.9, 0.1, 1.5


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _normal(shape, seed, dtype=torch.float32, size=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (size * torch.randn(shape, generator=g, device="cuda")).to(dtype)


def _close(what, off, tol, size):
    say(f"[muon] {what}: off {off / size:.2e}, allowed {tol / size:.2e}")
    assert off <= tol, what


def _checked(case):
    """Matrices that are compared: the first and the last of every run."""
    return sorted({at for run in M.runs(*case) for at in run})


@pytest.mark.parametrize("case", M.CASES, ids=str)
def test_orthogonalize(case):
    x = _normal(case, case[1], torch.bfloat16, 1e-3)
    x *= torch.logspace(-6, 6, case[0], device="cuda").bfloat16()[:, None, None]
    got = muon.orthogonalize(x)
    for b in _checked(case):
        want, err = R.orthogonalized_large(x[b])
        size = want.norm().item()
        _close(f"{case} matrix {b}", (got[b].double() - want).norm().item(), err + R.BF16 * (size + err), size)


@pytest.mark.parametrize("case", M.CASES, ids=str)
@pytest.mark.parametrize("bits,dtype,nesterov", [(32, torch.float32, True), (8, torch.bfloat16, False)])
def test_steps_from_a_state(case, bits, dtype, nesterov):
    p, g = _normal(case, 1, dtype, 0.02), _normal(case, 2, torch.bfloat16, 1e-3)
    old = _normal(case, 3, size=1e-3)
    look = _checked(case)
    kw = dict(lr=LR, beta=BETA, wd=WD, nesterov=nesterov, scale=SCALE)
    before = {b: p[b].double() for b in look}
    if bits == 32:
        new = old
        old = {b: old[b].double() for b in look}
        muon.muon_step(p, g, new, **kw)
    else:
        # any codes and scales are a state; the largest code of a block need not be 127
        codes = (64 * old / 1e-3).clamp(-127, 127).to(torch.int8)
        g8 = torch.Generator(device="cuda").manual_seed(4)
        scales = 1e-3 / 64 * (1 + torch.rand(muon.scales_shape(case), generator=g8, device="cuda"))
        old = {b: R.values(codes[b].cpu(), scales[b].cpu()).cuda() for b in look}
        muon.muon8_step(p, g, codes, scales, **kw)
    for b in look:
        gb = g[b].double()
        m = BETA * old[b] + (1 - BETA) * gb
        if bits == 32:
            # two products and a sum, each rounded to fp32 (beta too)
            tol = 3 * R.FP32 * (BETA * old[b].abs() + (1 - BETA) * gb.abs()) + R.FP32 * m.abs()
            assert bool(((new[b].double() - m).abs() <= tol).all())
        else:
            qc, qs = R.quantized(m.cpu())
            assert torch.equal(scales[b].cpu(), qs) and torch.equal(codes[b].cpu(), qc)
        x, err = R.orthogonalized_large(BETA * m + (1 - BETA) * gb if nesterov else m)
        want = before[b] * (1 - LR * WD) - LR * SCALE * x
        # U in fp32 is off by 2^-22 at most, far below the products' roundings
        tol = LR * SCALE * err * (1 + 2 ** -6)
        tol += (R.BF16 if dtype == torch.bfloat16 else 4 * R.FP32) * (want.norm().item() + tol)
        _close(f"{case} {bits} bits, matrix {b}", (p[b].double() - want).norm().item(), tol, LR * SCALE * x.norm().item())


def _with_spectrum(rows, cols, s, seed):
    """A matrix of these singular values, its singular vectors random."""
    n = len(s)
    g = torch.Generator().manual_seed(seed)
    left = torch.linalg.qr(torch.randn(rows, n, generator=g, dtype=torch.float64)).Q
    right = torch.linalg.qr(torch.randn(cols, n, generator=g, dtype=torch.float64)).Q
    return (left * torch.as_tensor(s, dtype=torch.float64)) @ right.T


SPECTRA = {
    "1/k": lambda n: 1.0 / torch.arange(1, n + 1),
    "two orders": lambda n: torch.logspace(0, -2, n),
    "one large": lambda n: torch.cat([torch.ones(1), torch.full((n - 1,), 0.02)]),
    "flat": torch.ones,
    "low rank": lambda n: torch.ones(n // 8),
}


@pytest.mark.parametrize("steps", [1, 2, 5])
@pytest.mark.parametrize("spectrum", SPECTRA)
@pytest.mark.parametrize("rows,cols", [(96, 160), (300, 330), (200, 1200), (1200, 200), (700, 1500)])
def test_orthogonalize_structured_spectra(rows, cols, spectrum, steps):
    """One workgroup to a matrix; products with steps one by one and in twos."""
    u = _with_spectrum(rows, cols, SPECTRA[spectrum](min(rows, cols)), rows).float().cuda()
    want, err = R.orthogonalized_large(u, steps=steps)
    size = want.norm().item()
    if spectrum == "flat":   # the diagonals of A and P do not average out
        err += R.flat_worst(min(rows, cols), steps) * size
    off = (muon.orthogonalize(u, steps=steps).double() - want).norm().item()
    _close(f"{rows}x{cols} {spectrum} steps={steps}", off, err + R.BF16 * (size + err), size)


def _special(which, rows, cols):
    u = torch.zeros(rows, cols)
    if which == "entry":
        u[rows - 1, cols - 1] = -3.0
    elif which == "row":
        u[rows // 2] = torch.linspace(-1, 2, cols)
    elif which == "column":
        u[:, cols // 2] = torch.linspace(-1, 2, rows)
    elif which == "diagonal":
        at = torch.arange(min(rows, cols))
        u[at, at] = torch.linspace(0.1, 1, min(rows, cols))
    elif which == "rank one":
        u[:] = torch.linspace(-1, 1, rows)[:, None] * torch.linspace(0.5, 1, cols)
    else:
        u[:64, :64] = 1.0
        u[64:130, 70:140] = -2.0
    return u


# what falls to rounding in the worst case grows fast with the steps
@pytest.mark.parametrize("which,steps", [("entry", 1), ("entry", 2), ("row", 1), ("row", 2), ("column", 1), ("diagonal", 1), ("diagonal", 2),
                                         ("diagonal", 3), ("rank one", 1), ("blocks", 1)])
@pytest.mark.parametrize("rows,cols", [(300, 330), (200, 1200), (1200, 200), (700, 1500)])
def test_orthogonalize_special_matrices(rows, cols, which, steps):
    """Singular vectors that are not spread over the entries, where roundings need
    not average out."""
    u = _special(which, rows, cols) if rows <= cols else _special(which, cols, rows).T.contiguous()
    want, err = R.orthogonalized_worst(u, steps=steps)
    size = want.norm().item()
    off = (muon.orthogonalize(u.cuda(), steps=steps).cpu().double() - want).norm().item()
    _close(f"{rows}x{cols} {which} steps={steps}", off, err + R.BF16 * (size + err), size)
