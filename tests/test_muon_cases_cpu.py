"""The sizes of the GPU tests reach every kernel for products, and the refusals of
the call that tells."""
import ctypes as C
import math
import random

import pytest
import torch

import muon_cases as M
import muon_reference as R
from memory_compressed_adaptive_amd import _lib as L


def test_the_cases_reach_every_product_kernel():
    rng = random.Random(1)
    log = lambda lo, hi: int(math.exp(rng.uniform(math.log(lo), math.log(hi))))  # noqa: E731
    reached = set()
    for _ in range(60000):
        batch, rows, cols = rng.choice([1, 1, 2, 3, 4, log(1, 200)]), log(8, 16000), log(8, 16000)
        reached |= M.kernels(batch, rows, cols)
    tested = set().union(*(M.kernels(*case) for case in M.CASES))
    assert reached - tested == set()
    # all six tiles in every role but X Xt in parts, which stops at 128
    assert len(tested) == 6 * 6 + 3


def test_the_cases_reach_several_runs():
    several = [(case, M.plan(*case), M.runs(*case)) for case in M.CASES if len(M.runs(*case)) > 1]
    assert {(p["tall"], p["pairs"]) for _, p, _ in several} >= {(0, 0), (0, 1), (1, 0), (1, 1)}
    assert any(r[-1][1] - r[-1][0] < r[0][1] - r[0][0] for _, _, r in several)
    for (batch, _, _), _, r in several:
        assert r[0][0] == 0 and r[-1][1] == batch - 1


def test_plan_refuses():
    fn, out = L.lib().ma_debug_muon_plan, (C.c_int64 * 9)()
    assert fn(1, 4, 4, None) == L.MA_EINVAL
    assert fn(0, 4, 4, out) == L.MA_EINVAL and fn(1, 0, 4, out) == L.MA_EINVAL and fn(1, 4, -1, out) == L.MA_EINVAL
    assert fn(1, 1 << 40, 4, out) == L.MA_EUNSUPPORTED
    assert fn(1, 64, 64, out) == L.MA_OK and list(out) == [1, 0, 0, 0, 0, 0, 0, 0, 0]


@pytest.mark.parametrize("shape", [(1, 64, 64), (144, 64, 768), (24, 2048, 16)])
def test_one_workgroup_matrices_have_no_products(shape):
    assert M.kernels(*shape) == set() and M.runs(*shape) == [(0, shape[0] - 1)]


def _rounded(u, steps, pairs, mistake=False):
    """The steps with X, A, P and the products of two steps rounded to fp16 here."""
    half = lambda t, s: (t * s).half().double() / s  # noqa: E731
    poly = lambda t, g: half(t[0] * eye + t[1] * g + t[2] * g @ g, 2.0 ** 12)  # noqa: E731
    ks, eye = R.triples(R.COEFFICIENTS, steps), torch.eye(u.shape[0], dtype=torch.float64)
    x, t = half(u / u.norm(), 2.0 ** 14), 0
    single = (steps // 2 + 1) // 2 * 2 if steps % 2 else -1
    while t < steps:
        gram = half(x @ x.T, 2.0 ** 14)
        if mistake:
            gram[-1, -1] = 0.0
        f = poly(ks[t], gram)
        if pairs and t != single:
            gram = half(half(f @ gram, 2.0 ** 12) @ f, 2.0 ** 14)
            f = half(poly(ks[t + 1], gram) @ f, 2.0 ** 8)
            t += 1
        x = half(f @ x, 2.0 ** 14)
        t += 1
    return x


def _special(which):
    u = torch.zeros(40, 90, dtype=torch.float64)
    if which == "entry":
        u[39, 89] = -3.0
    elif which == "row":
        u[39] = torch.linspace(-1, 2, 90)
    elif which == "diagonal":
        u[torch.arange(40), torch.arange(40)] = torch.linspace(0.1, 1, 40, dtype=torch.float64)
    else:
        u[:] = torch.linspace(-1, 1, 40)[:, None] * torch.linspace(0.5, 1, 90)
    return u


@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("which,steps", [("entry", 1), ("entry", 2), ("row", 1), ("row", 2), ("diagonal", 1), ("diagonal", 2),
                                         ("diagonal", 3), ("rank one", 1)])
def test_worst_bound_holds_for_roundings_made_on_the_cpu(which, steps, pairs):
    u = _special(which)
    want, err = R.orthogonalized_worst(u, steps=steps)
    assert err < 0.25 * want.norm().item()
    # what _rounded takes off the result itself is not in the bound
    assert (_rounded(u, steps, pairs) - want).norm().item() <= err + R.H * want.norm().item()
    # one element of A forgotten
    assert (_rounded(u, steps, pairs, mistake=True) - want).norm().item() > err


@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("steps", [1, 2, 5])
def test_flat_bound_holds_for_roundings_made_on_the_cpu(steps, pairs):
    flat = torch.linalg.qr(torch.randn(90, 40, dtype=torch.float64, generator=torch.Generator().manual_seed(1))).Q.T
    want, err = R.orthogonalized_large(flat, steps=steps)
    err += R.flat_worst(40, steps) * want.norm().item()
    assert (_rounded(flat, steps, pairs) - want).norm().item() <= err


def test_references_agree():
    g = torch.Generator().manual_seed(3)
    for shape in ((40, 90), (90, 40), (64, 64)):
        u = torch.randn(shape, generator=g, dtype=torch.float64)
        want, err = R.orthogonalized(u)
        large, err2 = R.orthogonalized_large(u)
        assert torch.allclose(large, want, rtol=0, atol=1e-12) and abs(err2 - err) <= 1e-6 * err
        assert torch.allclose(R.orthogonalized_worst(u)[0], want, rtol=0, atol=1e-12)
