"""The Muon operators in 64 bits, straight from their formulas, and how far the
kernels may be from them: bounds that follow from where they round.

One step maps X to p(X) = a X + b (X X^T) X + c (X X^T)^2 X, which acts on the
singular values alone.  The kernels round X, A = X X^T and P = a I + b A + c A A
to fp16: at most h = 2^-11 of each entry, h / sqrt(3) of it in the root mean
square of a rounding that falls anywhere.  fp32 sums of K products add about
sqrt(K) 2^-24 of the factors' norms, 2^-18 at K = 4096; h is taken 1/16 larger
for that and for second-order terms.

Worst case.  The map moves a perturbation of X by at most L times its 2-norm
(over all entries), L the largest |p'(s)| for 0 <= s <= |X|_2, so that with
s = |X|_2

    E' <= L (E + h |X|) + h s ((|b| + 2 |c| s^2) |A| + |P|).

It adds five steps' largest values up and comes to half the result's norm.

Random roundings.  In the basis of X's singular vectors, which every step keeps,
a perturbation e moves the end by: its part even under i <-> j times
S_ij = (F(s_i) - F(s_j)) / (s_i - s_j), its odd part times T_ij = (F(s_i) +
F(s_j)) / (s_i + s_j), F the remaining steps' polynomials one after the other,
and what lies outside the square part times F(s_i) / s_i.  A rounding of X has
entries of variance h^2/3 |X|^2 / (n m) there; one of P adds e_ij = d_ij s_j and
one of A e_ij = (b + c (s_i^2 + s_j^2)) d_ij s_j, with d symmetric.  Summed over
entries and steps this is the expected square of the error; FOUR times its root
is allowed.  This takes singular vectors that are spread over the entries: it is
used for random matrices, the worst case for special ones.

Two steps may be taken together: T = P1 A, the next A as T P1, Q = P2 P1 and the
second next X as Q X, with T, A and Q rounded to fp16 and the X between them not.
A rounding of Q acts like one of P2 would on P1 X, but with |Q| for |P2| and the
first X's singular values; one of T moves the next A by d_ij p1_j, one of P1 by
d_ij (A_j p1_j + A_i p1_i) (A, p1: eigenvalues), on top of its own rounding.  The
bound counts these and the roundings of the steps one by one.
"""
import torch

COEFFICIENTS = (3.4445, -4.7750, 2.0315)
H = 2.0 ** -11 * (1 + 1 / 16)
BF16 = 2.0 ** -8
FP32 = 2.0 ** -24
FOUR = 4.0


def triples(coefficients, steps):
    rows = coefficients if hasattr(coefficients[0], "__len__") else [coefficients] * steps
    # the coefficients reach the kernels as fp32 numbers
    return [tuple(torch.tensor(r, dtype=torch.float32).double().tolist()) for r in rows]


def _odd(s, ks):
    """The composed odd polynomial at s, and its derivative."""
    d = torch.ones_like(s)
    for a, b, c in ks:
        d = d * (a + 3 * b * s ** 2 + 5 * c * s ** 4)
        s = s * (a + b * s ** 2 + c * s ** 4)
    return s, d


def _moves(s, ks):
    """(S, T, F(s)/s) of the steps ks for singular values s > 0."""
    f, d = _odd(s, ks)
    gap, tot = s[:, None] - s[None, :], s[:, None] + s[None, :]
    near = gap.abs() < 1e-9
    even = torch.where(near, (d[:, None] + d[None, :]) / 2, (f[:, None] - f[None, :]) / torch.where(near, 1.0, gap))
    return even, (f[:, None] + f[None, :]) / tot, f / s


def _random(s, n, m, ks):
    total = 0.0
    for t, (a, b, c) in enumerate(ks):
        even, odd, out = _moves(s, ks[t:])
        var = H ** 2 / 3 * (s ** 2).sum() / (n * m)
        total += var * ((even ** 2 + odd ** 2).sum() / 2 + (m - n) * (out ** 2).sum())
        nxt, _ = _odd(s, ks[t:t + 1])
        even, odd, _ = _moves(nxt.abs().clamp(min=1e-300), ks[t + 1:])
        p = a + b * s ** 2 + c * s ** 4
        # d symmetric: d_ij s_j has the even part (s_i + s_j) / 2 and the odd part (s_j - s_i) / 2
        eo = (even * (s[:, None] + s[None, :]) / 2) ** 2 + (odd * (s[None, :] - s[:, None]) / 2) ** 2
        # the padding of P holds a on its diagonal, which no row of X meets
        var_p = H ** 2 / 3 * (p ** 2).sum() / n ** 2
        var_a = H ** 2 / 3 * (s ** 4).sum() / n ** 2 * (b + c * (s[:, None] ** 2 + s[None, :] ** 2)) ** 2
        total += ((var_p + var_a) * eo).sum()
        if t + 1 < len(ks):
            # this step and the next together
            lam, lam2 = s ** 2, nxt ** 2
            a2, b2, c2 = ks[t + 1]
            p2 = a2 + b2 * lam2 + c2 * lam2 ** 2
            after, _ = _odd(s, ks[t:t + 2])
            even2, odd2, _ = _moves(after.abs().clamp(min=1e-300), ks[t + 2:])
            unit = H ** 2 / 3 / n ** 2
            var_q = unit * ((p * p2) ** 2).sum()
            total += (var_q * ((even2 * (s[:, None] + s[None, :]) / 2) ** 2 + (odd2 * (s[None, :] - s[:, None]) / 2) ** 2)).sum()
            var_t = unit * ((p * lam) ** 2).sum() * p[None, :] ** 2
            var_p1 = unit * (p ** 2).sum() * ((lam * p)[:, None] + (lam * p)[None, :]) ** 2
            moved = (var_t + var_p1) * (b2 + c2 * (lam2[:, None] + lam2[None, :])) ** 2
            n1 = nxt.abs()
            total += (moved * ((even2 * (n1[:, None] + n1[None, :]) / 2) ** 2 + (odd2 * (n1[None, :] - n1[:, None]) / 2) ** 2)).sum()
        s = nxt.abs().clamp(min=1e-300)
    return FOUR * float(total) ** 0.5


def orthogonalized(u, steps=5, coefficients=COEFFICIENTS, eps=1e-7, worst=False):
    """(result, bound on the 2-norm of a kernel's error before its last rounding)
    for one matrix u, in 64 bits on the CPU."""
    u = u.detach().cpu().double()
    x = u.T if u.shape[0] > u.shape[1] else u
    x = x / max(x.norm().item(), eps)
    n, m = x.shape
    ks = triples(coefficients, steps)
    err = 0.0 if worst else _random(torch.linalg.svdvals(x).clamp(min=1e-300), n, m, ks)
    eye = torch.eye(n, dtype=torch.float64)
    for a, b, c in ks:
        gram = x @ x.T
        p = a * eye + b * gram + c * (gram @ gram)
        if worst:
            s = torch.linalg.matrix_norm(x, 2).item()
            grid = torch.linspace(0, 1, 2001, dtype=torch.float64) * s * 1.01
            big = (a + 3 * b * grid ** 2 + 5 * c * grid ** 4).abs().max().item()
            err = big * (err + H * x.norm().item())
            err += H * s * ((abs(b) + 2 * abs(c) * s * s) * gram.norm().item() + p.norm().item())
        x = p @ x
    return (x.T if u.shape[0] > u.shape[1] else x), err


def quantized(m):
    """(codes, scales) of a 64-bit momentum [rows, cols], on the CPU."""
    rows, cols = m.shape
    nb = -(-cols // 256)
    codes = torch.zeros(rows, cols, dtype=torch.int8)
    scales = torch.zeros(rows, nb, dtype=torch.float32)
    for k in range(nb):
        part = m[:, 256 * k: 256 * (k + 1)]
        top = part.abs().amax(1)
        step = (top / 127).float()
        bad = ~torch.isfinite(part).all(1)
        step[bad] = float("nan")
        q = torch.where(step[:, None] > 0, torch.round(part / step.double()[:, None]).clamp(-127, 127), 0.0)
        codes[:, 256 * k: 256 * (k + 1)] = torch.nan_to_num(q).to(torch.int8)
        scales[:, k] = step
    return codes, scales


def values(codes, scales):
    at = torch.arange(codes.shape[-1]) // 256
    return codes.double() * scales.double()[..., at]
