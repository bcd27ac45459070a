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


def orthogonalized_large(u, steps=5, coefficients=COEFFICIENTS, eps=1e-7):
    """(result, bound) as orthogonalized gives them for random roundings, where u
    is: 64-bit products on the GPU for large matrices.  The singular values come
    from the Gram matrix, near enough for a bound."""
    u = u.detach().double()
    x = (u.T if u.shape[0] > u.shape[1] else u).contiguous()
    x = x / max(x.norm().item(), eps)
    n, m = x.shape
    ks = triples(coefficients, steps)
    s = torch.linalg.eigvalsh((x @ x.T.contiguous()).cpu()).clamp(min=0).sqrt().clamp(min=1e-300).to(u.device)
    err = _random(s, n, m, ks)
    for a, b, c in ks:
        gram = x @ x.T.contiguous()
        ax = gram @ x
        x = a * x + b * ax + c * (gram @ ax)
    return (x.T if u.shape[0] > u.shape[1] else x), err


def orthogonalized_worst(u, steps=5, coefficients=COEFFICIENTS, eps=1e-7):
    """(result, bound) in the worst case, steps taken one by one or in twos (a
    single one of an odd number in the middle), whichever bound is larger.

    How far each entry can be off, to first order, every rounding being h of its
    entry at most and none of them averaging out.  |M| holds the entries'
    magnitudes; dX starts as h |X|:  dA = dX |X|' + |X| dX' + h |A|;
    dP = |b| dA + |c| (|A| dA + dA |A|) + h |P|;  of a single step
    dX <- |P| dX + dP |X| + h |P X|.  Of two:  dT = |P1| dA + dP1 |A| + h |T|;
    dA' = |T| dP1 + dT |P1| + h |A'|;  dP2 as dP, of A';
    dQ = |P2| dP1 + dP2 |P1| + h |Q|;  dX <- |Q| dX + dQ |X| + h |Q X|.  The last
    product is not rounded."""
    u = u.detach().cpu().double()
    x0 = (u.T if u.shape[0] > u.shape[1] else u).contiguous()
    x0 = x0 / max(x0.norm().item(), eps)
    ks = triples(coefficients, steps)
    eye = torch.eye(x0.shape[0], dtype=torch.float64)

    def poly(k, gram, dgram):
        p = k[0] * eye + k[1] * gram + k[2] * (gram @ gram)
        size = gram.abs()
        return p, abs(k[1]) * dgram + abs(k[2]) * (size @ dgram + dgram @ size) + H * p.abs()

    def times(l, dl, r, dr):
        d = l @ r
        return d, l.abs() @ dr + dl @ r.abs() + H * d.abs()

    def follow(pairs):
        x, dx, t = x0, H * x0.abs(), 0
        single = (steps // 2 + 1) // 2 * 2 if steps % 2 else -1
        while t < steps:
            gram, dgram = times(x, dx, x.T, dx.T)
            f, df = poly(ks[t], gram, dgram)
            if pairs and t != single:
                second, dsecond = times(*times(f, df, gram, dgram), f, df)
                p2, dp2 = poly(ks[t + 1], second, dsecond)
                f, df = times(p2, dp2, f, df)
                t += 1
            x, dx = times(f, df, x, dx)
            t += 1
        return x, (dx - H * x.abs()).norm().item()

    x, err = follow(False)
    err = max(err, follow(True)[1])
    return (x.T if u.shape[0] > u.shape[1] else x), err


def flat_worst(n, steps=5, coefficients=COEFFICIENTS):
    """For n equal singular values A, P and their products are multiples of I: all
    entries of a diagonal are rounded alike, and X is off by one factor.  The
    largest that factor can be (relative to the result), each rounding being h at
    most; the recursion of orthogonalized_worst for numbers, but with the slope of
    the polynomials.  Roundings of X are
    not in it."""
    ks = triples(coefficients, steps)

    def follow(pairs):
        s, err, t = n ** -0.5, 0.0, 0
        single = (steps // 2 + 1) // 2 * 2 if steps % 2 else -1
        while t < steps:
            take = ks[t:t + 2] if pairs and t != single else ks[t:t + 1]
            end, slope = _odd(torch.tensor(s, dtype=torch.float64), take)
            a, b, c = take[0]
            gram = s * s
            p1 = a + b * gram + c * gram * gram
            da = H * gram
            moved = dp1 = abs(b + 2 * c * gram) * da + H * abs(p1)
            if len(take) == 2:
                a, b, c = take[1]
                tt = p1 * gram
                gram2 = tt * p1
                dt = gram * dp1 + abs(p1) * da + H * abs(tt)
                da2 = abs(p1) * dt + abs(tt) * dp1 + H * gram2
                p2 = a + b * gram2 + c * gram2 * gram2
                dp2 = abs(b + 2 * c * gram2) * da2 + H * abs(p2)
                moved = abs(p1) * dp2 + abs(p2) * dp1 + H * abs(p1 * p2)
            err = abs(slope.item()) * err + s * moved
            s = abs(end.item())
            t += len(take)
        return err / s

    return max(follow(False), follow(True))
