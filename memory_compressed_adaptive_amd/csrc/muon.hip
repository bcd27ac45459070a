// Host side of the Muon operators: argument checks, the workspace's layout and
// the launches, all on the caller's stream.  The C ABI is declared and
// documented in include/microadam.h.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>

#include "host.hpp"
#include "microadam.h"
#include "muon_kernels.hpp"

using namespace microadam;

namespace {

constexpr int64_t kMaxElems = int64_t(1) << 33;     // of one matrix: keeps every launch's grid in range
constexpr int64_t kMaxSide = int64_t(1) << 21;      // 256 rows' bytes stay under 2^31
constexpr int kNormParts = 2048;                    // most partial sums of squares for one matrix
// A batch is cut into runs of matrices of at most this much workspace (with 256
// MiB 48 of 768 x 768 take 820 us instead of 770; 1 GiB is no better).
constexpr size_t kWorkspaceAim = size_t(512) << 20;

struct Coefficients { float v[kMaxSteps][3]; };

int64_t round_up(int64_t v, int64_t to) { return (v + to - 1) / to * to; }

// LDS that muon_small_kernel needs for n x m; 0 if it has no kernel for n.
int64_t small_lds(int64_t n, int64_t m) {
  const int64_t mp = round_up(m, 32);
  switch ((n + 31) / 32) {
    case 1: return SmallLds<1>::bytes(mp);
    case 2: return SmallLds<2>::bytes(mp);
    case 3: return SmallLds<3>::bytes(mp);
    case 4: return SmallLds<4>::bytes(mp);
    default: return 0;
  }
}

int small_parts(int64_t n) {
  return n <= 32 ? SmallLds<1>::kParts : n <= 64 ? SmallLds<2>::kParts : n <= 96 ? SmallLds<3>::kParts : SmallLds<4>::kParts;
}

bool fits_small(int64_t n, int64_t m, uint32_t runs) {
  const int64_t bytes = small_lds(n, m);
  return bytes > 0 && bytes <= 160 * 1024 && runs <= (uint32_t)(kSmallWaves * (n <= 32 ? SmallLds<1>::kRuns : SmallLds<4>::kRuns));
}

using Tile64 = Tile<64, 64, 2, 2, 64, 4, 2>;
using Tile128 = Tile<128, 128, 2, 2, 64, 2>;
using Tile128Deep = Tile<128, 128, 4, 2, 64, 4>;   // alone on a CU
using Tile192 = Tile<192, 192, 2, 2, 64, 3>;
using Tile256x192 = Tile<256, 192, 4, 2, 64, 2>;
using Tile256 = Tile<256, 256, 4, 2, 64, 2>;

// How a product is made: which tile, and (X X^T) in how many parts.
struct Choice {
  int kind;
  int parts;
  size_t bytes;   // the parts' sums
  double time;    // expected, in microseconds
};

int64_t count_tiles(int64_t m, int64_t n, int bm, int bn, bool symmetric) {
  const int64_t tm = (m + bm - 1) / bm, tn = (n + bn - 1) / bn;
  if (!symmetric) return tm * tn;
  int64_t tiles = 0;
  for (int64_t j = 0; j < tn; ++j) tiles += tiles_beside((int)j, bm, bn, (int)tm);
  return tiles;
}

// The tile with the shortest expected time.  Workgroups go over the 256 CUs in
// rounds; a round takes so long for 64 of the summed index and so long for its
// beginning and end (microseconds, measured on products that fill the card and
// on ones that do not; "alone": at most one workgroup on a CU).  Large tiles
// read less for each product; smaller ones waste less of the last round and of
// the half that a symmetric result leaves out (n = 4096: 136 tiles of 256 or 253
// of 192; 11008 x 4096 takes 2.64 ms without the 192 tile, 2.58 with it).
// Where parameters are read and written (`out`), the end is bound by memory, and
// two workgroups to a CU hide it.  Parts of the summed index fill the card where
// there are few tiles; their sums cost another launch and their way through
// memory (five steps of 2048 x 8192: 729 us without, 700 with).
Choice pick(int64_t m, int64_t n, int64_t k, int64_t chunk, bool symmetric, bool out, bool may_split) {
  const struct { int kind, bm, bn, per_cu; double alone, full, ends, out; } kinds[] = {
      {256, 256, 256, 1, 1.76, 1.76, 5.0, 14.0},
      {250, 256, 192, 1, 1.38, 1.38, 4.5, 12.0},
      {192, 192, 192, 1, 1.14, 1.14, 4.0, 10.0},
      {128, 128, 128, 2, 0.60, 1.02, 3.5, 6.0},
      {129, 128, 128, 1, 0.45, 0.95, 3.5, 6.0},
      {64, 64, 64, 2, 0.26, 0.40, 2.5, 3.5}};
  Choice best = {0, 1, 0, 0.0};
  double least = 0.0;
  for (const auto &t : kinds) {
    const int64_t tiles = count_tiles(m, n, t.bm, t.bn, symmetric) * chunk;
    for (int parts = 1; parts <= (may_split && t.bm <= 128 ? 32 : 1) && (parts == 1 || k / 64 >= 4 * parts); parts *= 2) {
      const int64_t groups = tiles * parts, whole = groups / (256 * t.per_cu), rest = groups - whole * 256 * t.per_cu;
      const double its = (double)((k / 64 + parts - 1) / parts), ends = out ? t.out : t.ends;
      const size_t bytes = parts > 1 ? (size_t)groups * t.bm * t.bn * 4 : 0;
      if (bytes > (size_t)64 << 20) break;
      double time = (double)whole * (its * t.full + ends) +
                    (rest == 0 ? 0.0 : its * (rest > 256 || whole > 0 ? t.full : t.alone) + ends);
      // their sums are written and read at 3 TB/s, by a tile's workgroup at 0.1
      if (parts > 1) time += 4.0 + (double)bytes / 3e6 + std::max((double)bytes / 3e6, (double)bytes / (double)tiles / 1e5);
      if (!best.kind || time < least) best = {t.kind, parts, bytes, time}, least = time;
    }
  }
  return best;
}

// How a batch of r x c matrices is cut and laid out in the workspace.
struct Plan {
  int64_t r, c, n, m;       // n <= m: the wide orientation's sides
  bool tall;
  // a workgroup for each matrix, no workspace: wherever LDS holds it (144 of 64 x
  // 768: 117 us as separate launches, 32 so; 64 x 64: 55 and 15)
  bool small;
  bool pairs;               // two steps are taken together
  bool diagonal;            // what rounding takes off P's diagonal is added back
  int64_t np, mp;           // padded
  int64_t chunk;            // matrices at a time
  MuonRun run;              // how waves go over the stored matrix
  uint32_t runs;
  int nparts;
  Choice gram, poly, update, last;   // tiles of the products of `chunk` matrices
  size_t x_bytes, a_bytes, part_bytes, lost_bytes, sum_bytes, bytes;

  Plan(int64_t batch, int64_t rows, int64_t cols) : r(rows), c(cols) {
    tall = r > c;
    n = std::min(r, c);
    m = std::max(r, c);
    np = round_up(n, 64);
    mp = round_up(m, 64);
    run.log_lanes = 6;
    while (run.log_lanes > 0 && (2 << run.log_lanes) >= c) --run.log_lanes;   // 4 columns to a lane
    const int64_t wide = 4 << run.log_lanes, at_once = 64 >> run.log_lanes;
    run.segs = (int)((c + wide - 1) / wide);
    run.groups = (int)((r + at_once - 1) / at_once);
    run.blocks = (int)((c + kMomentumBlock - 1) / kMomentumBlock);
    runs = (uint32_t)run.groups * (uint32_t)run.segs;
    nparts = (int)std::min<int64_t>(kNormParts, (runs + 15) / 16);   // four runs to a wave
    const size_t one = 2 * 2 * (size_t)(np * mp) + 3 * 2 * (size_t)(np * np) + 4 * (size_t)np + 8 * (size_t)nparts;
    small = fits_small(n, m, runs);
    if (small) { bytes = 256; return; }
    chunk = std::max<int64_t>(1, std::min<int64_t>(std::min<int64_t>(batch, 65535), (int64_t)(kWorkspaceAim / one)));
    const int64_t calls = (batch + chunk - 1) / chunk;
    chunk = (batch + calls - 1) / calls;   // runs of one length (4 of 4096 x 4096 as 2 + 2: 5.46 ms, as 3 + 1: 5.54)
    x_bytes = (size_t)round_up(2 * chunk * np * mp, 256);
    a_bytes = (size_t)round_up(2 * chunk * np * np, 256);
    part_bytes = (size_t)round_up(8 * chunk * nparts, 256);
    gram = pick(np, np, mp, chunk, true, false, true);
    poly = pick(np, np, np, chunk, true, false, false);
    update = pick(mp, np, np, chunk, false, false, false);
    last = pick(mp, np, np, chunk, false, true, false);
    // three products of the short side take the place of two with the long one
    // (11008 x 4096: 3.19 ms for five steps one by one, 2.66 two together; 2048 x
    // 8192: 726 and 627 us); with few rows, what rounding does to the diagonals
    // of P1 and T does not average out (37 x 3000: error 3.0e-3 against 1.4e-3)
    pairs = n > 128 && 3 * m >= 4 * n && gram.time + update.time > 1.1 * 3.0 * poly.time;
    // where A stays near a multiple of I; it takes a tenth of P X's time, so the
    // last product, of which nothing follows, goes without (wide matrices of 300 to
    // 1024 rows: error 2.2e-4 to 2.9e-4 after one step, 2.9e-4 to 4.4e-4 after two)
    diagonal = m >= 2 * n;
    lost_bytes = (size_t)round_up(4 * chunk * np, 256);
    sum_bytes = (size_t)round_up((int64_t)gram.bytes, 256);
    bytes = 2 * x_bytes + 3 * a_bytes + part_bytes + lost_bytes + sum_bytes;
  }
};

bool sizes_ok(int64_t batch, int64_t rows, int64_t cols) {
  return batch >= 0 && rows >= 0 && cols >= 0 && batch <= (int64_t(1) << 31) && rows <= kMaxSide && cols <= kMaxSide &&
         (rows == 0 || cols <= kMaxElems / rows);
}

// Whether the iterates stay inside the fp16 formats: with every singular value
// in [0, hi], a step maps s to s (a + b s^2 + c s^4); a + b x + c x^2 are the
// eigenvalues of P.  Extremes of both lie at ends or where a derivative is 0.
bool coefficients_ok(const float *k, int steps, const char **why) {
  double hi = 1.0;
  for (int t = 0; t < steps; ++t) {
    const double a = k[3 * t], b = k[3 * t + 1], c = k[3 * t + 2];
    if (!std::isfinite(a) || !std::isfinite(b) || !std::isfinite(c)) { *why = "not finite"; return false; }
    double xs[5] = {0.0, hi * hi, 0.0, 0.0, 0.0};
    int nx = 2;
    if (c != 0.0) xs[nx++] = -b / (2 * c);           // of a + b x + c x^2
    const double disc = 9 * b * b - 20 * a * c;      // of s (a + b s^2 + c s^4): a + 3 b x + 5 c x^2 = 0
    if (disc >= 0) {
      // both roots from the sum that cannot cancel, so that none is lost where c is tiny beside b
      const double q = -0.5 * (3 * b + std::copysign(std::sqrt(disc), b));
      if (c != 0.0) xs[nx++] = q / (5 * c);
      if (q != 0.0) xs[nx++] = a / q;
    }
    double top = 0.0;
    for (int q = 0; q < nx; ++q) {
      const double x = xs[q];
      if (!(x >= 0.0 && x <= hi * hi)) continue;
      const double p = a + b * x + c * x * x;
      if (!(std::fabs(p) <= 15.0)) { *why = "an eigenvalue of a I + b A + c A A can pass 15"; return false; }
      top = std::max(top, std::fabs(p) * std::sqrt(x));
    }
    hi = top * 1.01;                                 // with room for the roundings
    if (!(hi <= 1.95)) { *why = "a singular value can pass 1.95"; return false; }
    if (hi < 1e-3) { *why = "the singular values vanish"; return false; }
  }
  return true;
}

template <class T, int ROLE>
void product_t(MuonProduct a, int64_t chunk, hipStream_t s) {
  a.tiles_m = (int)((a.m + T::BM - 1) / T::BM);
  a.tiles_n = (int)((a.n + T::BN - 1) / T::BN);
  a.tiles = (int)count_tiles(a.m, a.n, T::BM, T::BN, ROLE != kUpdate && ROLE != kOut && ROLE != kOutTall);
  const int64_t groups = (int64_t)a.tiles * (ROLE == kGramPart ? a.parts : 1);
  if (ROLE != kGramPart && ROLE != kGramSum) a.parts = 1;
  // small tiles: a row of the grid for each matrix; else the kernel divides
  const dim3 grid = T::BM == 64 ? dim3((unsigned)groups, (unsigned)chunk) : dim3((unsigned)(groups * chunk));
  hipLaunchKernelGGL((muon_product_kernel<T, ROLE>), grid, dim3(T::kThreads), 0, s, a);
}

template <int ROLE>
void product(const MuonProduct &a, int64_t chunk, int kind, hipStream_t s) {
  if constexpr (ROLE != kGramPart && ROLE != kGramSum) {
    if (kind == 256) return product_t<Tile256, ROLE>(a, chunk, s);
    if (kind == 250) return product_t<Tile256x192, ROLE>(a, chunk, s);
    if (kind == 192) return product_t<Tile192, ROLE>(a, chunk, s);
  }
  switch (kind) {
    case 129: return product_t<Tile128Deep, ROLE>(a, chunk, s);
    case 128: return product_t<Tile128, ROLE>(a, chunk, s);
    default: return product_t<Tile64, ROLE>(a, chunk, s);
  }
}

template <int NB, int MOM>
hipError_t launch_small(int64_t batch, const MuonInput &in, const MuonRun &r, MuonSmall small, const MuonTarget &o,
                        size_t lds, hipStream_t s) {
  const hipError_t e = hipFuncSetAttribute((const void *)muon_small_kernel<NB, MOM>, hipFuncAttributeMaxDynamicSharedMemorySize,
                                           160 * 1024);
  if (e != hipSuccess) return e;
  for (small.b0 = 0; small.b0 < batch; small.b0 += 1 << 21)   // 2^31 threads in a launch
    hipLaunchKernelGGL((muon_small_kernel<NB, MOM>), dim3((unsigned)std::min<int64_t>(batch - small.b0, 1 << 21)),
                       dim3(64 * kSmallWaves),
                       lds, s, in, r, small, o);
  return hipGetLastError();
}

template <int MOM>
hipError_t run_small(const Plan &p, int64_t batch, const MuonInput &in, const MuonTarget &o, int steps, const Coefficients &k,
                     float eps, hipStream_t s) {
  MuonSmall small = {};
  for (int t = 0; t < steps; ++t)
    for (int e = 0; e < 3; ++e) small.k[t][e] = k.v[t][e];
  small.steps = steps;
  small.tall = p.tall;
  small.mp = (int)round_up(p.m, 32);
  small.eps = eps;
  // Two steps together save X X^T and P X once, for three short products: a
  // quarter of the time at 64 x 768, a loss below six times as wide as high.
  small.pairs = p.n <= 64 && p.m >= 6 * round_up(p.n, 32);
  small.single = steps & 1 ? 0 : -1;   // first: A is most nearly a multiple of I then
  // parts of at least four products of 16
  small.parts = 1;
  while (2 * small.parts <= small_parts(p.n) && small.mp / 16 / (2 * small.parts) >= 4) small.parts *= 2;
  const size_t lds = (size_t)small_lds(p.n, p.m);
  switch ((p.n + 31) / 32) {
    case 1: return launch_small<1, MOM>(batch, in, p.run, small, o, lds, s);
    case 2: return launch_small<2, MOM>(batch, in, p.run, small, o, lds, s);
    case 3: return launch_small<3, MOM>(batch, in, p.run, small, o, lds, s);
    default: return launch_small<4, MOM>(batch, in, p.run, small, o, lds, s);
  }
}

template <int MOM>
hipError_t run(const Plan &p, int64_t batch, const MuonInput &in, const MuonTarget &o, int steps, const Coefficients &k,
               float eps, void *workspace, hipStream_t s) {
  char *w = (char *)workspace;
  _Float16 *x0 = (_Float16 *)w, *x1 = (_Float16 *)(w + p.x_bytes);
  w += 2 * p.x_bytes;
  _Float16 *ga = (_Float16 *)w, *gp = (_Float16 *)(w + p.a_bytes), *gt = (_Float16 *)(w + 2 * p.a_bytes);
  w += 3 * p.a_bytes;
  double *part = (double *)w;
  float *lost = (float *)(w + p.part_bytes);
  float *sums = (float *)(w + p.part_bytes + p.lost_bytes);
  const int64_t nm = p.np * p.mp, nn = p.np * p.np;
  for (int64_t b0 = 0; b0 < batch; b0 += p.chunk) {
    const int64_t cb = std::min(p.chunk, batch - b0);
    hipLaunchKernelGGL((muon_norm_kernel<MOM>), dim3((unsigned)p.nparts, (unsigned)cb), dim3(256), 0, s, in,
                       p.run, b0, part, p.nparts);
    const int64_t sp = p.tall ? p.np : p.mp, tp = p.tall ? p.mp : p.np;
    _Float16 *x = x0, *nx = x1;
    const int64_t wide = 4 << p.run.log_lanes, across = (sp + wide - 1) / wide;
    // (a wave that goes over more than 16 rows at once would pass a block of 16)
    const bool few = p.run.log_lanes >= 2 && across * ((tp + 63) / 64) * cb < 512;
    const int rows = few ? 16 : 64;
    const dim3 lg((unsigned)across, (unsigned)((tp + rows - 1) / rows), (unsigned)cb);
    const auto load = p.tall ? (few ? muon_load_kernel<MOM, true, 16> : muon_load_kernel<MOM, true, 64>)
                             : (few ? muon_load_kernel<MOM, false, 16> : muon_load_kernel<MOM, false, 64>);
    hipLaunchKernelGGL(load, lg, dim3(256), 0, s, in, p.run, b0, part, p.nparts, eps, x, sp, tp);
    // steps in pairs, a single one (of an odd number) in the middle
    const int single = p.pairs ? (steps & 1 ? (steps / 2 + 1) / 2 * 2 : -1) : 0;
    for (int t = 0; t < steps;) {
      const bool two = p.pairs && t != single;
      MuonProduct a = {};
      a.l = a.r = x;
      a.l_mat = a.r_mat = nm;
      a.l_ld = a.r_ld = a.k = p.mp;
      a.m = a.n = p.np;
      a.d = ga;
      a.unit = 1.f / kScaleX;
      if (p.gram.parts > 1) {
        a.parts = p.gram.parts;
        a.sums = sums;
        product<kGramPart>(a, cb, p.gram.kind, s);
        product<kGramSum>(a, cb, p.gram.kind, s);
      } else {
        product<kGram>(a, cb, p.gram.kind, s);
      }
      // l r -> d, of symmetric matrices
      const auto square = [&](const _Float16 *l, const _Float16 *r, _Float16 *d, float unit) {
        a.l = l, a.r = r, a.d = d, a.unit = unit;
        product<kGram>(a, cb, p.poly.kind, s);
      };
      const auto poly = [&](const _Float16 *of, _Float16 *d, int step) {
        a.l = a.r = of, a.d = d;
        a.a = k.v[step][0], a.b = k.v[step][1], a.c = k.v[step][2];
        product<kPoly>(a, cb, p.poly.kind, s);
      };
      a.l_mat = a.r_mat = nn;
      a.l_ld = a.r_ld = a.k = p.np;
      // the last product has no step after it that would carry the rounding on
      float *const keep = p.diagonal && t + (two ? 2 : 1) < steps ? lost : nullptr;
      a.lost = two ? nullptr : keep;
      a.lost_unit = 1.f / kScaleP;
      poly(ga, gp, t);
      const _Float16 *factor = gp;
      float unit = 1.f / kScaleP;
      if (two) {
        square(gp, ga, gt, 1.f / kScaleX);                        // T = P A
        square(gt, gp, ga, kScaleX / (kScaleP * kScaleP));        // the next A
        poly(ga, gt, t + 1);
        a.lost = keep;
        a.lost_unit = 1.f / kScaleQ;
        square(gt, gp, ga, kScaleQ / (kScaleP * kScaleP));        // P2 P1
        factor = ga;
        unit = 1.f / kScaleQ;
      }
      t += two ? 2 : 1;
      a.l = x, a.l_mat = nm, a.l_ld = a.m = p.mp;
      a.r = factor;
      if (t < steps) {
        a.d = nx;
        a.unit = unit;
        product<kUpdate>(a, cb, p.update.kind, s);
        std::swap(x, nx);
        continue;
      }
      a.out = o;
      a.unit = unit / kScaleX;
      a.b0 = b0;
      if (p.tall) {   // the fastest index of `out` is P's
        std::swap(a.l, a.r);
        std::swap(a.l_mat, a.r_mat);
        std::swap(a.l_ld, a.r_ld);
        std::swap(a.m, a.n);
        product<kOutTall>(a, cb, p.last.kind, s);
      } else {
        product<kOut>(a, cb, p.last.kind, s);
      }
    }
  }
  return hipGetLastError();
}

// Checks that all calls share; MA_OK and *empty when there is nothing to do.
int check(const char *who, int64_t batch, int64_t rows, int64_t cols, int steps, const float *coefficients, float eps,
          const void *workspace, size_t workspace_bytes, bool *empty) {
  *empty = false;
  if (batch < 0 || rows < 0 || cols < 0) return fail(MA_EINVAL, "%s: batch, rows and cols must be >= 0", who);
  if (!sizes_ok(batch, rows, cols)) return fail(MA_EUNSUPPORTED, "%s: a matrix of more than 2^33 elements or a side over 2^21", who);
  if (steps < 1 || steps > kMaxSteps) return fail(MA_EINVAL, "%s: steps must be in 1..%d", who, kMaxSteps);
  if (!coefficients) return fail(MA_EINVAL, "%s: null coefficients", who);
  if (!(eps > 0.f) || !std::isfinite(eps)) return fail(MA_EINVAL, "%s: eps must be positive and finite", who);
  const char *why = "";
  if (!coefficients_ok(coefficients, steps, &why)) return fail(MA_EINVAL, "%s: coefficients: %s", who, why);
  if (!batch || !rows || !cols) { *empty = true; return MA_OK; }
  const Plan p(batch, rows, cols);
  if (!workspace || ((uintptr_t)workspace & 255u)) return fail(MA_EINVAL, "%s: the workspace must be 256-byte aligned", who);
  if (workspace_bytes < p.bytes)
    return fail(MA_EINVAL, "%s: a workspace of %zu bytes, %zu are needed", who, workspace_bytes, p.bytes);
  return MA_OK;
}

// Strides count up; what is written must not overlap (what is read may: a
// stride of 0 reads one matrix or one row again).  Either the matrices lie one
// after the other, or their rows side by side (column blocks of one matrix).
bool strides_ok(int64_t batch, int64_t rows, int64_t cols, int64_t row, int64_t bat, bool written) {
  if (row < 0 || bat < 0) return false;
  if (!written) return true;
  if (rows > 1 && row < cols) return false;
  if (batch <= 1 || (__int128)bat >= (__int128)(rows - 1) * row + cols) return true;
  return bat >= cols && (__int128)row >= (__int128)(batch - 1) * bat + cols;
}

constexpr const char *kStrides = "negative strides, or a written array's rows or matrices overlap";

int aligned_runs(const void *p, int elem, int64_t row, int64_t bat, int64_t rows, int64_t batch) {
  return ((uintptr_t)p & (uintptr_t)(4 * elem - 1)) == 0 && (rows == 1 || row % 4 == 0) && (batch == 1 || bat % 4 == 0);
}

int device_of(hipStream_t stream, int *dev) {
  if (!stream || stream == hipStreamLegacy || stream == hipStreamPerThread) return hipGetDevice(dev) == hipSuccess ? MA_OK : MA_EHIP;
  return hipStreamGetDevice(stream, dev) == hipSuccess ? MA_OK : MA_EHIP;
}

MuonTarget target(void *params, int type, int64_t row, int64_t bat, int64_t batch, int64_t rows, int64_t cols, double lr,
                  double wd, double scale) {
  return {params, type == MA_TYPE_BF16, 1, aligned_runs(params, type == MA_TYPE_BF16 ? 2 : 4, row, bat, rows, batch), row, bat,
          rows, cols, (float)(1.0 - lr * wd), (float)(lr * scale)};
}

Coefficients copy(const float *k, int steps) {
  Coefficients c = {};
  for (int t = 0; t < steps; ++t)
    for (int e = 0; e < 3; ++e) c.v[t][e] = k[3 * t + e];
  return c;
}

template <int MOM>
int enqueue(const char *who, int64_t batch, const MuonInput &in, const MuonTarget &o, int steps, const float *coefficients,
            float eps, void *workspace, hipStream_t stream) {
  int dev = 0;
  if (device_of(stream, &dev) != MA_OK) return fail(MA_EHIP, "%s: the stream has no device", who);
  DeviceGuard guard(dev);
  if (!guard.ok) return fail(MA_EHIP, "%s: device %d cannot be made current", who, dev);
  const Plan p(batch, in.r, in.c);
  const Coefficients k = copy(coefficients, steps);
  const hipError_t e = p.small ? run_small<MOM>(p, batch, in, o, steps, k, eps, stream)
                                            : run<MOM>(p, batch, in, o, steps, k, eps, workspace, stream);
  if (e != hipSuccess) return fail(MA_EHIP, "%s: launch failed: %s", who, hipGetErrorString(e));
  return MA_OK;
}

// what ma_muon_step and ma_muon8_step share
int check_step(const char *who, int64_t batch, int64_t rows, int64_t cols, const void *params, int p_type, int64_t p_row,
               int64_t p_batch, const uint16_t *grads, int64_t g_row, int64_t g_batch, double lr, double beta, double wd,
               double scale) {
  if (p_type != MA_TYPE_F32 && p_type != MA_TYPE_BF16) return fail(MA_EINVAL, "%s: unknown type %d", who, p_type);
  if (!params || !grads) return fail(MA_EINVAL, "%s: null pointer", who);
  if (((uintptr_t)params & (p_type == MA_TYPE_F32 ? 3u : 1u)) || ((uintptr_t)grads & 1u))
    return fail(MA_EINVAL, "%s: misaligned pointer", who);
  if (!(beta >= 0.0 && beta < 1.0)) return fail(MA_EINVAL, "%s: beta must be in [0, 1)", who);
  if (!std::isfinite(lr) || !std::isfinite(scale) || !(wd >= 0.0) || !std::isfinite(wd))
    return fail(MA_EINVAL, "%s: lr, scale and wd must be finite, wd >= 0", who);
  if (!strides_ok(batch, rows, cols, p_row, p_batch, true) || !strides_ok(batch, rows, cols, g_row, g_batch, false))
    return fail(MA_EINVAL, "%s: %s", who, kStrides);
  return MA_OK;
}

}  // namespace

extern "C" {

size_t ma_orthogonalize_workspace(int64_t batch, int64_t rows, int64_t cols) {
  if (!sizes_ok(batch, rows, cols) || !batch || !rows || !cols) return 0;
  return Plan(batch, rows, cols).bytes;
}

int ma_debug_muon_plan(int64_t batch, int64_t rows, int64_t cols, int64_t *out) {
  clear_error();
  const char *who = "ma_debug_muon_plan";
  if (!out) return fail(MA_EINVAL, "%s: null pointer", who);
  if (batch < 1 || rows < 1 || cols < 1) return fail(MA_EINVAL, "%s: batch, rows and cols must be >= 1", who);
  if (!sizes_ok(batch, rows, cols)) return fail(MA_EUNSUPPORTED, "%s: a matrix of more than 2^33 elements or a side over 2^21", who);
  const Plan p(batch, rows, cols);
  for (int e = 0; e < 9; ++e) out[e] = 0;
  out[0] = p.small;
  out[1] = p.tall;
  if (p.small) return MA_OK;
  out[2] = p.chunk;
  out[3] = p.pairs;
  out[4] = p.gram.kind;
  out[5] = p.gram.parts;
  out[6] = p.poly.kind;
  out[7] = p.update.kind;
  out[8] = p.last.kind;
  return MA_OK;
}

int ma_orthogonalize(int64_t batch, int64_t rows, int64_t cols, const void *x, int x_type, int64_t x_row, int64_t x_batch,
                     uint16_t *out, int64_t out_row, int64_t out_batch, int steps, const float *coefficients, float eps,
                     void *workspace, size_t workspace_bytes, hipStream_t stream) {
  clear_error();
  const char *who = "ma_orthogonalize";
  bool empty;
  if (const int rc = check(who, batch, rows, cols, steps, coefficients, eps, workspace, workspace_bytes, &empty)) return rc;
  if (x_type != MA_TYPE_F32 && x_type != MA_TYPE_BF16) return fail(MA_EINVAL, "%s: unknown type %d", who, x_type);
  if (empty) return MA_OK;
  const int elem = x_type == MA_TYPE_F32 ? 4 : 2;
  if (!x || !out) return fail(MA_EINVAL, "%s: null pointer", who);
  if (((uintptr_t)x & (uintptr_t)(elem - 1)) || ((uintptr_t)out & 1u)) return fail(MA_EINVAL, "%s: misaligned pointer", who);
  if (!strides_ok(batch, rows, cols, x_row, x_batch, false) || !strides_ok(batch, rows, cols, out_row, out_batch, true))
    return fail(MA_EINVAL, "%s: %s", who, kStrides);
  MuonInput in = {};
  in.x = x, in.x_bf16 = x_type == MA_TYPE_BF16, in.x_row = x_row, in.x_batch = x_batch;
  in.r = rows, in.c = cols;
  in.vec = aligned_runs(x, elem, x_row, x_batch, rows, batch);
  const MuonTarget o = {out, 1, 0, aligned_runs(out, 2, out_row, out_batch, rows, batch), out_row, out_batch, rows, cols, 1.f, 0.f};
  return enqueue<kMomNone>(who, batch, in, o, steps, coefficients, eps, workspace, stream);
}

int ma_muon_step(int64_t batch, int64_t rows, int64_t cols, void *params, int p_type, int64_t p_row, int64_t p_batch,
                 const uint16_t *grads, int64_t g_row, int64_t g_batch, float *momentum, double lr, double beta, double wd,
                 double scale, int nesterov, int steps, const float *coefficients, float eps, void *workspace,
                 size_t workspace_bytes, hipStream_t stream) {
  clear_error();
  const char *who = "ma_muon_step";
  bool empty;
  if (const int rc = check(who, batch, rows, cols, steps, coefficients, eps, workspace, workspace_bytes, &empty)) return rc;
  if (empty) return MA_OK;
  if (const int rc = check_step(who, batch, rows, cols, params, p_type, p_row, p_batch, grads, g_row, g_batch, lr, beta, wd, scale))
    return rc;
  if (!momentum || ((uintptr_t)momentum & 3u)) return fail(MA_EINVAL, "%s: null or misaligned momentum", who);
  MuonInput in = {};
  in.x = grads, in.x_bf16 = 1, in.x_row = g_row, in.x_batch = g_batch;
  in.mom = momentum, in.beta = beta, in.nesterov = nesterov != 0;
  in.r = rows, in.c = cols;
  in.vec = aligned_runs(grads, 2, g_row, g_batch, rows, batch) && ((uintptr_t)momentum & 15u) == 0 && cols % 4 == 0;
  const MuonTarget o = target(params, p_type, p_row, p_batch, batch, rows, cols, lr, wd, scale);
  return enqueue<kMom32>(who, batch, in, o, steps, coefficients, eps, workspace, stream);
}

int ma_muon8_step(int64_t batch, int64_t rows, int64_t cols, void *params, int p_type, int64_t p_row, int64_t p_batch,
                  const uint16_t *grads, int64_t g_row, int64_t g_batch, int8_t *codes, float *scales, double lr, double beta,
                  double wd, double scale, int nesterov, int steps, const float *coefficients, float eps, void *workspace,
                  size_t workspace_bytes, hipStream_t stream) {
  clear_error();
  const char *who = "ma_muon8_step";
  bool empty;
  if (const int rc = check(who, batch, rows, cols, steps, coefficients, eps, workspace, workspace_bytes, &empty)) return rc;
  if (empty) return MA_OK;
  if (const int rc = check_step(who, batch, rows, cols, params, p_type, p_row, p_batch, grads, g_row, g_batch, lr, beta, wd, scale))
    return rc;
  if (!codes || !scales || ((uintptr_t)scales & 3u)) return fail(MA_EINVAL, "%s: null or misaligned momentum", who);
  MuonInput in = {};
  in.x = grads, in.x_bf16 = 1, in.x_row = g_row, in.x_batch = g_batch;
  in.codes = codes, in.scales = scales, in.beta = beta, in.nesterov = nesterov != 0;
  in.r = rows, in.c = cols;
  in.vec = aligned_runs(grads, 2, g_row, g_batch, rows, batch) && ((uintptr_t)codes & 3u) == 0 && cols % 4 == 0;
  const MuonTarget o = target(params, p_type, p_row, p_batch, batch, rows, cols, lr, wd, scale);
  return enqueue<kMom8>(who, batch, in, o, steps, coefficients, eps, workspace, stream);
}

int ma_momentum8_values(int64_t rows, int64_t cols, const int8_t *codes, const float *scales, float *out, hipStream_t stream) {
  clear_error();
  const char *who = "ma_momentum8_values";
  if (rows < 0 || cols < 0) return fail(MA_EINVAL, "%s: rows and cols must be >= 0", who);
  if (!rows || !cols) return MA_OK;
  if (rows > (int64_t(1) << 46) / cols) return fail(MA_EUNSUPPORTED, "%s: more than 2^46 elements", who);
  if (!codes || !scales || !out || ((uintptr_t)scales & 3u) || ((uintptr_t)out & 3u))
    return fail(MA_EINVAL, "%s: null or misaligned pointer", who);
  int dev = 0;
  if (device_of(stream, &dev) != MA_OK) return fail(MA_EHIP, "%s: the stream has no device", who);
  DeviceGuard guard(dev);
  if (!guard.ok) return fail(MA_EHIP, "%s: device %d cannot be made current", who, dev);
  const int vec = cols % 4 == 0 && ((uintptr_t)codes & 3u) == 0 && ((uintptr_t)out & 15u) == 0;
  const int64_t segs = rows * ((cols + 255) / 256);
  const unsigned grid = (unsigned)std::min<int64_t>((segs + 3) / 4, 256 * 32);
  hipLaunchKernelGGL(momentum8_values_kernel, dim3(grid), dim3(256), 0, stream, codes, scales, out, rows, cols, vec);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return fail(MA_EHIP, "%s: launch failed: %s", who, hipGetErrorString(e));
  return MA_OK;
}

}  // extern "C"
