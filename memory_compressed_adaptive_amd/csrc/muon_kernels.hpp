// Kernels of the Muon operators for gfx950: the momentum update (32-bit, or 8
// bits with a scale for every 256 elements of a row), and the Newton-Schulz
// products that bring all singular values of an update near 1.
//
// With U an r x c matrix, n = min(r, c), m = max(r, c) and X (n x m) its wide
// orientation, X0 = U / max(|U|_F, eps) and every step does
//
//   A = X X^T        (n x n, symmetric)
//   P = a I + b A + c A A   (n x n, symmetric)
//   X <- P X
//
// Two steps can be taken together: A and every polynomial of it commute, so
// that with P1 = p1(A) the next A is P1 A P1, and the second step's X is
// (P2 P1) X: the products with the long side, X X^T and P X, are made once for
// two steps, for three more products of the short side (T = P1 A, T P1 and
// P2 P1), all symmetric.  No intermediate X is rounded then; the roundings of T
// and P2 P1 take its place, and the error stays what it was (simulated: within
// a fifth).  Three steps together would not: what rounding does to small
// eigenvalues of A grows twelvefold with each.
//
// Number formats.  X, A and P are held in fp16, scaled by 2^14, 2^14 and 2^12,
// and every product is summed in fp32.  All of them are bounded: the host
// refuses coefficients for which a singular value could pass 1.95 or an
// eigenvalue of P 15, so |X| <= 1.95, |A| <= 3.8 and |P| <= 15 and nothing
// reaches fp16's largest value; an entry 2^-28 of that largest one still has
// all 11 bits.  Each rounding to fp16 is off by at most 2^-11 of a value.  In
// bf16 (2^-8) the result of five steps is off by 1.0e-2 (2-norm over 2-norm,
// random 768 x 768 matrices), in fp16 by 1.2e-3, at the same matrix rate; the
// rounding of the bf16 result alone is 1.7e-3.
//
// Layout.  X is held once, in its wide orientation.  Sides are padded with zeros
// to a multiple of 64 (the products keep the padding of X and A zero), so the
// summed index needs no bounds.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace microadam {

typedef _Float16 half8 __attribute__((ext_vector_type(8)));
typedef _Float16 half4 __attribute__((ext_vector_type(4)));
typedef float float16v __attribute__((ext_vector_type(16)));

constexpr float kScaleX = 16384.f;   // of X and of A
constexpr float kScaleP = 4096.f;   // of P and of P A
constexpr float kScaleQ = 256.f;    // of a product of two P
constexpr int kMomentumBlock = 256;  // elements of a row that share a scale

enum { kMomNone = 0, kMom32 = 1, kMom8 = 2 };

// What the momentum pass reads and writes for one batch of r x c matrices.
struct MuonInput {
  const void *x;            // U itself (kMomNone: f32 or bf16) or the gradient (bf16)
  int x_bf16;
  int64_t x_row, x_batch;   // strides in elements
  float *mom;               // kMom32, contiguous
  int8_t *codes;            // kMom8, contiguous
  float *scales;            // kMom8: [batch][r][ceil(c / 256)]
  double beta;
  int nesterov;
  int64_t r, c;
  int vec;                  // runs of 4 elements are aligned everywhere
};

__device__ __forceinline__ float bf16_f32(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }

typedef float float2v __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

// two values rounded to nearest even, the first in the low half (one instruction)
__device__ __forceinline__ uint32_t f32x2_bf16(float lo, float hi) {
  union { bf16x2 b; uint32_t u; } w;
  w.b = __builtin_convertvector((float2v{lo, hi}), bf16x2);
  return w.u;
}

// Where four consecutive elements of a row lie: element offsets into x, into
// the contiguous momentum and into its scales, and how many of the four are
// inside the matrix (0 or less: none).
struct MuonSpot {
  int64_t x, mat, scale;
  int n;
};

// What memory holds of them (zeros outside the matrix).  Reading and using them
// are apart, so that a kernel can have several reads on their way.
struct MuonRaw {
  float g[4];
  float mo[4];    // kMom32
  uint32_t w;     // kMom8: four codes
  float s;        // and their scale
};

template <int MOM>
__device__ __forceinline__ MuonRaw muon_raw(const MuonInput &I, const MuonSpot &at) {
  MuonRaw R = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}, 0u, 0.f};
  if (I.vec && at.n >= 4) {
    if (MOM != kMomNone || I.x_bf16) {
      const uint2 w = *(const uint2 *)((const uint16_t *)I.x + at.x);
      R.g[0] = __uint_as_float(w.x << 16);
      R.g[1] = __uint_as_float(w.x & 0xffff0000u);
      R.g[2] = __uint_as_float(w.y << 16);
      R.g[3] = __uint_as_float(w.y & 0xffff0000u);
    } else {
      const float4 w = *(const float4 *)((const float *)I.x + at.x);
      R.g[0] = w.x, R.g[1] = w.y, R.g[2] = w.z, R.g[3] = w.w;
    }
    if (MOM == kMom32) {
      const float4 w = *(const float4 *)(I.mom + at.mat);
      R.mo[0] = w.x, R.mo[1] = w.y, R.mo[2] = w.z, R.mo[3] = w.w;
    }
    if (MOM == kMom8) R.w = *(const uint32_t *)(I.codes + at.mat);
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (e >= at.n) continue;
      R.g[e] = MOM != kMomNone || I.x_bf16 ? bf16_f32(((const uint16_t *)I.x)[at.x + e]) : ((const float *)I.x)[at.x + e];
      if (MOM == kMom32) R.mo[e] = I.mom[at.mat + e];
      if (MOM == kMom8) R.w |= (uint32_t)(uint8_t)I.codes[at.mat + e] << (8 * e);
    }
  }
  if (MOM == kMom8 && at.n > 0) R.s = I.scales[at.scale];
  return R;
}

// The matrix to orthogonalise (u) and the new momentum (m32, m64) of those four
// elements; 0 outside the matrix.  m64: the 8-bit form's momentum, which
// decides its codes.  It is formed in 64 bits: a code lies where a product and
// a sum would each have moved it in fp32 about once in 1e5 elements, and what
// is written is then what the formula gives, on any machine; the pass is bound
// by memory either way.
template <int MOM>
__device__ __forceinline__ void muon_elems(const MuonInput &I, const MuonRaw &R, int n, float u[4], float m32[4],
                                           double m64[4]) {
  if (MOM == kMomNone) {
#pragma unroll
    for (int e = 0; e < 4; ++e) u[e] = R.g[e];
    return;
  }
  const float b32 = (float)I.beta, o32 = (float)(1.0 - I.beta);
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if (MOM == kMom32) {
      m32[e] = R.mo[e] * b32 + R.g[e] * o32;
    } else {
      // a block whose scale is NaN holds NaN; outside the matrix is 0
      m64[e] = e < n ? I.beta * ((double)(int8_t)(R.w >> (8 * e)) * (double)R.s) + (1.0 - I.beta) * (double)R.g[e] : 0.0;
      m32[e] = (float)m64[e];
    }
    u[e] = I.nesterov ? m32[e] * b32 + R.g[e] * o32 : m32[e];
  }
}

// Another lane's value by data-parallel primitives (a permute through LDS would
// take ten times as long).  kCtrl: 0xb1 and 0x4e exchange lanes within four,
// 0x141 and 0x140 mirror eight and sixteen.
template <int kCtrl>
__device__ __forceinline__ double dpp_f64(double v) {
  union { double d; int i[2]; } a, b;
  a.d = v;
  b.i[0] = __builtin_amdgcn_mov_dpp(a.i[0], kCtrl, 0xf, 0xf, true);
  b.i[1] = __builtin_amdgcn_mov_dpp(a.i[1], kCtrl, 0xf, 0xf, true);
  return b.d;
}

// The largest of `lanes` consecutive lanes' values (a power of two), in all of them.
__device__ __forceinline__ double lanes_max(double v, int lanes) {
  if (lanes > 1) v = fmax(v, dpp_f64<0xb1>(v));
  if (lanes > 2) v = fmax(v, dpp_f64<0x4e>(v));
  if (lanes > 4) v = fmax(v, dpp_f64<0x141>(v));
  if (lanes > 8) v = fmax(v, dpp_f64<0x140>(v));
  if (lanes > 16) v = fmax(v, __shfl_xor(v, 16, 64));
  if (lanes > 32) v = fmax(v, __shfl_xor(v, 32, 64));
  return v;
}

// The sum of a wave's values, in the same order every time.
__device__ __forceinline__ double wave_sum(double v) {
  v += dpp_f64<0xb1>(v);
  v += dpp_f64<0x4e>(v);
  v += dpp_f64<0x141>(v);
  v += dpp_f64<0x140>(v);
  v += __shfl_xor(v, 16, 64);
  return v + __shfl_xor(v, 32, 64);
}

// Writes their new momentum.  kMom8: `lanes` consecutive lanes hold a block of
// 256 (or the row's short last one, or the whole of a shorter row), and `first`
// is true in the one that holds its first element.  All lanes of a wave call it.
template <int MOM>
__device__ __forceinline__ void muon_store_momentum(const MuonInput &I, const MuonSpot &at, int lanes, bool first,
                                                    const float m32[4], const double m64[4]) {
  if (MOM == kMomNone) return;
  const bool run = I.vec && at.n >= 4;
  if (MOM == kMom32) {
    if (run) {
      *(float4 *)(I.mom + at.mat) = make_float4(m32[0], m32[1], m32[2], m32[3]);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (e < at.n) I.mom[at.mat + e] = m32[e];
    }
    return;
  }
  // the largest magnitude is 127 steps; a block with a non-finite value gets
  // the scale NaN and codes 0, and reads back as NaN.  A NaN counts as an
  // infinity here (fmax would drop it).
  double top = 0.0;
#pragma unroll
  for (int e = 0; e < 4; ++e) top = fmax(top, m64[e] == m64[e] ? fabs(m64[e]) : (double)__builtin_inff());
  top = lanes_max(top, lanes);
  const bool bad = !(top < (double)__builtin_inff());
  // top / 127 and 1 / step by a reciprocal and corrections; the operands are far
  // from the ends of fp64's range, so a division's scaling is not needed
  double quot = top * (1.0 / 127.0);
  quot = fma(fma(-127.0, quot, top), 1.0 / 127.0, quot);
  const float step = bad ? __builtin_nanf("") : (float)quot;
  const double d = (double)step;
  double inv = 0.0;
  if (step > 0.f) {
    inv = __builtin_amdgcn_rcp(d);
    inv = fma(fma(-d, inv, 1.0), inv, inv);
    inv = fma(fma(-d, inv, 1.0), inv, inv);
  }
  uint32_t w = 0;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    // m / step, corrected once: the product alone falls beside a half that the
    // quotient is exactly (73.5 / 49), and rounds to the odd code then
    double q = m64[e] * inv;
    q = fma(fma(-q, d, m64[e]), inv, q);
    const double q8 = bad ? 0.0 : fmin(fmax(rint(q), -127.0), 127.0);
    w |= ((uint32_t)(int32_t)q8 & 0xffu) << (8 * e);
  }
  if (run) {
    *(uint32_t *)(I.codes + at.mat) = w;
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (e < at.n) I.codes[at.mat + e] = (int8_t)(w >> (8 * e));
  }
  if (first && at.n > 0) I.scales[at.scale] = step;
}

// How waves go over a stored matrix: 2^log_lanes lanes to a row (4 columns each;
// 64, or fewer for narrow matrices) and so 64 >> log_lanes rows at once.
struct MuonRun {
  int log_lanes;
  int segs;        // runs along a row: ceil(c / (4 lanes))
  int groups;      // of rows
  int blocks;      // scales in a row
};

// Run `first`, then every `stride`-th.  What depends on the lane is set up once;
// a step is a few scalar instructions.
struct MuonWalk {
  int group, seg;              // uniform: which rows, which part of them
  int groups, segs, log_rows, log_wide, step_group, step_seg;
  int di, dj, r, c, blocks;
  int64_t x0, mat0, scale0, x_row;

  __device__ __forceinline__ MuonWalk(const MuonInput &I, const MuonRun &run, int64_t b, int lane, uint32_t first,
                                      uint32_t stride) {
    segs = run.segs;
    log_rows = 6 - run.log_lanes;
    log_wide = 2 + run.log_lanes;
    di = lane >> run.log_lanes;
    dj = 4 * (lane & ((1 << run.log_lanes) - 1));
    r = (int)I.r;
    c = (int)I.c;
    groups = run.groups;
    blocks = run.blocks;
    group = (int)first, seg = 0;
    step_group = (int)stride, step_seg = 0;
    if (segs > 1) {
      group = (int)(first / (uint32_t)segs);
      seg = (int)(first - (uint32_t)group * segs);
      step_group = (int)(stride / (uint32_t)segs);
      step_seg = (int)(stride - (uint32_t)step_group * segs);
    }
    x_row = I.x_row;
    x0 = b * I.x_batch + di * I.x_row + dj;
    mat0 = (b * I.r + di) * I.c + dj;
    scale0 = (b * I.r + di) * blocks;
  }
  __device__ __forceinline__ bool more() const { return group < groups; }
  __device__ __forceinline__ int row() const { return group << log_rows; }   // of lane 0
  __device__ __forceinline__ int col() const { return seg << log_wide; }
  __device__ __forceinline__ MuonSpot spot() const {
    const int i = row(), j = col(), left = c - dj - j;
    return {x0 + ((int64_t)i * x_row + j), mat0 + ((int64_t)i * c + j), scale0 + ((int64_t)i * blocks + seg), i + di < r ? left : 0};
  }
  __device__ __forceinline__ void next() {
    group += step_group;
    seg += step_seg;
    if (seg >= segs) seg -= segs, ++group;
  }
};

// ------------------------------------------------------------------ |U|_F
// Sum of squares of U in 64 bits (a gradient's squares can pass either end of
// fp32's range): block p of matrix b writes part[b][p].  No atomics, so results
// do not depend on timing.  Four reads of a lane are on their way at a time.
template <int MOM>
__global__ __launch_bounds__(256) void muon_norm_kernel(MuonInput I, MuonRun run, int64_t b0, double *part, int nparts) {
  const int lane = (int)(threadIdx.x & 63u), wave = (int)(threadIdx.x >> 6);
  const int64_t lb = blockIdx.y, b = b0 + lb;
  double sum = 0.0;
  MuonWalk walk(I, run, b, lane, __builtin_amdgcn_readfirstlane(blockIdx.x * 4 + wave), (uint32_t)nparts * 4);
  while (walk.more()) {
    MuonRaw R[4];
    int n[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const MuonSpot at = walk.spot();   // past the last run: past the last row, zeros
      n[e] = at.n;
      R[e] = muon_raw<MOM>(I, at);
      walk.next();
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      float u[4], m32[4];
      double m64[4];
      muon_elems<MOM>(I, R[e], n[e], u, m32, m64);
#pragma unroll
      for (int f = 0; f < 4; ++f) sum += (double)u[f] * (double)u[f];
    }
  }
  sum = wave_sum(sum);
  __shared__ double s[4];
  if (lane == 0) s[wave] = sum;
  __syncthreads();
  if (threadIdx.x == 0) part[lb * nparts + blockIdx.x] = (s[0] + s[1]) + (s[2] + s[3]);
}

// 1 / max(|U|_F, eps) from the sum of squares; NaN if that is NaN, 0 if it is
// infinite.  The hardware's reciprocal root has at least 14 bits; each
// correction doubles them.
__device__ __forceinline__ double muon_factor(double squares, float eps) {
  const double least = (double)eps * (double)eps;
  const double s = squares > least ? squares : least;   // (a NaN is put back below)
  double y = __builtin_amdgcn_rsq(s);
#pragma unroll
  for (int e = 0; e < 3; ++e) y = fma(y * 0.5, fma(-s * y, y, 1.0), y);
  return squares < __builtin_inf() ? y : squares == squares ? 0.0 : squares;
}

// ------------------------------------------------------------------ momentum, X0
// Writes the new momentum, and X0 in its wide orientation with zeros in the
// padding: as the matrix is stored, or transposed if that is tall.  A block of
// 256 threads takes kLoadRows rows x 4 * lanes columns of the stored
// matrix: 64, or 16 where that gives few blocks (768 x 768: 36 blocks take 11
// us, 144 take 5; 64 >> log_lanes rows, what a wave goes over at once, must fit
// in it).  sp, tp: the stored orientation's padded columns and rows.
template <int MOM, bool TALL, int kLoadRows>
__global__ __launch_bounds__(256) void muon_load_kernel(MuonInput I, MuonRun run, int64_t b0, const double *part, int nparts,
                                                        float eps, _Float16 *X, int64_t sp, int64_t tp) {
  __shared__ double s4[4];
  __shared__ _Float16 tile[TALL ? kLoadRows : 1][256 + 4];
  const int lanes = 1 << run.log_lanes;
  const int lane = (int)(threadIdx.x & 63u), wave = (int)(threadIdx.x >> 6);
  const int64_t lb = blockIdx.z, b = b0 + lb;
  const int64_t i0 = (int64_t)blockIdx.y * kLoadRows, j0 = (int64_t)blockIdx.x * (4 * lanes);
  const int col = 4 * (lane & (lanes - 1)), rows = 64 >> run.log_lanes;
  const int64_t j = j0 + col;
  double sum = 0.0;
  for (int p = (int)threadIdx.x; p < nparts; p += 256) sum += part[lb * nparts + p];
  sum = wave_sum(sum);
  if (lane == 0) s4[wave] = sum;
  __syncthreads();
  const double scale = (double)kScaleX * muon_factor((s4[0] + s4[1]) + (s4[2] + s4[3]), eps);
  X += lb * sp * tp;
  for (int q0 = wave * rows; q0 < kLoadRows; q0 += 16 * rows) {
    MuonRaw R[4];
    MuonSpot at[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int q = q0 + e * 4 * rows + (lane >> run.log_lanes);
      const int64_t i = i0 + q;
      at[e] = {b * I.x_batch + i * I.x_row + j, (b * I.r + i) * I.c + j, (b * I.r + i) * run.blocks + j / kMomentumBlock,
               q < kLoadRows && i < I.r ? (int)(I.c - j) : 0};
      R[e] = muon_raw<MOM>(I, at[e]);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (q0 + e * 4 * rows >= kLoadRows) break;
      const int q = q0 + e * 4 * rows + (lane >> run.log_lanes);
      float u[4], m32[4];
      double m64[4] = {0, 0, 0, 0};
      muon_elems<MOM>(I, R[e], at[e].n, u, m32, m64);
      half4 h;
#pragma unroll
      for (int f = 0; f < 4; ++f) h[f] = f < at[e].n ? (_Float16)(float)((double)u[f] * scale) : (_Float16)0.f;
      muon_store_momentum<MOM>(I, at[e], lanes, j % kMomentumBlock == 0, m32, m64);
      if (TALL) *(half4 *)&tile[q][col] = h;
      else if (j < sp && i0 + q < tp) *(half4 *)(X + (i0 + q) * sp + j) = h;
    }
  }
  if (!TALL) return;
  __syncthreads();
  // transposed: 8 consecutive rows of a column to a lane
  constexpr int kOcts = kLoadRows / 8;
  const int rg = (int)threadIdx.x % kOcts;
  for (int cc = (int)threadIdx.x / kOcts; cc < 4 * lanes; cc += 256 / kOcts) {
    half8 h;
#pragma unroll
    for (int e = 0; e < 8; ++e) h[e] = tile[8 * rg + e][cc];
    if (j0 + cc < sp && i0 + 8 * rg < tp) *(half8 *)(X + (j0 + cc) * tp + i0 + 8 * rg) = h;
  }
}

// Where the orthogonalised matrices go: rows x cols elements each.
struct MuonTarget {
  void *out;
  int bf16, update;     // update: theta <- theta * decay - rate * x; otherwise (bf16) x itself
  int vec;              // runs of 4 elements are aligned
  int64_t row, batch, rows, cols;
  float decay, rate;
};

// Four consecutive elements of it: where, how many are inside the matrix (n, as
// in MuonSpot), and what they held (32-bit values, or 16-bit ones in pairs).
// Reading and writing are apart, so that the reads are under way while other
// elements are written.
struct MuonOld {
  int64_t at;
  int n;
  uint32_t w[4];
};

// kPlain: it is known that nothing is updated (and the result is bf16).
template <bool kPlain>
__device__ __forceinline__ MuonOld read_out(const MuonTarget &T, int64_t at, int n) {
  MuonOld o = {at, n, {0u, 0u, 0u, 0u}};
  if (kPlain || !T.update) return o;
  if (T.bf16) {
    const uint16_t *p = (const uint16_t *)T.out + at;
    if (T.vec && n >= 4) {
      const uint2 w = *(const uint2 *)p;
      o.w[0] = w.x, o.w[1] = w.y;
    } else {
#pragma unroll
      for (int f = 0; f < 4; ++f)
        if (f < n) o.w[f >> 1] |= (uint32_t)p[f] << (16 * (f & 1));
    }
  } else {
    const uint32_t *p = (const uint32_t *)T.out + at;
    if (T.vec && n >= 4) {
      const uint4 w = *(const uint4 *)p;
      o.w[0] = w.x, o.w[1] = w.y, o.w[2] = w.z, o.w[3] = w.w;
    } else {
#pragma unroll
      for (int f = 0; f < 4; ++f)
        if (f < n) o.w[f] = p[f];
    }
  }
  return o;
}

// Four consecutive sums of the last product go there.
template <bool kPlain>
__device__ __forceinline__ void write_out(const MuonTarget &T, const MuonOld &o, float unit, float4 sums) {
  const float v[4] = {sums.x * unit, sums.y * unit, sums.z * unit, sums.w * unit};
  float x[4];
  if (kPlain || T.bf16) {
#pragma unroll
    for (int f = 0; f < 4; ++f) {
      const float old = __uint_as_float(f & 1 ? o.w[f >> 1] & 0xffff0000u : o.w[f >> 1] << 16);
      x[f] = !kPlain && T.update ? old * T.decay - T.rate * v[f] : v[f];
    }
    uint16_t *p = (uint16_t *)T.out + o.at;
    const uint32_t lo = f32x2_bf16(x[0], x[1]), hi = f32x2_bf16(x[2], x[3]);
    if (T.vec && o.n >= 4) {
      *(uint2 *)p = make_uint2(lo, hi);
    } else {
#pragma unroll
      for (int f = 0; f < 4; ++f)
        if (f < o.n) p[f] = (uint16_t)((f < 2 ? lo : hi) >> (16 * (f & 1)));
    }
  } else {
#pragma unroll
    for (int f = 0; f < 4; ++f) x[f] = __uint_as_float(o.w[f]) * T.decay - T.rate * v[f];
    float *p = (float *)T.out + o.at;
    if (T.vec && o.n >= 4) {
      *(float4 *)p = make_float4(x[0], x[1], x[2], x[3]);
    } else {
#pragma unroll
      for (int f = 0; f < 4; ++f)
        if (f < o.n) p[f] = x[f];
    }
  }
}

// ------------------------------------------------------------------ products
// D[n][m] = sum over k of L(m, k) R(n, k), fp32 sums.
enum {
  kGram = 0,     // A = X X^T:               L = R = X; and any product of symmetric matrices that commute
  kPoly = 1,     // P = a I + b A + c A A:   L = R = A
  kUpdate = 2,   // X' = P X:                L = X^T, R = P
  kOut = 3,      // the last X', with L and R as in kUpdate, written where the caller wants it
  kOutTall = 4,  // the same for a tall matrix, whose rows are the columns of X': L = P, R = X^T
  // A where X is so wide that its few tiles would leave most CUs idle: the
  // summed index is cut into parts, whose sums are added in their order
  kGramPart = 5,
  kGramSum = 6,
};

struct MuonProduct {
  const _Float16 *l, *r;
  int64_t l_mat, r_mat;     // elements from one matrix to the next
  int64_t l_ld, r_ld;       // and from one row of the stored array to the next
  int64_t k;
  _Float16 *d;              // [N][M]
  int64_t m, n;
  int tiles_m, tiles_n, tiles;   // of one matrix
  int parts;                // kGramPart, kGramSum
  float *sums;              // their fp32 sums: [matrix][tile][part][a tile's elements as its waves hold them]
  float a, b, c;            // kPoly
  float unit;               // the others: from a sum to the result
  // What rounding takes off the diagonal of P (or of a product of two), in real
  // units, [matrix][n]: written with it where not null, and added by kUpdate as
  // that many times the old X.  The diagonal holds most of a P while A is
  // small, and nearly the same value all along: its rounding would scale X as a
  // whole (440 x 6000: error 2.1e-3 without, 1.1e-3 with).  Null for the last
  // product: that rounding, at most 2^-11 of the result, meets no further step.
  float *lost;
  float lost_unit;
  MuonTarget out;           // kOut: element (n, m) of matrix b0 + i goes to its row n, column m
  int64_t b0;
};

// One workgroup makes a BM x BN tile of D with WM x WN waves, in steps of BK of
// the summed index.  The panels of both operands go from memory straight into
// LDS, S stages of them: while one is multiplied, the next S-1 are on their
// way.  A wave holds the fragments for the next 16 in registers, so that LDS
// reads run under the matrix instructions; the only barrier of a step stands
// before its last 16, when all fragments of the stage are in registers, and
// the copies that refill the stage are issued between that last 16's products
// and the next step's first.
//
// Panels come in two kinds.  Rows: the summed index is contiguous in memory; a
// panel is B rows of BK, and a lane's 8 values are one b128 read.  Columns:
// the other index is contiguous (X as the operand X^T of P X); a panel is BK
// rows of B, and a lane's 8 values are two b64 reads that transpose a 4 x 16
// block of 16-bit values among 16 lanes.  So X is kept in one orientation.
//
// Banks (64 of 4 bytes; a read serves 256 bytes a cycle).  Rows: 16-byte chunk
// c of row r lies at c ^ (r / 2 & 7), two rows being 256 bytes, so that 16 lanes
// (rows) of a b128 read take different banks (with c ^ (r & 7) every read
// counted four cycles of conflicts on top of its four).  Columns: 64-byte
// chunk c of row k lies at c ^ k modulo the chunks in 256 bytes, so that the
// four rows of a transposing read do.  The copies to LDS write their lanes one
// after the other; the order is made by which chunk a lane loads.
template <int BM_, int BN_, int WM_, int WN_, int BK_, int S_, int G_ = 1>
struct Tile {
  static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, BK = BK_, S = S_;
  static constexpr int G = G_, kGroups = BK / 16 / G;   // fragments are read for 16 G of the summed index at a time
  static_assert(kGroups % 2 == 0 && kGroups * 16 * G == BK, "the two sets of fragments take turns");
  static constexpr int kWaves = WM * WN, kThreads = 64 * kWaves;
  static constexpr int TM = BM / WM, TN = BN / WN, FM = TM / 32, FN = TN / 32;   // a wave's part, in 32 x 32 products
  static constexpr int LI = BM * BK / 512 / kWaves, RI = BN * BK / 512 / kWaves; // 1 KiB copies of a wave
  static constexpr int kStageBytes = (BM + BN) * BK * 2;
  static_assert(LI * 512 * kWaves == BM * BK && RI * 512 * kWaves == BN * BK, "copies divide evenly among the waves");
  static_assert(BK == 64, "LDS orders are made for it");
  static constexpr int kOutBytes = kWaves * 32 * (TM * 4 + 16);   // the epilogue's part of LDS
  static constexpr int kLds = S * kStageBytes > kOutBytes ? S * kStageBytes : kOutBytes;
  static_assert(kLds <= 160 * 1024, "LDS of a CU");
};

typedef int int4v __attribute__((ext_vector_type(4)));
typedef short short4v __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) short4v lds_short4;

// A buffer resource over `bytes` bytes at p (uniform); loads past them give 0
// and touch no memory.
__device__ __forceinline__ int4v buffer_of(uint64_t p, uint64_t bytes) {
  int4v r;
  r[0] = __builtin_amdgcn_readfirstlane((int)(uint32_t)p);
  r[1] = __builtin_amdgcn_readfirstlane((int)((uint32_t)(p >> 32) & 0xffff));
  r[2] = __builtin_amdgcn_readfirstlane((int)((uint32_t)(bytes >> 32) ? 0xffffffffu : (uint32_t)bytes));
  r[3] = 0x00020000;
  return r;
}

// 16 bytes a lane, from p + voff to LDS at `lds` + 16 * lane.  In asm, because
// after the builtin the compiler waits for every such copy before any later
// LDS read; here the waits are the kernel's own (stage_wait).  m0, which holds
// the LDS address, is an operand: the compiler writes it and knows what it
// holds.  A wait state belongs between that and the copy.
__device__ __forceinline__ void copy_to_lds(int4v p, uint32_t lds, uint32_t voff) {
  asm volatile("s_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" :: "{m0}"(lds), "v"(voff), "s"(p) : "memory");
}

// This wave's copies are done but for the last N, and so are its LDS reads;
// then all waves meet.
template <int N>
__device__ __forceinline__ void stage_wait() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" :: "n"(N) : "memory");
}

// One wave's LDS writes are done before its later reads of other lanes' values.
__device__ __forceinline__ void wave_lds_fence() {
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  __builtin_amdgcn_wave_barrier();
}

// How many tiles of row tj of a symmetric result are made: those that hold an
// element (n, m) with m <= n.
__host__ __device__ __forceinline__ int tiles_beside(int tj, int bm, int bn, int tiles_m) {
  const int n = (bn * (tj + 1) + bm - 1) / bm;
  return n < tiles_m ? n : tiles_m;
}

// Which tile (ti along M, tj along N) of which matrix a workgroup makes.
// Workgroups go to the eight XCDs in turn; each XCD gets one run of tiles,
// taken in blocks of 4 x 4, so that the panels its 32 CUs read at a time fit
// its L2.  SYM: only tiles with ti <= tj, the others are their mirror images.
// (Not so where tiles are not square, which are used where one round takes all.)
// Small tiles are taken as they come: their products are short, and L2 holds
// what they read.
template <bool SYM, bool PLAIN, bool PARTS, int BM, int BN>
__device__ __forceinline__ void tile_of(const MuonProduct &A, int &lb, int &ti, int &tj, int &part) {
  uint32_t at = blockIdx.x;
  if (!PLAIN) {
    const uint32_t total = gridDim.x, xcd = at & 7, per = total >> 3, rem = total & 7;
    at = xcd * per + (xcd < rem ? xcd : rem) + (at >> 3);
  }
  part = 0;
  if (PARTS) {
    part = (int)(at % (uint32_t)A.parts);
    at /= (uint32_t)A.parts;
  }
  lb = (int)blockIdx.y;
  int r = (int)at;
  if (!PLAIN) {
    lb = (int)(at / (uint32_t)A.tiles);
    r = (int)(at - (uint32_t)lb * A.tiles);
  }
  if (SYM && BM != BN) {
    tj = 0;
    for (int n; (n = tiles_beside(tj, BM, BN, A.tiles_m)) <= r; ++tj) r -= n;
    ti = r;
  } else if (SYM && PLAIN) {
    int y = (int)((sqrtf(8.f * (float)r + 1.f) - 1.f) * 0.5f);
    while (y * (y + 1) / 2 > r) --y;
    while ((y + 1) * (y + 2) / 2 <= r) ++y;
    ti = r - y * (y + 1) / 2;
    tj = y;
  } else if (PLAIN) {
    tj = r / A.tiles_m;
    ti = r - tj * A.tiles_m;
  } else if (SYM) {
    // before row block J lie 4J (4J + 1) / 2 tiles
    int J = (int)((sqrtf(4.f + 32.f * (float)r) - 2.f) * 0.0625f);
    while (8 * J * J + 2 * J > r) --J;
    while (8 * (J + 1) * (J + 1) + 2 * (J + 1) <= r) ++J;
    r -= 8 * J * J + 2 * J;
    const int h = A.tiles_n - 4 * J < 4 ? A.tiles_n - 4 * J : 4;
    if (r < 4 * h * J) {
      const int I = r / (4 * h);
      r -= I * 4 * h;
      ti = 4 * I + (r & 3);
      tj = 4 * J + (r >> 2);
    } else {
      r -= 4 * h * J;
      const int y = r >= 6 ? 3 : r >= 3 ? 2 : r >= 1 ? 1 : 0;
      ti = 4 * J + r - y * (y + 1) / 2;
      tj = 4 * J + y;
    }
  } else {
    const int J = r / (4 * A.tiles_m), h = A.tiles_n - 4 * J < 4 ? A.tiles_n - 4 * J : 4;
    r -= J * 4 * A.tiles_m;
    ti = r / h;
    tj = 4 * J + r - ti * h;
  }
  lb = __builtin_amdgcn_readfirstlane(lb);
  ti = __builtin_amdgcn_readfirstlane(ti);
  tj = __builtin_amdgcn_readfirstlane(tj);
  part = __builtin_amdgcn_readfirstlane(part);
}

// Where 16-byte chunk g of a B-wide panel in LDS comes from: bytes from the
// panel's start in memory, with rows of ld bytes.
template <bool COLS, int B>
__device__ __forceinline__ uint32_t panel_source(int g, uint32_t ld) {
  if (COLS) {
    constexpr int kRow = B / 8;   // chunks in a row
    const int row = g / kRow, p = g % kRow;
    constexpr int kIn = B % 128 == 0 ? 4 : 2;   // 64-byte chunks that are exchanged, in 256 bytes (128: two rows of them)
    const int x = kIn == 4 ? row & 3 : row >> 1 & 1;
    return (uint32_t)row * ld + (uint32_t)(p ^ (x << 2)) * 16;
  }
  const int row = g / 8, p = g % 8;
  return (uint32_t)row * ld + (uint32_t)(p ^ (row / 2 & 7)) * 16;
}

// A lane's 8 values for the product at 16 * ks: index `at` + (lane & 31) of the
// panel, summed index 16 * ks + 8 * (lane / 32) + 0..7.
template <bool COLS, int B>
__device__ __forceinline__ half8 panel_read(const char *panel, int at, int ks, int lane) {
  if (COLS) {
    // lanes 16q..16q+15 transpose 4 rows of 16 columns: lane s of them points
    // at row s / 4, columns 4 (s & 3) ..+3 and gets column s of the four rows
    union { short4v s[2]; half8 h; } u;
    const int s = lane & 15, col = at + (lane & 16) + 4 * (s & 3);
    const int c16 = col >> 3, rest = (col & 7) * 2;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int row = 16 * ks + 8 * (lane >> 5) + 4 * e + (s >> 2);
      constexpr int kIn = B % 128 == 0 ? 4 : 2;
      const int x = kIn == 4 ? row & 3 : row >> 1 & 1;
      u.s[e] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
          (lds_short4 *)(panel + row * (B * 2) + ((c16 ^ (x << 2)) * 16 + rest)));
    }
    return u.h;
  }
  const int row = at + (lane & 31);
  return *(const half8 *)(panel + row * 128 + (((2 * ks + (lane >> 5)) ^ (row / 2 & 7)) * 16));
}

template <class T, int ROLE>
__global__ __launch_bounds__(T::kThreads) void muon_product_kernel(MuonProduct A) {
  constexpr bool LC = ROLE == kUpdate || ROLE == kOut, RC = ROLE == kOutTall, OUT = ROLE == kOut || ROLE == kOutTall;
  constexpr bool SYM = ROLE == kGram || ROLE == kPoly || ROLE == kGramPart || ROLE == kGramSum;
  __shared__ __attribute__((aligned(1024))) char smem[T::kLds];
  const int lane = (int)(threadIdx.x & 63u), wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int wm = wave % T::WM * T::TM, wn = wave / T::WM * T::TN;
  int lb, ti, tj, part;
  tile_of<SYM, T::BM == 64, ROLE == kGramPart, T::BM, T::BN>(A, lb, ti, tj, part);
  const int64_t m0 = (int64_t)ti * T::BM, n0 = (int64_t)tj * T::BN;

  constexpr int kSums = T::kWaves * T::FM * T::FN * 1024;   // of a tile
  float *sums = A.sums + ((int64_t)lb * A.tiles + (ti + (int64_t)tj * (tj + 1) / 2)) * A.parts * kSums + wave * (T::FM * T::FN * 1024) + lane * 4;
  const int steps = (int)(A.k / T::BK), first = ROLE == kGramPart ? (int)((int64_t)steps * part / A.parts) : 0;
  const int nk = ROLE == kGramPart ? (int)((int64_t)steps * (part + 1) / A.parts) - first : steps;

  // Panels that pass the matrix: rows past its last read as zeros (the buffer
  // ends there); columns past a row's last read the next row, and only reach
  // elements of D past its sides, which are not stored.
  const int64_t l_ld = 2 * A.l_ld, r_ld = 2 * A.r_ld;   // bytes of a row; 256 rows stay under 2^31
  const char *pl = (const char *)(A.l + lb * A.l_mat) + (LC ? 2 * m0 : m0 * l_ld) + first * (T::BK * 2);
  const char *pr = (const char *)(A.r + lb * A.r_mat) + (RC ? 2 * n0 : n0 * r_ld) + first * (T::BK * 2);
  const int64_t nl = (const char *)(A.l + (lb + 1) * A.l_mat) - pl, nr = (const char *)(A.r + (lb + 1) * A.r_mat) - pr;
  const int64_t sl = LC ? T::BK * l_ld : T::BK * 2, sr = RC ? T::BK * r_ld : T::BK * 2;   // to the next step
  uint32_t vl[T::LI], vr[T::RI];
#pragma unroll
  for (int i = 0; i < T::LI; ++i) vl[i] = panel_source<LC, T::BM>((wave + i * T::kWaves) * 64 + lane, (uint32_t)l_ld);
#pragma unroll
  for (int i = 0; i < T::RI; ++i) vr[i] = panel_source<RC, T::BN>((wave + i * T::kWaves) * 64 + lane, (uint32_t)r_ld);
  const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char *)smem + wave * 1024;

  // copy i of step t into stage `to`
  auto copy = [&](int i, int4v bl, int4v br, int to) {
    const uint32_t at = lds0 + to * T::kStageBytes;
    if (i < T::LI) copy_to_lds(bl, at + i * (T::kWaves * 1024), vl[i]);
    else copy_to_lds(br, at + T::BM * T::BK * 2 + (i - T::LI) * (T::kWaves * 1024), vr[i - T::LI]);
  };
  constexpr int kCopies = T::LI + T::RI;

  float16v acc[T::FM][T::FN];
#pragma unroll
  for (int i = 0; i < T::FM; ++i)
#pragma unroll
    for (int j = 0; j < T::FN; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.f;

  constexpr int G = T::G;
  half8 x[2][T::FM * G], y[2][T::FN * G];
  constexpr int kFragments = G * (T::FM + T::FN);
  auto fragment = [&](int at, int stage, int group, half8 *fx, half8 *fy) {
    const char *p = smem + stage * T::kStageBytes;
    const int g = at / (T::FM + T::FN), i = at % (T::FM + T::FN), j = i - T::FM;
    if (j < 0) fx[g * T::FM + i] = panel_read<LC, T::BM>(p, wm + 32 * i, group * G + g, lane);
    else fy[g * T::FN + j] = panel_read<RC, T::BN>(p + T::BM * T::BK * 2, wn + 32 * j, group * G + g, lane);
  };
  auto fragments = [&](int stage, int group, half8 *fx, half8 *fy) {
#pragma unroll
    for (int at = 0; at < kFragments; ++at) fragment(at, stage, group, fx, fy);
  };
  constexpr int kProducts = G * T::FM * T::FN;
  auto product = [&](int at, const half8 *fx, const half8 *fy) {
    const int g = at / (T::FM * T::FN), j = at / T::FM % T::FN, i = at % T::FM;
    acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(fx[g * T::FM + i], fy[g * T::FN + j], acc[i][j], 0, 0, 0);
  };

  // A's part of the tile (kPoly) or the old X's (kUpdate), whole rows at a time
  // and 32 rows ahead, the first of them before the main loop (read four elements
  // at a time by the lanes that need them, A took 20 000 cycles of a 192 x 192
  // tile's 150 000)
  constexpr bool kBeside = ROLE == kPoly || ROLE == kUpdate;
  constexpr int kRowChunks = T::TM / 8, kTrips = kBeside ? 32 * kRowChunks / 64 : 1;
  half8 beside[2][kTrips];
  float keep[2] = {0.f, 0.f};   // kUpdate: what P's diagonal lacks at this lane's row
  const bool use_beside = ROLE == kPoly || (ROLE == kUpdate && A.lost != nullptr);   // uniform
  auto read_beside = [&](int j) {
#pragma unroll
    for (int g = 0; g < kTrips; ++g) {
      const int row = (g * 64 + lane) / kRowChunks, c = (g * 64 + lane) % kRowChunks;
      const int64_t nn = n0 + wn + 32 * j + row, mm = m0 + wm + 8 * c;
      beside[j & 1][g] = half8{0, 0, 0, 0, 0, 0, 0, 0};
      if (nn < A.n && mm < A.m) beside[j & 1][g] = *(const half8 *)(A.l + lb * A.l_mat + nn * A.l_ld + mm);
    }
    const int64_t nn = n0 + wn + 32 * j + (lane & 31);
    if (ROLE == kUpdate) keep[j & 1] = nn < A.n ? A.lost[lb * A.n + nn] : 0.f;
  };
  if (use_beside) read_beside(0);
  // Copies past the last step go to an empty buffer, so that the loop has one
  // shape and a wait counts the same copies at every step.
  uint64_t al = (uint64_t)pl, ar = (uint64_t)pr, el = (uint64_t)nl, er = (uint64_t)nr;   // of the next step to copy
  int to_copy = nk;
  int4v bl, br;
  auto next_copy = [&]() {
    bl = buffer_of(al, to_copy > 0 ? el : 0);
    br = buffer_of(ar, to_copy > 0 ? er : 0);
    --to_copy;
    al += (uint64_t)sl, el -= (uint64_t)sl;
    ar += (uint64_t)sr, er -= (uint64_t)sr;
  };
  // The copies that refill a stage are issued in the last group of its step and
  // the first of the next.  All in one group, 64 KiB for a 256 x 256 tile in a
  // quarter of a step, was twice what a CU takes in (2048 x 8192: 597 us against
  // 572); over three groups the last of them come late (2% slower).
  constexpr int kShare = (kCopies + 1) / 2;
  if (ROLE != kGramSum) {
#pragma unroll
    for (int t = 0; t < T::S; ++t) {
      next_copy();
#pragma unroll
      for (int i = 0; i < (t + 1 < T::S ? kCopies : kShare); ++i) copy(i, bl, br, t);
    }
    stage_wait<(T::S - 2) * kCopies + kShare>();
    fragments(0, 0, x[0], y[0]);
    int stage = 0, before = T::S - 1;
    for (int t = 0; t < nk; ++t) {
      const int next = stage + 1 == T::S ? 0 : stage + 1;
#pragma unroll
      for (int g = 0; g < T::kGroups; ++g) {
        const bool last = g + 1 == T::kGroups;
        if (last) {
          // the next stage is whole, and nobody reads this one any more
          __builtin_amdgcn_sched_barrier(0);
          stage_wait<(T::S - 2) * kCopies>();
          next_copy();
        }
        // the next fragments' reads and the copies are spread over the products
        const int from = last ? 0 : kShare, to = last ? kShare : g == 0 ? kCopies : kShare;
        constexpr int kEach = (kShare + kProducts - 1) / kProducts, kEachRead = (kFragments + kProducts - 1) / kProducts;
#pragma unroll
        for (int q = 0; q < kProducts; ++q) {
          __builtin_amdgcn_sched_barrier(0);
          product(q, x[g & 1], y[g & 1]);
#pragma unroll
          for (int c = q * kEachRead; c < (q + 1) * kEachRead && c < kFragments; ++c)
            fragment(c, last ? next : stage, last ? 0 : g + 1, x[(g + 1) & 1], y[(g + 1) & 1]);
#pragma unroll
          for (int c = from + q * kEach; c < from + (q + 1) * kEach; ++c)
            if (c < to) copy(c, bl, br, last ? stage : before);
        }
      }
      before = stage;
      stage = next;
    }
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  if (ROLE == kGramPart) {
#pragma unroll
    for (int i = 0; i < T::FM; ++i)
#pragma unroll
      for (int j = 0; j < T::FN; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q)
          *(float4 *)(sums + (int64_t)part * kSums + (i * T::FN + j) * 1024 + q * 256) =
              make_float4(acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]);
    return;
  }
  if (ROLE == kGramSum) {
#pragma unroll 2
    for (int p = 0; p < A.parts; ++p)
#pragma unroll
      for (int i = 0; i < T::FM; ++i)
#pragma unroll
        for (int j = 0; j < T::FN; ++j)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const float4 v = *(const float4 *)(sums + (int64_t)p * kSums + (i * T::FN + j) * 1024 + q * 256);
            acc[i][j][4 * q] += v.x, acc[i][j][4 * q + 1] += v.y, acc[i][j][4 * q + 2] += v.z, acc[i][j][4 * q + 3] += v.w;
          }
  }
  __syncthreads();   // the stages' LDS is the epilogue's now

  // Each wave brings 32 rows (n) x TM of its part through LDS at a time, so
  // that memory is written in whole runs of a row.
  char *mine = smem + wave * (32 * (T::TM * 4 + 16));
  constexpr int kOutChunks = T::TM / 4, kOutTrips = 32 * kOutChunks / 64;
  auto out_spot = [&](int j, int g) {
    const int row = (g * 64 + lane) / kOutChunks, c = (g * 64 + lane) % kOutChunks;
    const int64_t nn = n0 + wn + 32 * j + row, mm = m0 + wm + 4 * c;
    return read_out<false>(A.out, (A.b0 + lb) * A.out.batch + nn * A.out.row + mm, nn < A.out.rows ? (int)(A.out.cols - mm) : 0);
  };
  MuonOld old[OUT ? kOutTrips : 1];
  if (OUT) {
#pragma unroll
    for (int g = 0; g < kOutTrips; ++g) old[g] = out_spot(0, g);
  }
#pragma unroll
  for (int j = 0; j < T::FN; ++j) {
    const int64_t nb = n0 + wn + 32 * j, mb = m0 + wm;
    if (OUT) {
      float4 v[kOutTrips];
      constexpr int kStride = T::TM * 4 + 16;
#pragma unroll
      for (int i = 0; i < T::FM; ++i)
#pragma unroll
        for (int q = 0; q < 4; ++q)
          *(float4 *)(mine + (lane & 31) * kStride + (32 * i + 8 * q + 4 * (lane >> 5)) * 4) =
              make_float4(acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]);
      wave_lds_fence();
#pragma unroll
      for (int g = 0; g < kOutTrips; ++g) {
        const int row = (g * 64 + lane) / kOutChunks, c = (g * 64 + lane) % kOutChunks;
        v[g] = *(const float4 *)(mine + row * kStride + c * 16);
      }
      // the old values of the next 32 rows are read before these are written
#pragma unroll
      for (int g = 0; g < kOutTrips; ++g) {
        const MuonOld o = old[g];
        if (j + 1 < T::FN) old[g] = out_spot(j + 1, g);
        write_out<false>(A.out, o, A.unit, v[g]);
      }
      wave_lds_fence();
      continue;
    }
    constexpr int kStride = T::TM * 2 + 16;
    const int64_t dn = A.m;   // elements of a row of D
    _Float16 *d = A.d + lb * A.m * A.n;
    if (use_beside) {
#pragma unroll
      for (int g = 0; g < kTrips; ++g) {
        const int row = (g * 64 + lane) / kRowChunks, c = (g * 64 + lane) % kRowChunks;
        *(half8 *)(mine + row * kStride + c * 16) = beside[j & 1][g];
      }
      if (j + 1 < T::FN) read_beside(j + 1);
      wave_lds_fence();
    }
#pragma unroll
    for (int i = 0; i < T::FM; ++i) {
      const bool diagonal = SYM && nb == mb + 32 * i;   // uniform: this 32 x 32 block holds the diagonal
      float own = 0.f;                                  // and this lane, if it does, this element of it
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int r = 32 * i + 8 * q + 4 * (lane >> 5);
        half4 h, s = {0, 0, 0, 0};
        if (use_beside) s = *(const half4 *)(mine + (lane & 31) * kStride + r * 2);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float v = acc[i][j][4 * q + e];
          float o = v * A.unit;
          if (ROLE == kUpdate) o += keep[j & 1] * (float)s[e];
          if (ROLE == kPoly) {
            o = (A.b * (kScaleP / kScaleX)) * (float)s[e] + (A.c * (kScaleP / (kScaleX * kScaleX))) * v;
            if (diagonal && (lane & 31) == 8 * q + 4 * (lane >> 5) + e) o += A.a * kScaleP;
          }
          if (SYM) own = (lane & 31) == 8 * q + 4 * (lane >> 5) + e ? o : own;
          h[e] = (_Float16)o;
        }
        *(half4 *)(mine + (lane & 31) * kStride + r * 2) = h;
      }
      if (SYM && diagonal && A.lost && (lane >> 2 & 1) == lane >> 5 && nb + (lane & 31) < A.n)
        A.lost[lb * A.n + nb + (lane & 31)] = (own - (float)(_Float16)own) * A.lost_unit;
    }
    wave_lds_fence();
#pragma unroll
    for (int g = lane; g < 32 * kRowChunks; g += 64) {
      const int row = g / kRowChunks, c = g % kRowChunks;
      const half8 h = *(const half8 *)(mine + row * kStride + c * 16);
      // of a symmetric result the 32 x 32 blocks with m <= n
      if (nb + row < A.n && mb + 8 * c < A.m && (!SYM || mb + 8 * c < nb + 32)) *(half8 *)(d + (nb + row) * dn + mb + 8 * c) = h;
    }
    if (SYM && mb < nb) {
      // their mirror image: lane s of 16 gets column s of 4 rows at a time
      const int s = lane & 15, oct = lane >> 4;
#pragma unroll
      for (int c = 0; c < T::TM / 16; ++c) {
        if (mb + 16 * c >= nb) continue;
        union { short4v s[2]; half8 h; } u;
#pragma unroll
        for (int e = 0; e < 2; ++e)
          u.s[e] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
              (lds_short4 *)(mine + (8 * oct + 4 * e + (s >> 2)) * kStride + (16 * c + 4 * (s & 3)) * 2));
        const int64_t mm = mb + 16 * c + s, nn = nb + 8 * oct;
        if (mm < A.m && nn < A.n) *(half8 *)(d + mm * dn + nn) = u.h;
      }
    }
    wave_lds_fence();
  }
}

// ------------------------------------------------------------------ a whole matrix in one workgroup
// Matrices whose X, A and P fit a CU's LDS take one launch: momentum, norm, all
// steps and the result, one workgroup of 16 waves for each matrix.  What bounds
// it is latency: a step is three short products with a barrier after each.  The
// other way is 2 + 3 steps launches, of at least 3 us each.
//
// NB = ceil(n / 32) blocks of rows.  The symmetric products have NB (NB + 1) / 2
// tiles of 32 x 32; where there are few, the summed index of X X^T is cut among
// the waves and the parts are added in a fixed order.  P X is made in place: a
// wave reads all of a panel of 32 columns into registers before it writes any
// of it, and no other wave needs that panel.  Rows in LDS are 16 bytes longer
// than their content: 16 consecutive rows of a b128 read then start in
// different banks.
//
// The matrix is read once: a lane keeps its elements of U until the norm is
// known.  X0 is U times the power of two that puts its norm in (1/2, 1] 2^14,
// and what is left of the factor 1 / max(|U|, eps) goes into the fp32 results
// of the first step's products, which costs no rounding.
//
// P's diagonal holds most of it, the same value all along while A is small: its
// rounding to fp16 would scale the whole of X.  What the rounding takes off is
// kept beside P and multiplied as a diagonal matrix, two more matrix
// instructions to a block (64 x 64: error 1.6e-3 without, 1.2e-3 with).
constexpr int kMaxSteps = 64;
constexpr int kSmallWaves = 16;

struct MuonSmall {
  float k[kMaxSteps][3];
  int steps, tall;
  int mp;               // m rounded up to 32
  int parts;            // of the summed index of X X^T
  int pairs, single;    // steps are taken two together, but for this one
  float eps;
  int64_t b0;           // first matrix of this launch
};

template <int NB>
struct SmallLds {
  static constexpr int kRow = 64 * NB + 16;                 // of A and P
  static constexpr int kTiles = NB * (NB + 1) / 2;
  static constexpr int kParts = NB == 1 ? 8 : NB == 2 ? 4 : NB == 3 ? 2 : 1;   // at most; a power of two
  static constexpr int kScratch = kParts / 2 * kTiles * 4096;
  static constexpr int kRuns = NB == 1 ? 20 : 16;   // runs of 64 x 4 elements that a wave can keep
  static constexpr bool kPairs = NB <= 2;                   // a wider matrix that fits is not wide enough for them
  static constexpr int kSquares = kPairs ? 3 : 2;           // n x n matrices: A, P, and T
  static constexpr int64_t bytes(int64_t mp) {
    return 32 * NB * (2 * mp + 16) + kSquares * 32 * NB * kRow + kScratch + 8 * kSmallWaves + 3 * 64 * NB;
  }
};

template <int NB, int MOM>
__global__ __launch_bounds__(64 * kSmallWaves) void muon_small_kernel(MuonInput I, MuonRun run, MuonSmall S, MuonTarget out) {
  using L = SmallLds<NB>;
  extern __shared__ __attribute__((aligned(16))) char sm[];
  const int lane = (int)(threadIdx.x & 63u), wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int64_t b = S.b0 + blockIdx.x;
  const int xrow = 2 * S.mp + 16;
  char *const X = sm, *const A = X + 32 * NB * xrow, *const P = A + 32 * NB * L::kRow;
  char *const Tm = P + (L::kPairs ? 32 * NB * L::kRow : 0);
  float *const scratch = (float *)(A + L::kSquares * 32 * NB * L::kRow);
  double *const red = (double *)((char *)scratch + L::kScratch);
  // what rounding took off the diagonals of P, P2 and P2 P1, in their units
  _Float16 *const d0 = (_Float16 *)(red + kSmallWaves), *const d1 = d0 + 32 * NB, *const dq = d1 + 32 * NB;

  // U and its norm, the new momentum, zeros for X's padding
  if ((S.tall ? I.c : I.r) != 32 * NB || (S.tall ? I.r : I.c) != S.mp) {
    for (int at = (int)threadIdx.x * 16; at < 32 * NB * xrow; at += 1024 * kSmallWaves)
      *(float4 *)(X + at) = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  constexpr int kGroup = MOM == kMomNone ? 4 : 2;   // reads under way in a lane (registers bound it)
  float u[L::kRuns][4];
  double sum = 0.0;
  {
    MuonWalk walk(I, run, b, lane, wave, kSmallWaves);
#pragma unroll
    for (int g = 0; g < L::kRuns; g += kGroup) {
      if (!walk.more()) continue;
      MuonRaw R[kGroup];
      MuonSpot at[kGroup];
#pragma unroll
      for (int e = 0; e < kGroup; ++e) {
        at[e] = walk.spot();   // past the last run: past the last row, zeros
        R[e] = muon_raw<MOM>(I, at[e]);
        walk.next();
      }
#pragma unroll
      for (int e = 0; e < kGroup; ++e) {
        float m32[4];
        double m64[4] = {0, 0, 0, 0};
        muon_elems<MOM>(I, R[e], at[e].n, u[g + e], m32, m64);
        muon_store_momentum<MOM>(I, at[e], 1 << run.log_lanes, walk.dj == 0, m32, m64);
#pragma unroll
        for (int f = 0; f < 4; ++f) sum += (double)u[g + e][f] * (double)u[g + e][f];
      }
    }
  }
  sum = wave_sum(sum);
  if (lane == 0) red[wave] = sum;
  __syncthreads();
  double total = red[0];
#pragma unroll
  for (int w = 1; w < kSmallWaves; ++w) total += red[w];
  // 1 / max(|U|, eps) = rest * 2^pow, rest in [1, 2); all NaN if the norm is not finite
  const double factor = muon_factor(total, S.eps);
  int pow = 0;
  const double frac = frexp(factor, &pow);   // in [1/2, 1)
  const bool fine = factor > 0.0 && factor < (double)__builtin_inff();
  const float rest = fine ? (float)(2.0 * frac) : __builtin_nanf("");
  const int shift = fine ? pow - 1 + 14 : 0;
  {
    // two factors: one could leave fp32's range
    const float up = ldexpf(1.f, shift / 2), up2 = ldexpf(1.f, shift - shift / 2);
    MuonWalk walk(I, run, b, lane, wave, kSmallWaves);
    const int to = S.tall ? walk.dj * xrow + 2 * walk.di : walk.di * xrow + 2 * walk.dj;
#pragma unroll
    for (int g = 0; g < L::kRuns; ++g) {
      if (!walk.more()) continue;
      const int i = walk.row(), j = walk.col(), n = i + walk.di < walk.r ? walk.c - walk.dj - j : 0;
      _Float16 h[4];
#pragma unroll
      for (int f = 0; f < 4; ++f) h[f] = (_Float16)(u[g][f] * up * up2);
      if (!S.tall) {
        // past the last column u is 0, and so is the padding
        if (n > 0) *(half4 *)(X + to + i * xrow + 2 * j) = half4{h[0], h[1], h[2], h[3]};
      } else {
#pragma unroll
        for (int f = 0; f < 4; ++f)
          if (f < n) *(_Float16 *)(X + to + (j + f) * xrow + 2 * i) = h[f];
      }
      walk.next();
    }
  }
  __syncthreads();

  const int half = lane >> 5, row = lane & 31;
  // tile t of the upper triangle, row by row of blocks j >= i
  auto tile_at = [&](int t, int &ti, int &tj) {
    tj = t >= 6 ? 3 : t >= 3 ? 2 : t >= 1 ? 1 : 0;
    ti = t - tj * (tj + 1) / 2;
  };
  auto zero = [](float16v &v) {
#pragma unroll
    for (int e = 0; e < 16; ++e) v[e] = 0.f;
  };
  // four values (m, m + 1, ..) of column n of a symmetric tile, and their mirror image
  auto put = [&](char *to, int ti, int tj, int q, half4 h) {
    const int n = 32 * tj + row, m = 32 * ti + 8 * q + 4 * half;
    *(half4 *)(to + n * L::kRow + m * 2) = h;
    if (ti < tj) {
#pragma unroll
      for (int e = 0; e < 4; ++e) *(_Float16 *)(to + (m + e) * L::kRow + n * 2) = h[e];
    }
  };

  // a panel of 32 columns of X as fragments; the whole of it is in registers
  // before anything of it is written
  auto panel = [&](int jp, half8 *x) {
    const int s = lane & 15;
    const char *px = X + (8 * half + (s >> 2)) * xrow + (32 * jp + (lane & 16) + 4 * (s & 3)) * 2;
#pragma unroll
    for (int k = 0; k < 2 * NB; ++k) {
      union { short4v s[2]; half8 h; } w;
      w.s[0] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_short4 *)(px + 16 * k * xrow));
      w.s[1] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_short4 *)(px + (16 * k + 4) * xrow));
      x[k] = w.h;
    }
    wave_lds_fence();
  };

  // block `blk` of a diagonal matrix as two fragments: a lane's value stands at
  // its row's place among the 8 it holds of one of them
  const int place = row - 8 * half;
  auto diagonal = [&](const _Float16 *d, int blk, half8 f[2]) {
    union { _Float16 h; uint16_t u; } v;
    v.h = d[32 * blk + row];
    const uint32_t w = (uint32_t)v.u << (16 * (place & 1));
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      union { uint32_t w[4]; half8 h; } to;
#pragma unroll
      for (int e = 0; e < 4; ++e) to.w[e] = place >> 1 == 8 * k + e ? w : 0u;
      f[k] = to.h;
    }
  };

  const char *F = P;          // X <- F X, in units of `unit`
  const _Float16 *fd = d0;    // and what F's diagonal lacks
  float unit = 1.f / kScaleP;
  for (int t = 0; t < S.steps;) {
    const bool two = L::kPairs && S.pairs && t != S.single;
    const float left = t == 0 ? rest : 1.f;
    // A = X X^T: wave = part * kTiles + tile
    {
      const int tile = wave % L::kTiles, part = wave / L::kTiles;
      int ti, tj;
      tile_at(tile, ti, tj);
      float16v acc, acc2;
      zero(acc);
      zero(acc2);
      if (part < S.parts) {
        const int nk = S.mp / 16, k0 = nk * part / S.parts, k1 = nk * (part + 1) / S.parts;
        const char *pl = X + (32 * ti + row) * xrow + 16 * half, *pr = X + (32 * tj + row) * xrow + 16 * half;
        int k = k0;
        for (; k + 2 <= k1; k += 2) {
          const half8 l0 = *(const half8 *)(pl + 32 * k), r0 = *(const half8 *)(pr + 32 * k);
          const half8 l1 = *(const half8 *)(pl + 32 * k + 32), r1 = *(const half8 *)(pr + 32 * k + 32);
          acc = __builtin_amdgcn_mfma_f32_32x32x16_f16(l0, r0, acc, 0, 0, 0);
          acc2 = __builtin_amdgcn_mfma_f32_32x32x16_f16(l1, r1, acc2, 0, 0, 0);
        }
        if (k < k1)
          acc = __builtin_amdgcn_mfma_f32_32x32x16_f16(*(const half8 *)(pl + 32 * k), *(const half8 *)(pr + 32 * k), acc, 0, 0, 0);
      }
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[e] += acc2[e];
      for (int off = S.parts / 2; off >= 1; off >>= 1) {
        float *slot = scratch + ((part & (off - 1)) * L::kTiles + tile) * 1024 + lane * 4;
        if (part >= off && part < 2 * off) {
#pragma unroll
          for (int q = 0; q < 4; ++q)
            *(float4 *)(slot + 256 * q) = make_float4(acc[4 * q], acc[4 * q + 1], acc[4 * q + 2], acc[4 * q + 3]);
        }
        __syncthreads();
        if (part < off) {
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const float4 v = *(const float4 *)(slot + 256 * q);
            acc[4 * q] += v.x, acc[4 * q + 1] += v.y, acc[4 * q + 2] += v.z, acc[4 * q + 3] += v.w;
          }
        }
        if (off > 1) __syncthreads();
      }
      if (part == 0) {
        const float to_a = left * left * (1.f / kScaleX);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          half4 h;
#pragma unroll
          for (int e = 0; e < 4; ++e) h[e] = (_Float16)(acc[4 * q + e] * to_a);
          put(A, ti, tj, q, h);
        }
      }
    }
    __syncthreads();
    // phase 0: P = a I + b A + c A A.  Of a pair also 1: T = P A, 2: A = T P,
    // 3: P2 of that, in T's place, 4: P2 P in A's.
    for (int ph = 0; ph < (two ? 5 : 1); ++ph) {
      if (wave < L::kTiles) {
        const bool poly = ph == 0 || ph == 3;
        const char *const lb = poly ? A : ph == 1 ? P : Tm, *const rb = poly || ph == 1 ? A : P;
        char *const to = ph == 0 ? P : ph == 1 || ph == 3 ? Tm : A;
        int ti, tj;
        tile_at(wave, ti, tj);
        float16v acc, acc2;
        zero(acc);
        zero(acc2);
        const char *pl = lb + (32 * ti + row) * L::kRow + 16 * half, *pr = rb + (32 * tj + row) * L::kRow + 16 * half;
#pragma unroll
        for (int k = 0; k < NB; ++k) {
          acc = __builtin_amdgcn_mfma_f32_32x32x16_f16(*(const half8 *)(pl + 64 * k), *(const half8 *)(pr + 64 * k), acc, 0, 0, 0);
          acc2 = __builtin_amdgcn_mfma_f32_32x32x16_f16(*(const half8 *)(pl + 64 * k + 32), *(const half8 *)(pr + 64 * k + 32),
                                                        acc2, 0, 0, 0);
        }
        if (L::kPairs && (ph == 1 || ph == 4)) {   // the left factor's diagonal
          half8 f[2];
          diagonal(ph == 1 ? d0 : d1, ti, f);
          acc = __builtin_amdgcn_mfma_f32_32x32x16_f16(f[0], *(const half8 *)(pr + 64 * ti), acc, 0, 0, 0);
          acc2 = __builtin_amdgcn_mfma_f32_32x32x16_f16(f[1], *(const half8 *)(pr + 64 * ti + 32), acc2, 0, 0, 0);
        }
        if (L::kPairs && (ph == 2 || ph == 4)) {   // the right one's
          half8 f[2];
          diagonal(d0, tj, f);
          acc = __builtin_amdgcn_mfma_f32_32x32x16_f16(*(const half8 *)(pl + 64 * tj), f[0], acc, 0, 0, 0);
          acc2 = __builtin_amdgcn_mfma_f32_32x32x16_f16(*(const half8 *)(pl + 64 * tj + 32), f[1], acc2, 0, 0, 0);
        }
        const int step = ph == 3 ? t + 1 : t;
        const float ka = poly ? S.k[step][0] * kScaleP : 0.f, kb = poly ? S.k[step][1] * (kScaleP / kScaleX) : 0.f;
        const float kc = poly     ? S.k[step][2] * (kScaleP / (kScaleX * kScaleX))
                         : ph == 1 ? 1.f / kScaleX
                         : ph == 2 ? kScaleX / (kScaleP * kScaleP)
                                   : kScaleQ / (kScaleP * kScaleP);
        float own = 0.f;   // this lane's element of the diagonal, if it has one
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int n = 32 * tj + row, m = 32 * ti + 8 * q + 4 * half;
          half4 s = {0, 0, 0, 0};
          if (poly) s = *(const half4 *)(A + n * L::kRow + m * 2);
          half4 h;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float o = kb * (float)s[e] + kc * (acc[4 * q + e] + acc2[4 * q + e]);
            if (n == m + e) o += ka;
            own = n == m + e ? o : own;
            h[e] = (_Float16)o;
          }
          put(to, ti, tj, q, h);
        }
        // (of phases 1 and 2 it is not used, and written over)
        if (ti == tj && (row >> 2 & 1) == half)
          (ph == 0 ? d0 : ph == 3 ? d1 : dq)[32 * tj + row] = (_Float16)(own - (float)(_Float16)own);
      }
      __syncthreads();
    }
    F = two ? A : P;
    fd = two ? dq : d0;
    unit = left * (two ? 1.f / kScaleQ : 1.f / kScaleP);
    t += two ? 2 : 1;
    if (t >= S.steps) break;
    // X <- F X, 32 columns at a time
    half8 fs[NB <= 2 ? NB : 1][2];
    if (NB <= 2) {
#pragma unroll
      for (int ib = 0; ib < NB; ++ib) diagonal(fd, ib, fs[NB <= 2 ? ib : 0]);
    }
    for (int jp = wave; jp < S.mp / 32; jp += kSmallWaves) {
      half8 x[2 * NB];
      panel(jp, x);
#pragma unroll
      for (int ib = 0; ib < NB; ++ib) {
        float16v acc;
        zero(acc);
        const char *pp = F + (32 * ib + row) * L::kRow + 16 * half;
        half8 *const f = fs[NB <= 2 ? ib : 0];
        if (NB > 2) diagonal(fd, ib, f);
#pragma unroll
        for (int k = 0; k < 2 * NB; ++k)
          acc = __builtin_amdgcn_mfma_f32_32x32x16_f16(x[k], *(const half8 *)(pp + 32 * k), acc, 0, 0, 0);
#pragma unroll
        for (int k = 0; k < 2; ++k) acc = __builtin_amdgcn_mfma_f32_32x32x16_f16(x[2 * ib + k], f[k], acc, 0, 0, 0);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          half4 h;
#pragma unroll
          for (int e = 0; e < 4; ++e) h[e] = (_Float16)(acc[4 * q + e] * unit);
          *(half4 *)(X + (32 * ib + row) * xrow + (32 * jp + 8 * q + 4 * half) * 2) = h;
        }
      }
    }
    __syncthreads();
  }

  // the last F X goes to memory
  const float kUnit = unit / kScaleX;
  const int r = lane >> 3, c = lane & 7;   // of a 32 x 32 block a lane writes rows r, r + 8, .., columns 4c..
  auto spots = [&](int jp, int ib, MuonOld *old) {
    const int i = S.tall ? 32 * jp + row : 32 * ib + r, j = S.tall ? 32 * ib + 4 * half : 32 * jp + 4 * c;
    const int64_t at = b * out.batch + i * out.row + j, step = S.tall ? 8 : 8 * out.row;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      if (MOM != kMomNone && S.tall && 32 * ib + 8 * q >= (int)out.cols) continue;   // uniform: all of it is padding
      const int n = S.tall ? (i < (int)out.rows ? (int)out.cols - j - 8 * q : 0) : i + 8 * q < (int)out.rows ? (int)out.cols - j : 0;
      old[q] = read_out<MOM == kMomNone>(out, at + q * step, n);
    }
  };
  // a panel's results; where a panel is one block, the old values of this
  // wave's next panel are read first
  constexpr bool kAhead = MOM != kMomNone && NB == 1;
  auto emit = [&](int jp, MuonOld *old, MuonOld *next) {
    half8 x[2 * NB];
    if (kAhead && jp + kSmallWaves < S.mp / 32) spots(jp + kSmallWaves, 0, next);
    panel(jp, x);
#pragma unroll
    for (int ib = 0; ib < NB; ++ib) {
      float16v acc;
      zero(acc);
      const char *pp = F + (32 * ib + row) * L::kRow + 16 * half;
      half8 f[2];
      diagonal(fd, ib, f);
      if (MOM != kMomNone && !kAhead) spots(jp, ib, old);
      if (S.tall) {
        // rows of the result are columns of X: a lane has four consecutive elements of one
#pragma unroll
        for (int k = 0; k < 2 * NB; ++k)
          acc = __builtin_amdgcn_mfma_f32_32x32x16_f16(*(const half8 *)(pp + 32 * k), x[k], acc, 0, 0, 0);
#pragma unroll
        for (int k = 0; k < 2; ++k) acc = __builtin_amdgcn_mfma_f32_32x32x16_f16(f[k], x[2 * ib + k], acc, 0, 0, 0);
        if (MOM == kMomNone) spots(jp, ib, old);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          if (32 * ib + 8 * q >= (int)out.cols) continue;
          write_out<MOM == kMomNone>(out, old[q], kUnit, make_float4(acc[4 * q], acc[4 * q + 1], acc[4 * q + 2], acc[4 * q + 3]));
        }
      } else {
#pragma unroll
        for (int k = 0; k < 2 * NB; ++k)
          acc = __builtin_amdgcn_mfma_f32_32x32x16_f16(x[k], *(const half8 *)(pp + 32 * k), acc, 0, 0, 0);
#pragma unroll
        for (int k = 0; k < 2; ++k) acc = __builtin_amdgcn_mfma_f32_32x32x16_f16(x[2 * ib + k], f[k], acc, 0, 0, 0);
        // A block goes through the panel's place in LDS (32 NB rows of 64
        // bytes), so that memory is written in whole rows of it.
        if (MOM == kMomNone && out.vec && (out.row & 7) == 0 && (out.batch & 7) == 0 && ((uintptr_t)out.out & 15) == 0 &&
            32 * jp + 32 <= (int)out.cols && 32 * ib + 32 <= (int)out.rows) {
          // bf16 results, a whole block of them: 16 bytes a lane
#pragma unroll
          for (int q = 0; q < 4; ++q)
            *(uint2 *)(X + row * xrow + 64 * jp + 16 * q + 8 * half) =
                make_uint2(f32x2_bf16(acc[4 * q] * kUnit, acc[4 * q + 1] * kUnit),
                           f32x2_bf16(acc[4 * q + 2] * kUnit, acc[4 * q + 3] * kUnit));
          wave_lds_fence();
          uint16_t *to = (uint16_t *)out.out + (b * out.batch + (32 * ib + (lane >> 2)) * out.row + 32 * jp + 8 * (lane & 3));
#pragma unroll
          for (int e = 0; e < 2; ++e)
            *(uint4 *)(to + 16 * e * out.row) = *(const uint4 *)(X + ((lane >> 2) + 16 * e) * xrow + 64 * jp + 16 * (lane & 3));
          wave_lds_fence();
        } else {
          // 16 rows of 32 fp32 results at a time: row i of them lies in rows 2i and 2i + 1
          if (MOM == kMomNone) spots(jp, ib, old);
#pragma unroll
          for (int p = 0; p < 2; ++p) {
            if (row >> 4 == p) {
#pragma unroll
              for (int q = 0; q < 4; ++q)
                *(float4 *)(X + (2 * (row & 15) + (q >> 1)) * xrow + 64 * jp + ((q & 1) * 8 + 4 * half) * 4) =
                    make_float4(acc[4 * q], acc[4 * q + 1], acc[4 * q + 2], acc[4 * q + 3]);
            }
            wave_lds_fence();
#pragma unroll
            for (int e = 0; e < 2; ++e)
              write_out<MOM == kMomNone>(out, old[2 * p + e], kUnit, *(const float4 *)(X + (2 * (r + 8 * e) + (c >> 2)) * xrow + 64 * jp + (c & 3) * 16));
            wave_lds_fence();
          }
        }
      }
    }
  };
  MuonOld one[4], two[4];
  if (kAhead) {
    if (wave < S.mp / 32) spots(wave, 0, one);
    for (int jp = wave; jp < S.mp / 32; jp += 2 * kSmallWaves) {
      emit(jp, one, two);
      if (jp + kSmallWaves < S.mp / 32) emit(jp + kSmallWaves, two, one);
    }
  } else {
    for (int jp = wave; jp < S.mp / 32; jp += kSmallWaves) emit(jp, one, two);
  }
}

// ------------------------------------------------------------------ reading the 8-bit momentum
__global__ __launch_bounds__(256) void momentum8_values_kernel(const int8_t *codes, const float *scales, float *out,
                                                               int64_t rows, int64_t cols, int vec) {
  const int lane = (int)(threadIdx.x & 63u), wave = (int)(threadIdx.x >> 6);
  const int64_t segs = (cols + 255) / 256, total = rows * segs;
  for (int64_t q = (int64_t)blockIdx.x * 4 + wave; q < total; q += (int64_t)gridDim.x * 4) {
    const int64_t i = q / segs, j = (q - i * segs) * 256 + 4 * lane, at = i * cols + j;
    const float s = scales[q];
    if (vec && j + 4 <= cols) {
      const uint32_t w = *(const uint32_t *)(codes + at);
      *(float4 *)(out + at) = make_float4((float)(int8_t)w * s, (float)(int8_t)(w >> 8) * s,
                                          (float)(int8_t)(w >> 16) * s, (float)(int8_t)(w >> 24) * s);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (j + e < cols) out[at + e] = (float)codes[at + e] * s;
    }
  }
}

}  // namespace microadam
