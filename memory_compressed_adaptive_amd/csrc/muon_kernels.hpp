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
// Layout.  All products take both operands with the summed index contiguous.
// X X^T and A A (A is its own transpose) have that; P X needs X^T, so X is
// kept in both orientations.  Sides are padded with zeros to a multiple of the
// tile: products keep the padding zero, so the main loops have no bounds.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace microadam {

typedef _Float16 half8 __attribute__((ext_vector_type(8)));
typedef _Float16 half4 __attribute__((ext_vector_type(4)));
typedef float float16v __attribute__((ext_vector_type(16)));

constexpr float kScaleX = 16384.f;   // of X and of A
constexpr float kScaleP = 4096.f;
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

__device__ __forceinline__ uint16_t f32_bf16(float f) {
  const uint32_t u = __float_as_uint(f);
  if ((u & 0x7fffffffu) > 0x7f800000u) return (uint16_t)((u >> 16) | 0x40u);
  return (uint16_t)((u + 0x7fffu + ((u >> 16) & 1u)) >> 16);
}

// Four consecutive inputs of row i (columns j..j+3; zeros past the last).
__device__ __forceinline__ void load4_in(const MuonInput &I, int64_t b, int64_t i, int64_t j, float v[4]) {
  const int64_t at = b * I.x_batch + i * I.x_row + j;
  if (I.x_bf16) {
    const uint16_t *p = (const uint16_t *)I.x + at;
    if (I.vec && j + 4 <= I.c) {
      const uint2 w = *(const uint2 *)p;
      v[0] = __uint_as_float(w.x << 16);
      v[1] = __uint_as_float(w.x & 0xffff0000u);
      v[2] = __uint_as_float(w.y << 16);
      v[3] = __uint_as_float(w.y & 0xffff0000u);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = j + e < I.c ? bf16_f32(p[e]) : 0.f;
    }
  } else {
    const float *p = (const float *)I.x + at;
    if (I.vec && j + 4 <= I.c) {
      const float4 w = *(const float4 *)p;
      v[0] = w.x, v[1] = w.y, v[2] = w.z, v[3] = w.w;
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = j + e < I.c ? p[e] : 0.f;
    }
  }
}

// The new momentum and the matrix to orthogonalise at row i, columns j..j+3
// (zeros past the last column).  m64: the 8-bit form's momentum, which decides
// its codes.  It is formed in 64 bits: a code lies where a product and a sum
// would each have moved it in fp32 about once in 1e5 elements, and what is
// written is then what the formula gives, on any machine; the pass is bound by
// memory either way.
template <int MOM>
__device__ __forceinline__ void muon_elems(const MuonInput &I, int64_t b, int64_t i, int64_t j, float u[4],
                                           float m32[4], double m64[4]) {
  float g[4];
  load4_in(I, b, i, j, g);
  if (MOM == kMomNone) {
#pragma unroll
    for (int e = 0; e < 4; ++e) u[e] = g[e];
    return;
  }
  const float b32 = (float)I.beta, o32 = (float)(1.0 - I.beta);
  const int64_t at = (b * I.r + i) * I.c + j;
  if (MOM == kMom32) {
    float mo[4];
    if (I.vec && j + 4 <= I.c) {
      const float4 w = *(const float4 *)(I.mom + at);
      mo[0] = w.x, mo[1] = w.y, mo[2] = w.z, mo[3] = w.w;
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) mo[e] = j + e < I.c ? I.mom[at + e] : 0.f;
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) m32[e] = mo[e] * b32 + g[e] * o32;
  } else {
    const double s = (double)I.scales[(b * I.r + i) * ((I.c + kMomentumBlock - 1) / kMomentumBlock) + j / kMomentumBlock];
    uint32_t w = 0;
    if (I.vec && j + 4 <= I.c) {
      w = *(const uint32_t *)(I.codes + at);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (j + e < I.c) w |= (uint32_t)(uint8_t)I.codes[at + e] << (8 * e);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      // a block whose scale is NaN holds NaN; columns past the last hold 0
      m64[e] = j + e < I.c ? I.beta * ((double)(int8_t)(w >> (8 * e)) * s) + (1.0 - I.beta) * (double)g[e] : 0.0;
      m32[e] = (float)m64[e];
    }
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) u[e] = I.nesterov ? m32[e] * b32 + g[e] * o32 : m32[e];
}

// ------------------------------------------------------------------ |U|_F
// Sum of squares of U in 64 bits (a gradient's squares can pass either end of
// fp32's range): block p of matrix b writes part[b][p].  One wave takes runs of
// 256 columns of a row; no atomics, so results do not depend on timing.
template <int MOM>
__global__ __launch_bounds__(256) void muon_norm_kernel(MuonInput I, int64_t b0, double *part, int nparts) {
  const int lane = (int)(threadIdx.x & 63u), wave = (int)(threadIdx.x >> 6);
  const int64_t lb = blockIdx.y, b = b0 + lb;
  const int64_t segs = (I.c + 255) / 256, total = I.r * segs;
  double sum = 0.0;
  for (int64_t q = (int64_t)blockIdx.x * 4 + wave; q < total; q += (int64_t)nparts * 4) {
    const int64_t i = q / segs, j = (q - i * segs) * 256 + 4 * lane;
    if (j < I.c) {
      float u[4], m32[4];
      double m64[4];
      muon_elems<MOM>(I, b, i, j, u, m32, m64);
#pragma unroll
      for (int e = 0; e < 4; ++e) sum += (double)u[e] * (double)u[e];
    }
  }
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) sum += __shfl_xor(sum, o, 64);
  __shared__ double s[4];
  if (lane == 0) s[wave] = sum;
  __syncthreads();
  if (threadIdx.x == 0) part[lb * nparts + blockIdx.x] = (s[0] + s[1]) + (s[2] + s[3]);
}

// 2^14 / max(|U|_F, eps), by every thread of a 256-thread block
__device__ __forceinline__ double block_scale(const double *part, int nparts, float eps, double *s4) {
  const int lane = (int)(threadIdx.x & 63u), wave = (int)(threadIdx.x >> 6);
  double sum = 0.0;
  for (int p = (int)threadIdx.x; p < nparts; p += 256) sum += part[p];
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) sum += __shfl_xor(sum, o, 64);
  if (lane == 0) s4[wave] = sum;
  __syncthreads();
  const double norm = sqrt((s4[0] + s4[1]) + (s4[2] + s4[3]));
  return (double)kScaleX / (norm >= (double)eps || norm != norm ? norm : (double)eps);
}

// ------------------------------------------------------------------ momentum, X0
// Writes the new momentum, and X0 in both orientations: S (the stored one, sp
// columns to a row) and T (its transpose, tp to a row), zeros in the padding.
// A block of 256 threads takes 64 rows x 256 columns of the stored matrix: 4
// columns to a lane, so that a wave holds the 256 elements of an 8-bit block.
constexpr int kLoadRows = 64, kLoadCols = 256;

template <int MOM>
__global__ __launch_bounds__(256) void muon_load_kernel(MuonInput I, int64_t b0, const double *part, int nparts,
                                                        float eps, _Float16 *S, int64_t sp, _Float16 *T, int64_t tp) {
  __shared__ double s4[4];
  __shared__ _Float16 tile[kLoadRows][kLoadCols + 4];
  const int lane = (int)(threadIdx.x & 63u), wave = (int)(threadIdx.x >> 6);
  const int64_t lb = blockIdx.z, b = b0 + lb;
  const double scale = block_scale(part + lb * nparts, nparts, eps, s4);
  const int64_t i0 = (int64_t)blockIdx.y * kLoadRows, j0 = (int64_t)blockIdx.x * kLoadCols, j = j0 + 4 * lane;
  S += lb * sp * tp;
  T += lb * sp * tp;
  for (int q = wave; q < kLoadRows; q += 4) {
    const int64_t i = i0 + q;
    half4 h = {0, 0, 0, 0};
    if (i < I.r) {   // uniform in the wave
      float u[4], m32[4];
      double m64[4] = {0, 0, 0, 0};
      if (j < I.c) {
        muon_elems<MOM>(I, b, i, j, u, m32, m64);
#pragma unroll
        for (int e = 0; e < 4; ++e) h[e] = j + e < I.c ? (_Float16)(float)((double)u[e] * scale) : (_Float16)0.f;
      }
      const int64_t at = (b * I.r + i) * I.c + j;
      if (MOM == kMom32 && j < I.c) {
        if (I.vec && j + 4 <= I.c) {
          *(float4 *)(I.mom + at) = make_float4(m32[0], m32[1], m32[2], m32[3]);
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (j + e < I.c) I.mom[at + e] = m32[e];
        }
      }
      if (MOM == kMom8) {
        // the largest magnitude is 127 steps; a block with a non-finite value
        // gets the scale NaN and codes 0, and reads back as NaN
        double top = 0.0;
        bool bad = false;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          bad |= !(fabs(m64[e]) < __builtin_inf());
          top = fmax(top, fabs(m64[e]));
        }
#pragma unroll
        for (int o = 32; o >= 1; o >>= 1) top = fmax(top, __shfl_xor(top, o, 64));
        bad = __any(bad);
        const float step = bad ? __builtin_nanf("") : (float)(top / 127.0);
        const double inv = step > 0.f ? 1.0 / (double)step : 0.0;
        uint32_t w = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const double q8 = bad ? 0.0 : fmin(fmax(rint(m64[e] * inv), -127.0), 127.0);
          w |= ((uint32_t)(int32_t)q8 & 0xffu) << (8 * e);
        }
        if (j < I.c) {
          if (I.vec && j + 4 <= I.c) {
            *(uint32_t *)(I.codes + at) = w;
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (j + e < I.c) I.codes[at + e] = (int8_t)(w >> (8 * e));
          }
        }
        if (lane == 0 && j0 < I.c) I.scales[(b * I.r + i) * ((I.c + 255) / 256) + j0 / 256] = step;
      }
    }
    if (j < sp && i < tp) *(half4 *)(S + i * sp + j) = h;
    *(half4 *)&tile[q][4 * lane] = h;
  }
  __syncthreads();
  // transposed: 8 consecutive rows of a column to a lane, 8 lanes to a column
  const int rg = (int)(threadIdx.x & 7u);
  for (int cc = (int)(threadIdx.x >> 3); cc < kLoadCols; cc += 32) {
    half8 h;
#pragma unroll
    for (int e = 0; e < 8; ++e) h[e] = tile[8 * rg + e][cc];
    if (j0 + cc < sp && i0 + 8 * rg < tp) *(half8 *)(T + (j0 + cc) * tp + i0 + 8 * rg) = h;
  }
}

// ------------------------------------------------------------------ products
// D = L R^T with L (M x K) and R (N x K), K contiguous in both, fp32 sums.
enum {
  kGram = 0,    // A = X X^T:                     L = R = X
  kPoly = 1,    // P = a I + b A + c A A:         L = R = A
  kUpdate = 2,  // X <- P X in both orientations: L = X^T, R = P
  kOut = 3,     // the last X, written where the caller wants it
};

struct MuonProduct {
  const _Float16 *l, *r;
  int64_t l_mat, r_mat;     // elements from one matrix to the next
  int64_t k;                // and the row stride of both
  _Float16 *d, *dt;         // d: [N][M]; dt: [M][N] (kUpdate)
  int64_t m, n;
  float a, b, c;
  // kOut: element (n, m) goes to out[b][n][m], rows x cols of them
  void *out;
  int out_bf16, update;     // update: theta <- theta * decay - rate * x
  int64_t out_row, out_batch, rows, cols;
  float decay, rate;
  int64_t b0;
};

constexpr int kTile = 64;

// Four waves of 32 x 32 over a 64 x 64 tile.
template <int ROLE>
__global__ __launch_bounds__(256) void muon_product_kernel(MuonProduct A) {
  __shared__ _Float16 sl[kTile][kTile + 8], sr[kTile][kTile + 8];
  const int lane = (int)(threadIdx.x & 63u), wave = (int)(threadIdx.x >> 6);
  const int wm = (wave & 1) * 32, wn = (wave >> 1) * 32;
  const int64_t m0 = (int64_t)blockIdx.x * kTile, n0 = (int64_t)blockIdx.y * kTile, lb = blockIdx.z;
  if (ROLE <= kPoly && m0 > n0) return;   // symmetric: the other half is this one's mirror image
  const _Float16 *l = A.l + lb * A.l_mat + m0 * A.k, *r = A.r + lb * A.r_mat + n0 * A.k;
  float16v acc;
#pragma unroll
  for (int e = 0; e < 16; ++e) acc[e] = 0.f;
  for (int64_t k0 = 0; k0 < A.k; k0 += kTile) {
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int at = (int)threadIdx.x + q * 256, row = at >> 3, col = (at & 7) * 8;
      *(half8 *)&sl[row][col] = *(const half8 *)(l + row * A.k + k0 + col);
      *(half8 *)&sr[row][col] = *(const half8 *)(r + row * A.k + k0 + col);
    }
    __syncthreads();
#pragma unroll
    for (int kk = 0; kk < kTile; kk += 16) {
      const half8 x = *(const half8 *)&sl[wm + (lane & 31)][kk + (lane >> 5) * 8];
      const half8 y = *(const half8 *)&sr[wn + (lane & 31)][kk + (lane >> 5) * 8];
      acc = __builtin_amdgcn_mfma_f32_32x32x16_f16(x, y, acc, 0, 0, 0);
    }
    __syncthreads();
  }
  const int64_t nn = n0 + wn + (lane & 31);
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int64_t mm = m0 + wm + 8 * q + 4 * (lane >> 5);   // and the next three
    float v[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = acc[4 * q + e];
    if (ROLE == kOut) {
      if (nn >= A.rows) continue;
      const int64_t at = (A.b0 + lb) * A.out_batch + nn * A.out_row + mm;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (mm + e >= A.cols) continue;
        const float x = v[e] * (1.f / (kScaleX * kScaleP));
        if (A.out_bf16) {
          uint16_t *p = (uint16_t *)A.out + at + e;
          *p = f32_bf16(A.update ? bf16_f32(*p) * A.decay - A.rate * x : x);
        } else {
          float *p = (float *)A.out + at + e;
          *p = A.update ? *p * A.decay - A.rate * x : x;
        }
      }
      continue;
    }
    half4 h;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      float x;
      if (ROLE == kGram) x = v[e] * (1.f / kScaleX);
      if (ROLE == kUpdate) x = v[e] * (1.f / kScaleP);
      if (ROLE == kPoly) {
        const float s = (float)A.l[lb * A.l_mat + nn * A.k + mm + e];
        x = (A.b * (kScaleP / kScaleX)) * s + (A.c * (kScaleP / (kScaleX * kScaleX))) * v[e];
        if (nn == mm + e) x += A.a * kScaleP;
      }
      h[e] = (_Float16)x;
    }
    _Float16 *d = A.d + lb * A.m * A.n;
    *(half4 *)(d + nn * A.m + mm) = h;
    _Float16 *dt = ROLE == kUpdate ? A.dt + lb * A.m * A.n : d;
    if (ROLE == kUpdate || m0 < n0) {
#pragma unroll
      for (int e = 0; e < 4; ++e) dt[(mm + e) * A.n + nn] = h[e];
    }
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
