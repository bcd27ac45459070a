// AdamW over a list of tensors for gfx950: the norm of all gradients, the step
// with its moments in 32 bits, and the step with its moments in 8 bits.
//
// The list travels in the kernel's arguments (no copy to the device, nothing to
// keep alive, and a captured launch holds its own), cut into chunks that the
// workgroups take in turn.  State arrays are laid out in blocks of 256 elements,
// each tensor starting a block, so that they are aligned whatever the
// parameters are; parameters and gradients may begin at any element.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace adamw_many {

constexpr int kBlock = 256;      // elements of a tensor that share their 8-bit moments' scales
constexpr int kThreads = 256;
constexpr int kRun = 8;          // consecutive elements of a thread
constexpr int kChunk = kThreads * kRun;
constexpr int kTable = 112;      // tensors of a launch: its arguments stay below 4 KiB
constexpr int kNormTable = 184;
constexpr int kNormChunk = 4 * kChunk;
constexpr int kNormGroups = 1024;   // partial sums of a launch, at most

struct Table {
  void *param[kTable];
  const void *grad[kTable];
  int64_t n[kTable];
  uint32_t block[kTable];   // first block of its states
  uint32_t first[kTable];   // first chunk; 2^32 - 1 past the last tensor
  uint32_t chunks;
};

struct NormTable {
  const void *grad[kNormTable];
  int64_t n[kNormTable];      // negative: bf16, -n - 1 elements
  uint32_t first[kNormTable];
  uint32_t chunks;
};

struct StepArgs {
  double lr, b1, b2, eps, wd;
  int64_t t;
  const int64_t *t_dev;
  const float *lr_dev, *scale;
};
static_assert(sizeof(Table) + sizeof(StepArgs) + 64 <= 4096 && sizeof(NormTable) + 64 <= 4096, "kernel arguments of 4 KiB");

// The tensor that chunk c belongs to: the last one that begins at or before it.
// One load and one ballot for every 64 tensors.
template <int N>
__device__ __forceinline__ int find(const uint32_t (&first)[N], uint32_t c) {
  const int lane = (int)(threadIdx.x & 63u);
  int at = -1;
#pragma unroll
  for (int k = 0; k < N; k += 64)
    at += __popcll(__ballot(k + lane < N && first[k + lane < N ? k + lane : 0] <= c));
  return __builtin_amdgcn_readfirstlane(at);
}

// What a step's elements share.
struct Step {
  double b1, b2, omb1, omb2;   // the last two with the gradients' factor
  float scale, lr, wd, eps, c1, c2;
};

__device__ __forceinline__ double power(double b, int64_t e) {
  double p = 1.0;
  for (; e; e >>= 1, b *= b)
    if (e & 1) p *= b;
  return p;
}

// False for a step that changes nothing: a factor that is NaN (the norm was not
// finite) or a count below 1.
__device__ __forceinline__ bool constants(const StepArgs &A, Step &k) {
  const int64_t t = A.t_dev ? *A.t_dev : A.t;
  const float scale = A.scale ? *A.scale : 1.f;
  if (t < 1 || scale != scale) return false;
  k.b1 = A.b1;
  k.b2 = A.b2;
  k.omb1 = (1.0 - A.b1) * scale;
  k.omb2 = (1.0 - A.b2) * scale * scale;
  k.scale = scale;
  k.lr = A.lr_dev ? *A.lr_dev : (float)A.lr;
  k.wd = (float)A.wd;
  k.eps = (float)A.eps;
  k.c1 = (float)(1.0 / (1.0 - power(A.b1, t)));
  k.c2 = (float)sqrt(1.0 / (1.0 - power(A.b2, t)));
  return true;
}

// Eight consecutive elements that begin at any element: the hardware takes 16-byte
// accesses at any address.
typedef float Floats __attribute__((ext_vector_type(4), aligned(4)));
typedef __bf16 Halves __attribute__((ext_vector_type(8), aligned(2)));

__device__ __forceinline__ void load(const float *p, float (&x)[kRun]) {
  const Floats a = *reinterpret_cast<const Floats *>(p), b = *reinterpret_cast<const Floats *>(p + 4);
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = a[i], x[i + 4] = b[i];
}
__device__ __forceinline__ void load(const __bf16 *p, float (&x)[kRun]) {
  const Halves a = *reinterpret_cast<const Halves *>(p);
#pragma unroll
  for (int i = 0; i < kRun; ++i) x[i] = (float)a[i];
}
__device__ __forceinline__ void store(float *p, const float (&x)[kRun]) {
  *reinterpret_cast<Floats *>(p) = Floats{x[0], x[1], x[2], x[3]};
  *reinterpret_cast<Floats *>(p + 4) = Floats{x[4], x[5], x[6], x[7]};
}
__device__ __forceinline__ void store(__bf16 *p, const float (&x)[kRun]) {   // to nearest even, once
  Halves a;
#pragma unroll
  for (int i = 0; i < kRun; ++i) a[i] = (__bf16)x[i];
  *reinterpret_cast<Halves *>(p) = a;
}

// The first `left` (below eight) of them; zeros for the others.
template <class T> __device__ __forceinline__ void load(const T *p, int64_t left, float (&x)[kRun]) {
#pragma unroll
  for (int i = 0; i < kRun; ++i) x[i] = i < left ? (float)p[i] : 0.f;
}
template <class T> __device__ __forceinline__ void store(T *p, int64_t left, const float (&x)[kRun]) {
#pragma unroll
  for (int i = 0; i < kRun; ++i)
    if (i < left) p[i] = (T)x[i];
}

// p - lr (u + wd p): the decay is not rounded apart from the rest.
__device__ __forceinline__ float moved(const Step &k, float p, float u) { return fmaf(-k.lr, fmaf(k.wd, p, u), p); }

// ------------------------------------------------------------ moments in 32 bits

template <class P, class G, bool COPY>
__global__ __launch_bounds__(kThreads) void step_kernel(Table T, StepArgs A, float *copy, float *m, float *v) {
  Step k;
  if (!constants(A, k)) return;
  const float b1 = (float)k.b1, b2 = (float)k.b2, omb1 = (float)(1.0 - k.b1), omb2 = (float)(1.0 - k.b2);
  for (uint32_t c = blockIdx.x; c < T.chunks; c += gridDim.x) {
    const int i = find(T.first, c);
    const int64_t n = T.n[i], at = (int64_t)(c - T.first[i]) * kChunk + threadIdx.x * kRun;
    if (at >= n) continue;
    const int64_t s = (int64_t)T.block[i] * kBlock + at, left = n - at;
    const G *grad = static_cast<const G *>(T.grad[i]) + at;
    P *param = static_cast<P *>(T.param[i]) + at;
    float g[kRun], p[kRun], mm[kRun], vv[kRun];
    if (left >= kRun) {
      load(grad, g);
      if (COPY) load(copy + s, p); else load(param, p);
      load(m + s, mm);
      load(v + s, vv);
    } else {
      load(grad, left, g);
      if (COPY) load(copy + s, left, p); else load(param, left, p);
      load(m + s, left, mm);
      load(v + s, left, vv);
    }
#pragma unroll
    for (int e = 0; e < kRun; ++e) {
      const float x = g[e] * k.scale;
      mm[e] = fmaf(b1, mm[e], omb1 * x);
      vv[e] = fmaf(b2, vv[e], omb2 * x * x);
      p[e] = moved(k, p[e], (mm[e] * k.c1) / fmaf(sqrtf(vv[e]), k.c2, k.eps));
    }
    if (left >= kRun) {
      store(param, p);
      if (COPY) store(copy + s, p);
      store(m + s, mm);
      store(v + s, vv);
    } else {
      store(param, left, p);
      if (COPY) store(copy + s, left, p);
      store(m + s, left, mm);
      store(v + s, left, vv);
    }
  }
}

// ------------------------------------------------------------- moments in 8 bits
// A block of 256 elements has two fp32 scales, sm = max |m| and sr = max sqrt(v).
// m is an int8 code c for sm c|c| / 127^2, sqrt(v) a uint8 code q for sr q^2 / 255^2:
// steps that grow with the value, so that m / sqrt(v) keeps a meaning far below a
// block's largest element, where even steps would read sqrt(v) as 0 and the
// update as m / eps.  A code is the nearest value's (of two equally near ones the
// larger); v > 0 never reads as 0.

constexpr double kM = 127.0 * 127.0, kR = 255.0 * 255.0;

// Half of a wave holds a block.
__device__ __forceinline__ uint32_t block_max(uint32_t x) {
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) x = max(x, (uint32_t)__shfl_xor((int)x, o, 64));
  return x;
}
__device__ __forceinline__ double block_max(double x) {
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) x = fmax(x, __shfl_xor(x, o, 64));
  return x;
}

// The code of the nearest c^2 to y, where exact(t) tells whether the value in 64
// bits has reached t.  In 32 bits sqrt(y - 1/4) is off by a few parts in 10^7 and
// rounds as the code does (between c^2 and (c-1)^2 lies (c - 1/2)^2 + 1/4), so
// only what is that near to a half asks again.
template <class F> __device__ __forceinline__ float nearest_code(float y, F exact) {
  const float s = __builtin_amdgcn_sqrtf(fmaxf(y - 0.25f, 0.f));
  float c = rintf(s);
  if (fabsf(s - c) > fmaf(s, -1e-6f, 0.5f)) {
    const float up = s > c ? c + 1.f : c;
    c = exact((double)(up * (up - 1.f)) + 0.5) ? up : up - 1.f;
  }
  return c;
}

template <class P, class G, bool COPY>
__global__ __launch_bounds__(kThreads) void step8_kernel(Table T, StepArgs A, float *copy, int8_t *cm, uint8_t *cv, float *sm,
                                                         float *sr) {
  Step k;
  if (!constants(A, k)) return;
  for (uint32_t c = blockIdx.x; c < T.chunks; c += gridDim.x) {
    const int i = find(T.first, c);
    const int64_t n = T.n[i], at = (int64_t)(c - T.first[i]) * kChunk + threadIdx.x * kRun;
    if ((at & ~(int64_t)(kBlock - 1)) >= n) continue;   // all 32 lanes of a block together
    const int64_t s = (int64_t)T.block[i] * kBlock + at, b = T.block[i] + at / kBlock, left = n - at;
    const G *grad = static_cast<const G *>(T.grad[i]) + at;
    P *param = static_cast<P *>(T.param[i]) + at;
    float g[kRun], p[kRun];
    if (left >= kRun) {
      load(grad, g);
      if (COPY) load(copy + s, p); else load(param, p);
    } else {
      load(grad, left, g);
      if (COPY) load(copy + s, left, p); else load(param, left, p);
    }
    const uint2 wm = *reinterpret_cast<const uint2 *>(cm + s), wv = *reinterpret_cast<const uint2 *>(cv + s);
    const double um = k.b1 * ((double)sm[b] * (1.0 / kM)), ur = (double)sr[b] * (1.0 / kR), uv = k.b2 * (ur * ur);
    double m[kRun], v[kRun];
    uint32_t top = 0;
    double vtop = 0.0;
#pragma unroll
    for (int e = 0; e < kRun; ++e) {
      const float a = (float)(int8_t)((e < 4 ? wm.x : wm.y) >> (8 * (e & 3)));
      const float q = (float)(uint8_t)((e < 4 ? wv.x : wv.y) >> (8 * (e & 3)));
      const double x = g[e], q2 = q * q;
      m[e] = fma((double)(a * fabsf(a)), um, x * k.omb1);
      v[e] = fma(q2 * q2, uv, x * x * k.omb2);
      if (e < left) {
        // a pattern above infinity's for a NaN, in m or in v; sqrt(1e76) is in fp32's range
        const bool fine = v[e] < 1e76;
        top = max(top, fine ? __float_as_uint((float)m[e]) & 0x7fffffffu : 0x7fc00000u);
        vtop = fmax(vtop, fine ? v[e] : 0.0);
      }
    }
    top = block_max(top);
    vtop = block_max(vtop);
    const bool bad = top >= 0x7f800000u;
    const float am = __uint_as_float(top), ar = (float)sqrt(vtop);
    // Estimates of the codes' values, and with them of sqrt(v), in 32 bits: good to 2^-22.
    // y^2 carries a factor of 2^64, so that no v that counts beside eps vanishes.
    const double im = am > 0.f ? kM * __builtin_amdgcn_rcp((double)am) : 0.0, ir = ar > 0.f ? kR * __builtin_amdgcn_rcp((double)ar) : 0.0;
    const double iv = ir * ir * 0x1p64, dr = (double)ar * (1.0 / kR);
    const float back = ar * (float)(0x1p-32 / kR) * k.c2;
    uint32_t om[2] = {0, 0}, ov[2] = {0, 0};
#pragma unroll
    for (int e = 0; e < kRun; ++e) {
      const float y = __builtin_amdgcn_sqrtf((float)(v[e] * iv));
      p[e] = moved(k, p[e], ((float)m[e] * k.c1) / fmaf(y, back, k.eps));
      const float a = fminf(nearest_code((float)(fabs(m[e]) * im), [&](double t) { return fabs(m[e]) * kM >= t * am; }), 127.f);
      float q = fminf(nearest_code(y * 0x1p-32f, [&](double t) { return v[e] >= (t * dr) * (t * dr); }), 255.f);
      if (v[e] > 0.0) q = fmaxf(q, 1.f);
      om[e >> 2] |= ((uint32_t)(int)(m[e] < 0.0 ? -a : a) & 0xffu) << (8 * (e & 3));
      ov[e >> 2] |= (uint32_t)q << (8 * (e & 3));
    }
    if (bad || am == 0.f) om[0] = om[1] = 0;
    if (bad || ar == 0.f) ov[0] = ov[1] = 0;
    if (left >= kRun) {
      store(param, p);
      if (COPY) store(copy + s, p);
      *reinterpret_cast<uint2 *>(cm + s) = make_uint2(om[0], om[1]);
      *reinterpret_cast<uint2 *>(cv + s) = make_uint2(ov[0], ov[1]);
    } else {
      store(param, left, p);
      if (COPY) store(copy + s, left, p);
#pragma unroll
      for (int e = 0; e < kRun; ++e)
        if (e < left) {
          cm[s + e] = (int8_t)(om[e >> 2] >> (8 * (e & 3)));
          cv[s + e] = (uint8_t)(ov[e >> 2] >> (8 * (e & 3)));
        }
    }
    if ((threadIdx.x & 31u) == 0) {
      sm[b] = bad ? __builtin_nanf("") : am;
      sr[b] = bad ? __builtin_nanf("") : ar;
    }
  }
}

// The moments that an 8-bit state stands for; blocks of 256, one half wave each.
__global__ __launch_bounds__(kThreads) void values8_kernel(const int8_t *cm, const uint8_t *cv, const float *sm, const float *sr,
                                                           float *m, float *v, int64_t blocks) {
  const int64_t stride = (int64_t)gridDim.x * (kChunk / kBlock);
  for (int64_t b = (int64_t)blockIdx.x * (kChunk / kBlock) + threadIdx.x / 32; b < blocks; b += stride) {
    const int64_t at = b * kBlock + (threadIdx.x & 31u) * kRun;
    const uint2 wm = *reinterpret_cast<const uint2 *>(cm + at), wv = *reinterpret_cast<const uint2 *>(cv + at);
    const double um = (double)sm[b] * (1.0 / kM), ur = (double)sr[b] * (1.0 / kR);
    float mm[kRun], vv[kRun];
#pragma unroll
    for (int e = 0; e < kRun; ++e) {
      const float a = (float)(int8_t)((e < 4 ? wm.x : wm.y) >> (8 * (e & 3)));
      const float q = (float)(uint8_t)((e < 4 ? wv.x : wv.y) >> (8 * (e & 3)));
      const double r = (double)(q * q) * ur;
      mm[e] = (float)((double)(a * fabsf(a)) * um);
      vv[e] = (float)(r * r);
    }
    store(m + at, mm);
    store(v + at, vv);
  }
}

// ------------------------------------------------------ the norm of all gradients
// Squares and sums in 64 bits: no gradient's square overflows or vanishes, and the
// order of the sums, fixed by the list, shows in no bit of a 32-bit result.

__device__ __forceinline__ double group_sum(double x, double *lds) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) x += __shfl_xor(x, o, 64);
  if ((threadIdx.x & 63u) == 0) lds[threadIdx.x >> 6] = x;
  __syncthreads();
  double s = 0.0;
#pragma unroll
  for (int w = 0; w < kThreads / 64; ++w) s += lds[w];
  return s;
}

template <class G> __device__ __forceinline__ double squares(const G *g, int64_t at, int64_t n) {
  double s = 0.0;
  for (int64_t e = at + threadIdx.x * kRun; e < at + kNormChunk && e < n; e += kChunk) {
    float x[kRun];
    if (n - e >= kRun) load(g + e, x); else load(g + e, n - e, x);
#pragma unroll
    for (int i = 0; i < kRun; ++i) s = fma((double)x[i], (double)x[i], s);
  }
  return s;
}

__global__ __launch_bounds__(kThreads) void norm_kernel(NormTable T, double *partial) {
  __shared__ double lds[kThreads / 64];
  double s = 0.0;
  for (uint32_t c = blockIdx.x; c < T.chunks; c += gridDim.x) {
    const int i = find(T.first, c);
    const int64_t n = T.n[i], at = (int64_t)(c - T.first[i]) * kNormChunk;
    s += n < 0 ? squares(static_cast<const __bf16 *>(T.grad[i]), at, -n - 1) : squares(static_cast<const float *>(T.grad[i]), at, n);
  }
  s = group_sum(s, lds);
  if (threadIdx.x == 0) partial[blockIdx.x] = s;
}

__global__ __launch_bounds__(kThreads) void norm_finish_kernel(const double *partial, int64_t parts, double max_norm, float *out,
                                                               int64_t *t) {
  __shared__ double lds[kThreads / 64];
  double s = 0.0;
  for (int64_t i = threadIdx.x; i < parts; i += kThreads) s += partial[i];
  s = group_sum(s, lds);
  if (threadIdx.x == 0) {
    const double norm = sqrt(s);
    const bool finite = norm < __builtin_inf();
    out[0] = (float)norm;
    out[1] = finite ? (float)fmin(1.0, max_norm / (norm + 1e-6)) : __builtin_nanf("");
    if (t && finite) ++*t;
  }
}

}  // namespace adamw_many
