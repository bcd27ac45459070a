// AdamW over a list of tensors for gfx950: the norm of all gradients, the step
// with its moments in 32 bits, and the step with its moments in 8 bits.
//
// The list travels in the kernel's arguments (no copy to the device, nothing to
// keep alive, and a captured launch holds its own), cut into chunks.  State arrays
// are laid out in blocks of 256 elements, each tensor starting a block, so that
// they are aligned whatever the parameters are; parameters and gradients may
// begin at any element.
//
// All of it is bound by memory, short lists by the launch: the norm reads 2 or 4 bytes an
// element, the step moves 22 to 30 with some 45 vector instructions, the 8-bit step 10
// to 18 with some 55.  The steps give each workgroup one chunk: in a loop, a wave's
// next loads would wait for its last stores, which retire in order with them (51.8
// million fp32 parameters: 279 us with 2048 workgroups in a loop, 251 with one chunk
// each, 5.4 TB/s; 405 million bf16 ones with copies 2290 and 2140, 5.3 TB/s; a copy of
// 1 GiB runs at 5.1).  Loads that bypass the caches
// made the steps 4% slower, such stores 0.5% faster but reading 8-bit moments twice
// as slow: neither is used.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace adamw_many {

constexpr int kBlock = 256;      // elements of a tensor that share their 8-bit moments' scales
constexpr int kThreads = 256;
constexpr double kM = 127.0 * 127.0, kR = 255.0 * 255.0;   // what the largest 8-bit codes stand for, in units of the smallest
constexpr int kRun = 8;          // consecutive elements of a thread
constexpr int kChunk = kThreads * kRun;
constexpr int kTable = 140;      // tensors of a launch: as many as its 4 KiB of arguments hold
constexpr int kNormTable = 250;
constexpr int64_t kEntry = int64_t(1) << 30;   // elements of an entry: a longer tensor takes several
constexpr uint32_t kMostChunks = 1u << 23;     // of a launch: a grid may have 2^32 - 1 threads
constexpr int kNormRuns = 4, kNormChunk = kNormRuns * kChunk;
constexpr int kSmallThreads = 1024, kSmallSpan = 64 * kRun, kSmallChunk = kNormRuns * kSmallSpan;
constexpr int kSmallChunks = 64;   // of a list that one workgroup takes, at most
constexpr int kNormGroups = 512;   // workgroups of a launch, at most: two to a CU

struct Table {
  void *param[kTable];
  const void *grad[kTable];
  uint32_t n[kTable];
  uint32_t block[kTable];   // first block of its states
  uint32_t first[kTable];   // first chunk; 2^32 - 1 past the last tensor
  uint32_t chunks;
};

constexpr uint32_t kIsBf16 = 1u << 31;

struct NormTable {
  const void *grad[kNormTable];
  uint32_t n[kNormTable];   // with kIsBf16 where it is
  uint32_t first[kNormTable];
  uint32_t chunks;
};

struct StepArgs {
  double b1, b2, um, uv;       // um, uv: beta1 and beta2 in the units of 8-bit codes
  float lr, eps, wd, c1, c2;   // the last two of t
  const int64_t *t_dev;
  const float *lr_dev, *scale;
};
static_assert(sizeof(Table) + sizeof(StepArgs) + 64 <= 4096 && sizeof(NormTable) + 64 <= 4096, "kernel arguments of 4 KiB");

// Finds the tensor that a chunk belongs to: the last one that begins at or before it.  Each lane
// holds the begin of every 64th tensor; a ballot counts those up to the chunk.
template <int N> struct Finder {
  uint32_t first[(N + 63) / 64];
  __device__ __forceinline__ explicit Finder(const uint32_t (&begins)[N]) {
#pragma unroll
    for (int k = 0; k < (N + 63) / 64; ++k) {
      const int i = 64 * k + (int)(threadIdx.x & 63u);
      first[k] = begins[min(i, N - 1)];
      if (i >= N) first[k] = ~0u;
    }
  }
  __device__ __forceinline__ int operator()(uint32_t c) const {
    int at = -1;
#pragma unroll
    for (int k = 0; k < (N + 63) / 64; ++k) at += __popcll(__ballot(first[k] <= c));
    return at;
  }
};

// What a step's elements share.
struct Step {
  double b1, b2, omb1, omb2;   // the last two with the gradients' factor
  float scale, lr, wd, eps, c1, c2;
};

// 1 / (1 - b1^t) and 1 / sqrt(1 - b2^t): by the same operations on the host, where t is known there.
__host__ __device__ inline double power(double b, int64_t e) {
  double p = 1.0;
  for (; e; e >>= 1, b *= b)
    if (e & 1) p *= b;
  return p;
}
__host__ __device__ inline float correction1(double b1, int64_t t) { return (float)(1.0 / (1.0 - power(b1, t))); }
__host__ __device__ inline float correction2(double b2, int64_t t) { return (float)(1.0 / sqrt(1.0 - power(b2, t))); }

// The same in all lanes: kept in scalar registers.
__device__ __forceinline__ float scalar(float x) { return __int_as_float(__builtin_amdgcn_readfirstlane(__float_as_int(x))); }
__device__ __forceinline__ double scalar(double x) {
  return __hiloint2double(__builtin_amdgcn_readfirstlane(__double2hiint(x)), __builtin_amdgcn_readfirstlane(__double2loint(x)));
}

// False for a step that changes nothing: a factor that is NaN (the norm was not
// finite) or a count below 1.
__device__ __forceinline__ bool constants(const StepArgs &A, Step &k) {
  const float scale = A.scale ? *A.scale : 1.f;
  if (scale != scale) return false;
  k.c1 = A.c1;
  k.c2 = A.c2;
  if (A.t_dev) {
    const int64_t t = *A.t_dev;
    if (t < 1) return false;
    k.c1 = scalar(correction1(A.b1, t));
    k.c2 = scalar(correction2(A.b2, t));
  }
  k.b1 = A.b1;
  k.b2 = A.b2;
  k.omb1 = scalar((1.0 - A.b1) * scale);
  k.omb2 = scalar((1.0 - A.b2) * scale * scale);
  k.scale = scale;
  k.lr = A.lr_dev ? *A.lr_dev : A.lr;
  k.wd = A.wd;
  k.eps = A.eps;
  return true;
}

// Pointers to device memory.  at(): to a lane's element, `lane` behind the first, which is the
// same in all lanes and stays in scalar registers, with a 32-bit offset in bytes behind it.
// Called where the access is: the compiler would rather keep a 64-bit address for each
// array in vector registers (18 of them in the 8-bit step).
template <class T> struct DeviceMemory { typedef __attribute__((address_space(1))) T type; };
template <class T> using Device = typename DeviceMemory<T>::type;
template <class T, class V> __device__ __forceinline__ Device<T> *at(V *array, int64_t first, uint32_t lane) {
  Device<T> *p = (Device<T> *)((T *)array + first);
  uint32_t bytes = lane * (uint32_t)sizeof(T);
  asm volatile("" : "+s"(p), "+v"(bytes));
  return (Device<T> *)((Device<const char> *)p + bytes);
}

// Eight consecutive elements that begin at any element: the hardware takes 16-byte
// accesses at any address.
typedef float Floats __attribute__((ext_vector_type(4), aligned(4)));
typedef __bf16 Halves __attribute__((ext_vector_type(8), aligned(2)));
typedef uint32_t Words __attribute__((ext_vector_type(2), aligned(8)));

__device__ __forceinline__ void load(const Device<float> *p, float (&x)[kRun]) {
  const Floats a = *(const Device<Floats> *)p, b = *(const Device<Floats> *)(p + 4);
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = a[i], x[i + 4] = b[i];
}
__device__ __forceinline__ void load(const Device<__bf16> *p, float (&x)[kRun]) {
  const Halves a = *(const Device<Halves> *)p;
#pragma unroll
  for (int i = 0; i < kRun; ++i) x[i] = (float)a[i];
}
__device__ __forceinline__ void store(Device<float> *p, const float (&x)[kRun]) {
  *(Device<Floats> *)p = Floats{x[0], x[1], x[2], x[3]};
  *(Device<Floats> *)(p + 4) = Floats{x[4], x[5], x[6], x[7]};
}
__device__ __forceinline__ void store(Device<__bf16> *p, const float (&x)[kRun]) {   // to nearest even, once
  Halves a;
#pragma unroll
  for (int i = 0; i < kRun; ++i) a[i] = (__bf16)x[i];
  *(Device<Halves> *)p = a;
}

// The first `left` (below eight) of them; zeros for the others.
template <class T> __device__ __forceinline__ void load(const T *p, int left, float (&x)[kRun]) {
#pragma unroll
  for (int i = 0; i < kRun; ++i) x[i] = i < left ? (float)p[i] : 0.f;
}
template <class T> __device__ __forceinline__ void store(T *p, int left, const float (&x)[kRun]) {
#pragma unroll
  for (int i = 0; i < kRun; ++i)
    if (i < left) p[i] = (T)x[i];
}

// p - lr (u + wd p): the decay is not rounded apart from the rest.
__device__ __forceinline__ float moved(const Step &k, float p, float u) { return fmaf(-k.lr, fmaf(k.wd, p, u), p); }

// ------------------------------------------------------------ moments in 32 bits
// In fp32 throughout, each operation rounded once; 48 registers, eight waves a SIMD.  (Runs
// of four elements, so that an access covers whole lines, were 8% faster where the list fits
// the last cache and 2% slower where it does not.)

template <class P, class G, bool COPY>
__global__ __launch_bounds__(kThreads) void step_kernel(Table T, StepArgs A, float *copies, float *ms, float *vs) {
  Step k;
  if (!constants(A, k)) return;
  const float b1 = scalar((float)k.b1), b2 = scalar((float)k.b2), omb1 = scalar((float)(1.0 - k.b1)), omb2 = scalar((float)(1.0 - k.b2));
  const uint32_t c = blockIdx.x;
  const int i = Finder<kTable>(T.first)(c);
  // where the chunk begins is the same in all lanes, what a lane adds the same in all chunks
  const int64_t from = (int64_t)(c - T.first[i]) * kChunk;
  const uint32_t o = threadIdx.x * kRun;
  const int left = (int)min((int64_t)T.n[i] - from, (int64_t)kChunk) - (int)o;
  if (left <= 0) return;
  const int64_t state = (int64_t)T.block[i] * kBlock + from;
  float g[kRun], p[kRun], m[kRun], v[kRun];
  if (left >= kRun) {
    load(at<const G>(T.grad[i], from, o), g);
    if (COPY) load(at<float>(copies, state, o), p); else load(at<P>(T.param[i], from, o), p);
    load(at<float>(ms, state, o), m);
    load(at<float>(vs, state, o), v);
  } else {
    load(at<const G>(T.grad[i], from, o), left, g);
    if (COPY) load(at<float>(copies, state, o), left, p); else load(at<P>(T.param[i], from, o), left, p);
    load(at<float>(ms, state, o), left, m);
    load(at<float>(vs, state, o), left, v);
  }
#pragma unroll
  for (int e = 0; e < kRun; ++e) {
    const float x = g[e] * k.scale;
    m[e] = fmaf(b1, m[e], omb1 * x);
    v[e] = fmaf(b2, v[e], omb2 * x * x);
    p[e] = moved(k, p[e], (m[e] * k.c1) / fmaf(sqrtf(v[e]), k.c2, k.eps));
  }
  if (left >= kRun) {
    store(at<P>(T.param[i], from, o), p);
    if (COPY) store(at<float>(copies, state, o), p);
    store(at<float>(ms, state, o), m);
    store(at<float>(vs, state, o), v);
  } else {
    store(at<P>(T.param[i], from, o), left, p);
    if (COPY) store(at<float>(copies, state, o), left, p);
    store(at<float>(ms, state, o), left, m);
    store(at<float>(vs, state, o), left, v);
  }
}

// ------------------------------------------------------------- moments in 8 bits
// A block of 256 elements has two fp32 scales, sm = max |m| and sr = max sqrt(v).
// m is an int8 code c for sm c|c| / 127^2, sqrt(v) a uint8 code q for sr q^2 / 255^2:
// steps that grow with the value, so that m / sqrt(v) keeps a meaning far below a
// block's largest element, where even steps would read sqrt(v) as 0 and the
// update as m / eps.  A code is the nearest value's (of two equally near ones the
// larger); v > 0 never reads as 0.

// Half of a wave holds a block, a lane eight elements.  (16 lanes with 16 elements each would
// share the work on maxima and scales better, but took 186 registers, two waves a SIMD:
// 772 us instead of 651 for 262 million bf16 parameters at that state of the kernel.)  The
// lanes' neighbours are read without going through LDS.
constexpr int kLanes = kBlock / kRun;
constexpr double kUp = 0x1p64, kDown = 0x1p-32;   // factor of m and v, and the inverse of its root

template <int CTRL> __device__ __forceinline__ uint32_t from_lane(uint32_t x) {
  return (uint32_t)__builtin_amdgcn_mov_dpp((int)x, CTRL, 0xf, 0xf, true);
}
template <int CTRL> __device__ __forceinline__ double from_lane(double x) {
  return __hiloint2double((int)from_lane<CTRL>((uint32_t)__double2hiint(x)), (int)from_lane<CTRL>((uint32_t)__double2loint(x)));
}
__device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) { return max(a, b); }
__device__ __forceinline__ double larger(double a, double b) {   // of numbers, or b: fmax() first quiets both
  double c;
  asm("v_max_f64 %0, %1, %2" : "=v"(c) : "v"(a), "v"(b));
  return c;
}
// the two rows of 16 of a half wave: the swap gives one row's value to both in `a`, the other's in `b`
__device__ __forceinline__ uint32_t rows_max(uint32_t x) {
  const auto r = __builtin_amdgcn_permlane16_swap(x, x, false, false);
  return larger(r[0], r[1]);
}
__device__ __forceinline__ double rows_max(double x) {
  const uint32_t hi = (uint32_t)__double2hiint(x), lo = (uint32_t)__double2loint(x);
  const auto h = __builtin_amdgcn_permlane16_swap(hi, hi, false, false), l = __builtin_amdgcn_permlane16_swap(lo, lo, false, false);
  return larger(__hiloint2double((int)h[0], (int)l[0]), __hiloint2double((int)h[1], (int)l[1]));
}
// lanes 1 and 2 apart by permuting, then by mirroring, then the two rows
template <class T> __device__ __forceinline__ T block_max(T x) {
  x = larger(x, from_lane<0xb1>(x));    // quad_perm 1 0 3 2
  x = larger(x, from_lane<0x4e>(x));    // quad_perm 2 3 0 1
  x = larger(x, from_lane<0x141>(x));   // row_half_mirror
  x = larger(x, from_lane<0x140>(x));   // row_mirror
  return rows_max(x);
}

// sqrt(x) of a positive x far from the ends of the range of 64 bits, to its last bits, by
// Goldschmidt's iteration (the library's root guards those ends).
__device__ __forceinline__ double root(double x) {
  const double r = __builtin_amdgcn_rsq(x);
  double s = x * r, h = 0.5 * r;
  const double e = fma(-h, s, 0.5);
  s = fma(s, e, s), h = fma(h, e, h);
  return fma(fma(-s, s, x), h, s);
}

// The code of the nearest c^2 to y is sqrt(y - 1/4) rounded: between c^2 and (c-1)^2 lies
// (c - 1/2)^2 + 1/4.  Adding 1.5 2^23 rounds to a whole number, to the even one half way, and
// leaves it in the low byte; so does the NaN of a y below 1/4, which holds a 0 there.
constexpr float kWhole = 12582912.f;
// Past 1/2 if s, which is off by up to 5.1e-7 of itself, is too near to a half for the whole number
// in t.  (In half steps of 2^-24: v and its product with iv 1 each, iv 6, halved by the root, which
// adds 2: y is off by 6 of them; doubled at worst by taking 1/4 off, plus 1, halved again, plus 2.)
__device__ __forceinline__ float doubt(float s, float t) { return fmaf(fabsf(s), 6e-7f, fabsf(s - (t - kWhole))); }
__device__ __forceinline__ float signed_like(float c, double m) { return copysignf(c, __int_as_float(__double2hiint(m))); }
// Four whole numbers' low bytes.
__device__ __forceinline__ uint32_t bytes(const float (&t)[kRun], int e) {
  const uint32_t lo = __builtin_amdgcn_perm(__float_as_uint(t[e + 1]), __float_as_uint(t[e]), 0x0c0c0400u);
  const uint32_t hi = __builtin_amdgcn_perm(__float_as_uint(t[e + 3]), __float_as_uint(t[e + 2]), 0x0c0c0400u);
  return __builtin_amdgcn_perm(hi, lo, 0x05040100u);
}
// 1/x, x far from the ends of the range of 32 bits, to its last bit.
__device__ __forceinline__ float inverse(float x) {
  const float r = __builtin_amdgcn_rcpf(x);
  return fmaf(fmaf(-x, r, 1.f), r, r);
}
// 0x80 in each byte of w that is 0, and perhaps in a 1 above such a one.
__device__ __forceinline__ uint32_t zero_bytes(uint32_t w) { return (w - 0x01010101u) & ~w & 0x80808080u; }
// The larger of the two whole numbers that s lies between if x is at least half way from the lower one's
// square to its own, in units of 1/`all` of `top`; decided in 64 bits.
__device__ __forceinline__ float decided(float s, double x, double top, double all) {
  const float up = ceilf(s);
  return x * all >= ((double)(up * (up - 1.f)) + 0.5) * top ? up : fmaxf(up - 1.f, 0.f);
}

// What is left of a word of four codes when only the first `left` count.
__device__ __forceinline__ uint32_t kept(uint32_t w, int left) {
  return left >= 4 ? w : left <= 0 ? 0u : w & ((1u << (8 * left)) - 1u);
}

// Written down plainly, this is bound by instructions: 960 us for 262 million bf16 parameters,
// whose bytes take 517 at a copy's rate.  64-bit operations cost what 32-bit ones do (4 cycles a
// wave; additions and products in 32 bits less), so moments are formed in 64 bits; what follows
// goes by 32-bit estimates of the codes' roots, good to a few parts in 10^7, and a lane with
// an element nearer to a border than that (one in 600) decides its codes again in 64 bits.
// 1/x and roots are the hardware's estimates: the update is off by a few parts in 10^7 of
// itself.  443 instructions a wave and 8 elements, 89 registers, five waves a SIMD (with four
// the same time, with six, and registers in memory, 545 us): 508 us in the fastest of a trace's
// calls, 530 in the median one, 5.0 TB/s.
template <class P, class G, bool COPY>
__global__ __launch_bounds__(kThreads, 5) void step8_kernel(Table T, StepArgs A, float *copies, int8_t *cm, uint8_t *cv, float *sm,
                                                            float *sr) {
  Step k;
  if (!constants(A, k)) return;
  // Moments are held 2^64 times as large (kUp): as 32-bit numbers they then reach down to m = 2^-190
  // and sqrt(v) = 2^-95.  u = m c1 / (sqrt(v) c2 + eps), with c1 and the 2^64 in the divisor.
  const float eps = scalar(k.eps * (float)kUp / k.c1), back0 = scalar((float)(kUp / kR) * k.c2 / k.c1);
  const double omb1 = scalar(k.omb1 * kUp), omb2 = scalar(k.omb2 * kUp);
  const uint32_t c = blockIdx.x;
  const int i = Finder<kTable>(T.first)(c);
  const int64_t from = (int64_t)(c - T.first[i]) * kChunk, block = T.block[i] + from / kBlock, state = block * kBlock;
  const uint32_t o = threadIdx.x * kRun, b = threadIdx.x / kLanes;
  const int rest = (int)min((int64_t)T.n[i] - from, (int64_t)kChunk), left = rest - (int)o;
  if ((int)(b * kBlock) >= rest) return;   // a block's lanes together
  const void *const grad = T.grad[i];
  void *const param = T.param[i];
  float g[kRun], p[kRun];
  // (first, so that nothing waits before all loads are on their way)
  Words wm = *(const Device<Words> *)at<int8_t>(cm, state, o), wv = *(const Device<Words> *)at<uint8_t>(cv, state, o);
  const float om = *at<float>(sm, block, b), ov = *at<float>(sr, block, b);
  if (left >= kRun) {
    load(at<const G>(grad, from, o), g);
    if (COPY) load(at<float>(copies, state, o), p); else load(at<P>(param, from, o), p);
  } else {
    load(at<const G>(grad, from, o), left, g);
    if (COPY) load(at<float>(copies, state, o), left, p); else load(at<P>(param, from, o), left, p);
    // what lies behind the tensor counts as nothing
    wm = Words{kept(wm.x, left), kept(wm.y, left - 4)}, wv = Words{kept(wv.x, left), kept(wv.y, left - 4)};
  }
  const double um = A.um * om, uv = A.uv * ((double)ov * (double)ov);
  double m[kRun], v[kRun], vtop = 0.0;
  float m32[kRun], v32[kRun];
  uint32_t top = 0;   // of |m| as a pattern: infinity's or above it for what is not finite
#pragma unroll
  for (int e = 0; e < kRun; ++e) {
    const float a = (float)(int8_t)((e < 4 ? wm.x : wm.y) >> (8 * (e & 3)));
    const uint32_t q = (uint8_t)((e < 4 ? wv.x : wv.y) >> (8 * (e & 3)));
    const double x = g[e], q2 = __umul24(q, q);
    m[e] = fma((double)(a * fabsf(a)), um, x * omb1);
    v[e] = fma(q2 * q2, uv, x * x * omb2);
    vtop = larger(v[e], vtop);
    m32[e] = (float)m[e], v32[e] = (float)v[e];
    top = max(top, __float_as_uint(m32[e]) & 0x7fffffffu);
  }
  top = block_max(top);
  vtop = block_max(vtop);
  const float at32 = __uint_as_float(top);
  float am = at32 * (float)(1.0 / kUp), ar = vtop > 0.0 ? (float)(root(vtop) * kDown) : 0.f;
  // where 32 bits do for the estimates and for what sqrt(v) is beside eps, and sm is no subnormal number
  const bool near = (at32 == 0.f || at32 >= 0x1p-62f) && at32 < 0x1p95f && ar >= 0x1p-70f && ar < 0x1p31f && ov == ov && k.eps >= 0x1p-80f && k.eps < 0x1p60f;
  bool bad = false;
  uint32_t nm[2] = {0, 0}, nv[2] = {0, 0};
  float worst = 1.f;
  if (at32 == 0.f && ar == 0.f && ov == ov) {   // no gradient yet: rows of tokens that did not occur
    worst = 0.f;
#pragma unroll
    for (int e = 0; e < kRun; ++e) p[e] = moved(k, p[e], 0.f);
  } else if (near) {
    const float im = at32 > 0.f ? inverse(at32) * (float)kM : 0.f, ir = inverse(ar) * (float)(kR * kDown), iv = ir * ir, back = ar * back0;
    float ta[kRun], tq[kRun];
    worst = 0.f;
#pragma unroll
    for (int e = 0; e < kRun; ++e) {
      const float y = __builtin_amdgcn_sqrtf(v32[e] * iv);
      p[e] = moved(k, p[e], m32[e] * __builtin_amdgcn_rcpf(fmaf(y, back, eps)));
      const float a = signed_like(__builtin_amdgcn_sqrtf(fmaf(fabsf(m32[e]), im, -0.25f)), m[e]);
      const float q = __builtin_amdgcn_sqrtf(y - 0.25f);
      ta[e] = a + kWhole, tq[e] = q + kWhole;
      worst = fmaxf(worst, fmaxf(doubt(a, ta[e]), doubt(q, tq[e])));
    }
    nm[0] = bytes(ta, 0), nm[1] = bytes(ta, 4), nv[0] = bytes(tq, 0), nv[1] = bytes(tq, 4);
    const uint32_t z0 = zero_bytes(nv[0]), z1 = zero_bytes(nv[1]);
    if (z0 | z1) {   // v > 0 is not 0
      uint32_t one[2] = {0, 0};
#pragma unroll
      for (int e = 0; e < kRun; ++e) one[e >> 2] |= (v[e] > 0.0 ? 1u : 0u) << (8 * (e & 3));
      nv[0] |= z0 >> 7 & one[0], nv[1] |= z1 >> 7 & one[1];
    }
  }
  if (worst > 0.5f) {   // in 64 bits
    if (!near) {        // a block's lanes together
      double mtop = 0.0, none = 0.0;
#pragma unroll
      for (int e = 0; e < kRun; ++e) {
        mtop = larger(fabs(m[e]), mtop);
        none += 0.0 * m[e] + 0.0 * v[e];
        const double r = v[e] > 0.0 ? root(v[e]) : 0.0;
        p[e] = moved(k, p[e], (float)(m[e] * (1.0 / kUp)) * k.c1 / fmaf((float)(r * kDown), k.c2, k.eps));
        __builtin_amdgcn_sched_barrier(0);   // one after the other: rare, and not to cost the others registers
      }
      top = block_max(none == 0.0 ? __float_as_uint((float)(mtop * (1.0 / kUp))) : 0x7fc00000u);
      am = __uint_as_float(top);
      bad = top >= 0x7f800000u || !(ar < __builtin_inff());
    }
    float ta[kRun], tq[kRun];
    const double mt = (double)am * kUp, vt = (double)ar / kDown, ia = kM / mt, iq = kR / vt;
#pragma unroll
    for (int e = 0; e < kRun; ++e) {
      const double r = v[e] > 0.0 ? root(v[e]) : 0.0;
      // (a subnormal scale can lie well below the largest value)
      const float a = fminf(decided(__builtin_amdgcn_sqrtf(fmaxf((float)fma(fabs(m[e]), ia, -0.25), 0.f)), fabs(m[e]), mt, kM), 127.f);
      const float q = fminf(decided(__builtin_amdgcn_sqrtf(fmaxf((float)fma(r, iq, -0.25), 0.f)), r, vt, kR), 255.f);
      ta[e] = am > 0.f ? signed_like(a, m[e]) + kWhole : kWhole;
      tq[e] = ar > 0.f ? fmaxf(q, v[e] > 0.0 ? 1.f : 0.f) + kWhole : kWhole;
      __builtin_amdgcn_sched_barrier(0);
    }
    nm[0] = bytes(ta, 0), nm[1] = bytes(ta, 4), nv[0] = bytes(tq, 0), nv[1] = bytes(tq, 4);
    if (bad) nm[0] = nm[1] = nv[0] = nv[1] = 0;
  }
  if (left >= kRun) {
    store(at<P>(param, from, o), p);
    if (COPY) store(at<float>(copies, state, o), p);
    *(Device<Words> *)at<int8_t>(cm, state, o) = Words{nm[0], nm[1]};
    *(Device<Words> *)at<uint8_t>(cv, state, o) = Words{nv[0], nv[1]};
  } else {
    store(at<P>(param, from, o), left, p);
    if (COPY) store(at<float>(copies, state, o), left, p);
    const auto c8 = at<int8_t>(cm, state, o);
    const auto q8 = at<uint8_t>(cv, state, o);
#pragma unroll
    for (int e = 0; e < kRun; ++e)
      if (e < left) {
        c8[e] = (int8_t)(nm[e >> 2] >> (8 * (e & 3)));
        q8[e] = (uint8_t)(nv[e >> 2] >> (8 * (e & 3)));
      }
  }
  if (threadIdx.x % kLanes == 0) {
    *at<float>(sm, block, b) = bad ? __builtin_nanf("") : am;
    *at<float>(sr, block, b) = bad ? __builtin_nanf("") : ar;
  }
}

// The moments that an 8-bit state stands for; blocks of 256, one half wave each.  10 bytes an
// element, 8 of them written: 262 million in 450 us (5.8 TB/s; 714 with 2048 workgroups in a loop).
__global__ __launch_bounds__(kThreads) void values8_kernel(const int8_t *cm, const uint8_t *cv, const float *sm, const float *sr,
                                                           float *m, float *v, int64_t blocks) {
  const int64_t b = (int64_t)blockIdx.x * (kChunk / kBlock) + threadIdx.x / kLanes;
  if (b < blocks) {
    const int64_t at = b * kBlock + threadIdx.x % kLanes * kRun;
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
    store((Device<float> *)m + at, mm);
    store((Device<float> *)v + at, vv);
  }
}

// ------------------------------------------------------ the norm of all gradients
// Squares and sums in 64 bits, which cost what 32 do: no gradient's square overflows or
// vanishes, and the order of the sums, fixed by the list, next to never shows in a 32-bit result.

template <int THREADS> __device__ __forceinline__ double group_sum(double x) {
  __shared__ double lds[THREADS / 64];
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) x += __shfl_xor(x, o, 64);
  if ((threadIdx.x & 63u) == 0) lds[threadIdx.x >> 6] = x;
  __syncthreads();
  double s = 0.0;
#pragma unroll
  for (int w = 0; w < THREADS / 64; ++w) s += lds[w];
  return s;
}

// A workgroup takes chunks of kNormChunk elements in turn, kNormRuns runs of a thread at once: it
// only reads, so what counts is how many loads are on their way.  809 million bf16 gradients:
// 346 us with one load of a thread at a time (1024 groups); with four, 253 (6.4 TB/s) with 512
// groups (247 in a trace), 278 with 384, 263 with 1024, 276 with 8192; with eight 260 with 512, with two 351.
// Eight gradients as they are loaded: nothing waits for them before the first is widened.
template <class G> struct Raw;
template <> struct Raw<float> {
  Floats a = {}, b = {};
  __device__ __forceinline__ void load(const Device<float> *p) { a = *(const Device<Floats> *)p, b = *(const Device<Floats> *)(p + 4); }
  __device__ __forceinline__ float operator[](int i) const { return i < 4 ? a[i] : b[i - 4]; }
};
template <> struct Raw<__bf16> {
  Halves a = {};
  __device__ __forceinline__ void load(const Device<__bf16> *p) { a = *(const Device<Halves> *)p; }
  __device__ __forceinline__ float operator[](int i) const { return (float)a[i]; }
};

// SPAN: elements that the threads which take a chunk together have in one run.
template <class G, int SPAN> __device__ __forceinline__ double squares(const void *grad, int64_t from, int64_t rest, uint32_t o) {
  Raw<G> x[kNormRuns];
  double s[kNormRuns] = {};
  const int n = (int)min(rest, (int64_t)(kNormRuns * SPAN)), left = n - (int)o;
  if (n == kNormRuns * SPAN) {
#pragma unroll
    for (int r = 0; r < kNormRuns; ++r) x[r].load(at<const G>(grad, from + r * SPAN, o));
  } else {
#pragma unroll
    for (int r = 0; r < kNormRuns; ++r)
      if (left - r * SPAN >= kRun) x[r].load(at<const G>(grad, from + r * SPAN, o));
  }
#pragma unroll
  for (int i = 0; i < kRun; ++i)
#pragma unroll
    for (int r = 0; r < kNormRuns; ++r) s[r] = fma((double)x[r][i], (double)x[r][i], s[r]);
  const int last = n & (kRun - 1);
  if (last && (int)o == (n - last) % SPAN) {   // a few behind the last run of eight: one thread's
    float y[kRun];
    load(at<const G>(grad, from + n - last, 0), last, y);
#pragma unroll
    for (int i = 0; i < kRun; ++i) s[0] = fma((double)y[i], (double)y[i], s[0]);
  }
  double sum = s[0];
#pragma unroll
  for (int r = 1; r < kNormRuns; ++r) sum += s[r];
  return sum;
}

// The chunks first, first + step, ... of a table's, SPAN * kNormRuns elements each.
template <int SPAN> __device__ __forceinline__ double squares(const NormTable &T, uint32_t first, uint32_t step, uint32_t o) {
  double s = 0.0;
  const Finder<kNormTable> find(T.first);
  for (uint32_t c = first; c < T.chunks; c += step) {
    const int i = find(c);
    const int64_t from = (int64_t)(c - T.first[i]) * (SPAN * kNormRuns), rest = (int64_t)(T.n[i] & ~kIsBf16) - from;
    s += T.n[i] & kIsBf16 ? squares<__bf16, SPAN>(T.grad[i], from, rest, o) : squares<float, SPAN>(T.grad[i], from, rest, o);
  }
  return s;
}

__device__ __forceinline__ void finish(double sum, double max_norm, float *out, int64_t *t) {
  const double norm = sqrt(sum);
  const bool finite = norm < __builtin_inf();
  out[0] = (float)norm;
  out[1] = finite ? (float)fmin(1.0, max_norm / (norm + 1e-6)) : __builtin_nanf("");
  if (t && finite) ++*t;
}

__global__ __launch_bounds__(kThreads) void norm_kernel(NormTable T, double *partial, int old) {
  const double s = group_sum<kThreads>(squares<kChunk>(T, blockIdx.x, gridDim.x, threadIdx.x * kRun));
  if (threadIdx.x == 0) partial[blockIdx.x] = (int)blockIdx.x < old ? partial[blockIdx.x] + s : s;
}

__global__ __launch_bounds__(kThreads) void norm_finish_kernel(const double *partial, int parts, double max_norm, float *out,
                                                               int64_t *t) {
  double s = 0.0;
  for (int i = threadIdx.x; i < parts; i += kThreads) s += partial[i];
  s = group_sum<kThreads>(s);
  if (threadIdx.x == 0) finish(s, max_norm, out, t);
}

// A short list in one launch: one workgroup, each of whose waves takes chunks of its own.  Against two
// launches, one tensor takes 2.5 us on the GPU instead of 3.9 and 8.2 us of the host's time instead of
// 10.5; 32 chunks 4.0 instead of 4.7 and 8.8 instead of 11.1; 64 chunks 5.8 instead of 4.6 and
// 9.1 instead of 11.2; 120 chunks 8.9 instead of 4.7 (a CU reads 64 bytes a cycle): up to 64 then.
// That is for eager calls, which the host holds up: a captured one, without its time, is
// even at 45 chunks and 1.2 us slower than two launches would be at 64.
__global__ __launch_bounds__(kSmallThreads) void norm_small_kernel(NormTable T, double max_norm, float *out, int64_t *t) {
  const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  const double s = group_sum<kSmallThreads>(squares<kSmallSpan>(T, wave, kSmallThreads / 64, threadIdx.x % 64 * kRun));
  if (threadIdx.x == 0) finish(s, max_norm, out, t);
}

}  // namespace adamw_many
