// Host side of the AdamW operators over many tensors (include/microadam.h):
// argument checks, the tables that the launches carry, and the launches.
#include <float.h>
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <cmath>
#include <exception>
#include <initializer_list>
#include <type_traits>
#include <vector>

#include "adamw_many_kernels.hpp"
#include "host.hpp"
#include "microadam.h"

using namespace adamw_many;
using microadam::clear_error;
using microadam::DeviceGuard;
using microadam::fail;

namespace {

constexpr int64_t kMost = int64_t(1) << 40;   // elements of a tensor, and of a state

bool type_ok(int t) { return t == MA_TYPE_F32 || t == MA_TYPE_BF16; }
bool misaligned(const void *p, int type) { return ((uintptr_t)p & (type == MA_TYPE_F32 ? 3u : 1u)) != 0; }
int64_t size_of(int type) { return type == MA_TYPE_F32 ? 4 : 2; }

int check_list(const char *who, int64_t count, const ma_tensor *tensors) {
  if (count < 0) return fail(MA_EINVAL, "%s: a negative count", who);
  if (count && !tensors) return fail(MA_EINVAL, "%s: null list", who);
  for (int64_t i = 0; i < count; ++i) {
    const ma_tensor &t = tensors[i];
    if (t.n < 0) return fail(MA_EINVAL, "%s: tensor %lld has a negative size", who, (long long)i);
    if (t.n > kMost) return fail(MA_EUNSUPPORTED, "%s: tensor %lld has more than 2^40 elements", who, (long long)i);
    if (!type_ok(t.g_type)) return fail(MA_EINVAL, "%s: tensor %lld: unknown type %d", who, (long long)i, (int)t.g_type);
    if (t.n && (!t.grad || misaligned(t.grad, t.g_type)))
      return fail(MA_EINVAL, "%s: tensor %lld: null or misaligned gradient", who, (long long)i);
  }
  return MA_OK;
}

struct Span {   // of memory that a call writes
  uintptr_t begin, end;
  Span(const void *p, uint64_t bytes) : begin((uintptr_t)p), end((uintptr_t)p + bytes) {}
  bool operator<(const Span &o) const { return begin < o.begin; }
  bool meets(const Span &o) const { return begin < o.end && o.begin < end; }
};

// What a step needs besides: states in order, and nothing that is written twice.
int check_step(const char *who, int64_t count, const ma_tensor *tensors, const ma_adamw_args *a, const float *copy, int64_t state_n,
               std::initializer_list<Span> states) {
  if (const int rc = check_list(who, count, tensors)) return rc;
  if (!a) return fail(MA_EINVAL, "%s: null arguments", who);
  if (!(a->beta1 >= 0.0 && a->beta1 < 1.0 && a->beta2 >= 0.0 && a->beta2 < 1.0))
    return fail(MA_EINVAL, "%s: beta1 and beta2 must be in [0, 1)", who);
  if (!(a->eps >= FLT_MIN && a->eps <= FLT_MAX)) return fail(MA_EINVAL, "%s: eps must be positive and finite (a normal fp32)", who);
  if (!std::isfinite(a->lr) || !(a->wd >= 0.0) || !std::isfinite(a->wd))
    return fail(MA_EINVAL, "%s: lr and wd must be finite, wd >= 0", who);
  if (!a->t_dev && a->t < 1) return fail(MA_EINVAL, "%s: t must be >= 1", who);
  if (((uintptr_t)a->t_dev & 7u) || ((uintptr_t)a->lr_dev & 3u) || ((uintptr_t)a->scale & 3u) || ((uintptr_t)copy & 15u))
    return fail(MA_EINVAL, "%s: misaligned pointer", who);
  if (state_n < 0 || state_n % kBlock) return fail(MA_EINVAL, "%s: the states' size must be a multiple of %d", who, kBlock);
  if (state_n > kMost) return fail(MA_EUNSUPPORTED, "%s: states of more than 2^40 elements", who);
  int64_t end = 0;
  std::vector<Span> spans;
  spans.reserve((size_t)count);
  bool sorted = true;
  for (int64_t i = 0; i < count; ++i) {
    const ma_tensor &t = tensors[i];
    if (!type_ok(t.p_type)) return fail(MA_EINVAL, "%s: tensor %lld: unknown type %d", who, (long long)i, (int)t.p_type);
    if (!t.n) continue;
    if (!t.param || misaligned(t.param, t.p_type))
      return fail(MA_EINVAL, "%s: tensor %lld: null or misaligned parameter", who, (long long)i);
    if (t.at < end || t.at % kBlock || t.at > state_n || t.n > state_n - t.at)
      return fail(MA_EINVAL, "%s: tensor %lld: its states must begin at a multiple of %d behind the last tensor's and end in the arrays",
                  who, (long long)i, kBlock);
    end = t.at + t.n;
    const Span s(t.param, (uint64_t)(t.n * size_of(t.p_type)));
    if (!spans.empty() && s.begin < spans.back().end) sorted = false;
    spans.push_back(s);
  }
  if (!sorted) std::sort(spans.begin(), spans.end());
  for (size_t i = 1; i < spans.size(); ++i)
    if (spans[i].meets(spans[i - 1])) return fail(MA_EINVAL, "%s: two parameters overlap", who);
  for (const Span *x = states.begin(); x != states.end(); ++x) {
    for (const Span *y = states.begin(); y != x; ++y)
      if (x->meets(*y)) return fail(MA_EINVAL, "%s: two of the states overlap", who);
    for (const Span &s : spans)
      if (x->meets(s)) return fail(MA_EINVAL, "%s: a state and a parameter overlap", who);
  }
  return MA_OK;
}

int device_of(hipStream_t stream, int *dev) {
  if (!stream || stream == hipStreamLegacy || stream == hipStreamPerThread) return hipGetDevice(dev) == hipSuccess ? MA_OK : MA_EHIP;
  return hipStreamGetDevice(stream, dev) == hipSuccess ? MA_OK : MA_EHIP;
}

// Runs f(), which returns a hipError_t, with the stream's device current.
template <class F> int on_device(const char *who, hipStream_t stream, F f) {
  int dev = 0;
  if (device_of(stream, &dev) != MA_OK) return fail(MA_EHIP, "%s: the stream has no device", who);
  DeviceGuard guard(dev);
  if (!guard.ok) return fail(MA_EHIP, "%s: device %d cannot be made current", who, dev);
  const hipError_t e = f();
  if (e != hipSuccess) return fail(MA_EHIP, "%s: launch failed: %s", who, hipGetErrorString(e));
  return MA_OK;
}

// Nothing may be thrown through the C boundary.
template <class F> int guarded(const char *who, F f) {
  clear_error();
  try {
    return f();
  } catch (const std::exception &) {   // of the list of parameters
    return fail(MA_ENOMEM, "%s: out of host memory", who);
  }
}

// launch(table) for every kTable entries of the tensors with these types.
template <class F> hipError_t each_table(int64_t count, const ma_tensor *tensors, int p_type, int g_type, F launch) {
  Table T;
  int used = 0;
  T.chunks = 0;
  const auto flush = [&] {
    std::fill(T.first + used, T.first + kTable, ~0u);
    const hipError_t e = launch(T);
    used = 0;
    T.chunks = 0;
    return e;
  };
  for (int64_t i = 0; i < count; ++i) {
    const ma_tensor &t = tensors[i];
    if (t.p_type != p_type || t.g_type != g_type) continue;
    for (int64_t from = 0; from < t.n; from += kEntry) {
      const int64_t n = std::min(t.n - from, kEntry);
      const uint32_t chunks = (uint32_t)((n + kChunk - 1) / kChunk);   // at most 2^19
      if (T.chunks + chunks > kMostChunks)
        if (const hipError_t e = flush(); e != hipSuccess) return e;
      T.param[used] = static_cast<char *>(t.param) + from * size_of(p_type);
      T.grad[used] = static_cast<const char *>(t.grad) + from * size_of(g_type);
      T.n[used] = (uint32_t)n;
      T.block[used] = (uint32_t)((t.at + from) / kBlock);
      T.first[used] = T.chunks;
      T.chunks += chunks;
      if (++used == kTable)
        if (const hipError_t e = flush(); e != hipSuccess) return e;
    }
  }
  return used ? flush() : hipSuccess;
}

// launch.template operator()<P, G, COPY>(table) over the whole list.
template <class F> hipError_t each_type(int64_t count, const ma_tensor *tensors, bool copy, F launch) {
  hipError_t e = each_table(count, tensors, MA_TYPE_F32, MA_TYPE_F32, [&](const Table &T) { return launch(T, (float *)0, (float *)0, std::false_type()); });
  if (e == hipSuccess)
    e = each_table(count, tensors, MA_TYPE_F32, MA_TYPE_BF16, [&](const Table &T) { return launch(T, (float *)0, (__bf16 *)0, std::false_type()); });
  if (e == hipSuccess)
    e = each_table(count, tensors, MA_TYPE_BF16, MA_TYPE_F32, [&](const Table &T) {
      return copy ? launch(T, (__bf16 *)0, (float *)0, std::true_type()) : launch(T, (__bf16 *)0, (float *)0, std::false_type());
    });
  if (e == hipSuccess)
    e = each_table(count, tensors, MA_TYPE_BF16, MA_TYPE_BF16, [&](const Table &T) {
      return copy ? launch(T, (__bf16 *)0, (__bf16 *)0, std::true_type()) : launch(T, (__bf16 *)0, (__bf16 *)0, std::false_type());
    });
  return e;
}

StepArgs step_args(const ma_adamw_args &a) {
  const int64_t n = a.t_dev ? 1 : a.t;
  return {a.beta1, a.beta2, a.beta1 * (kUp / kM), a.beta2 * (kUp / (kR * kR)), (float)a.lr, (float)a.eps, (float)a.wd, correction1(a.beta1, n), correction2(a.beta2, n),
          a.t_dev, a.lr_dev, a.scale};
}

// launch(table) for every kNormTable entries, in chunks of CHUNK elements.
template <int CHUNK, class F> hipError_t each_norm_table(int64_t count, const ma_tensor *tensors, F launch) {
  NormTable T;
  int used = 0;
  T.chunks = 0;
  const auto flush = [&] {
    std::fill(T.first + used, T.first + kNormTable, ~0u);
    const hipError_t e = launch(T);
    used = 0;
    T.chunks = 0;
    return e;
  };
  for (int64_t i = 0; i < count; ++i) {
    const ma_tensor &t = tensors[i];
    for (int64_t from = 0; from < t.n; from += kEntry) {
      const int64_t n = std::min(t.n - from, kEntry);
      T.grad[used] = static_cast<const char *>(t.grad) + from * size_of(t.g_type);
      T.n[used] = (uint32_t)n | (t.g_type == MA_TYPE_BF16 ? kIsBf16 : 0u);
      T.first[used] = T.chunks;
      T.chunks += (uint32_t)((n + CHUNK - 1) / CHUNK);
      if (++used == kNormTable)
        if (const hipError_t e = flush(); e != hipSuccess) return e;
    }
  }
  return used ? flush() : hipSuccess;
}

// Whether one workgroup takes a whole list.
bool is_small(int64_t count, const ma_tensor *tensors) {
  int64_t chunks = 0, used = 0;
  for (int64_t i = 0; i < count && chunks <= kSmallChunks; ++i) {
    chunks += (tensors[i].n + kSmallChunk - 1) / kSmallChunk;
    used += tensors[i].n > 0;
  }
  return chunks > 0 && chunks <= kSmallChunks && used <= kNormTable;
}

}  // namespace

extern "C" {

size_t ma_grad_norm_workspace(int64_t count) {
  return count > 0 ? kNormGroups * sizeof(double) : 0;
}

int ma_grad_norm(int64_t count, const ma_tensor *tensors, double max_norm, float *out, int64_t *t, void *workspace,
                 size_t workspace_bytes, hipStream_t stream) {
  const char *who = "ma_grad_norm";
  return guarded(who, [&] {
    if (const int rc = check_list(who, count, tensors)) return rc;
    if (!(max_norm > 0.0)) return fail(MA_EINVAL, "%s: max_norm must be positive", who);
    if (!out || ((uintptr_t)out & 3u)) return fail(MA_EINVAL, "%s: null or misaligned out", who);
    if ((uintptr_t)t & 7u) return fail(MA_EINVAL, "%s: misaligned count", who);
    if (count && (!workspace || ((uintptr_t)workspace & 255u)))
      return fail(MA_EINVAL, "%s: the workspace must be 256-byte aligned", who);
    if (workspace_bytes < ma_grad_norm_workspace(count))
      return fail(MA_EINVAL, "%s: a workspace of %zu bytes, %zu are needed", who, workspace_bytes, ma_grad_norm_workspace(count));
    return on_device(who, stream, [&] {
      double *partial = static_cast<double *>(workspace);
      int parts = 0;   // sums in `partial` so far: a launch adds to them, and may add more of them
      if (is_small(count, tensors))
        return each_norm_table<kSmallChunk>(count, tensors, [&](const NormTable &T) {
          hipLaunchKernelGGL(norm_small_kernel, dim3(1), dim3(kSmallThreads), 0, stream, T, max_norm, out, t);
          return hipGetLastError();
        });
      const hipError_t e = each_norm_table<kNormChunk>(count, tensors, [&](const NormTable &T) {
        const int grid = (int)std::min<uint32_t>(T.chunks, kNormGroups);
        hipLaunchKernelGGL(norm_kernel, dim3(grid), dim3(kThreads), 0, stream, T, partial, parts);
        parts = std::max(parts, grid);
        return hipGetLastError();
      });
      if (e != hipSuccess) return e;
      hipLaunchKernelGGL(norm_finish_kernel, dim3(1), dim3(kThreads), 0, stream, partial, parts, max_norm, out, t);
      return hipGetLastError();
    });
  });
}

int ma_adamw_many_step(int64_t count, const ma_tensor *tensors, const ma_adamw_args *args, float *copy, float *m, float *v,
                       int64_t state_n, hipStream_t stream) {
  const char *who = "ma_adamw_many_step";
  return guarded(who, [&] {
    if (count > 0 && state_n > 0 && (!m || !v || (((uintptr_t)m | (uintptr_t)v) & 15u)))
      return fail(MA_EINVAL, "%s: null or misaligned moments", who);
    const uint64_t bytes = 4 * (uint64_t)state_n;
    if (const int rc = check_step(who, count, tensors, args, copy, state_n, {{copy, copy ? bytes : 0}, {m, bytes}, {v, bytes}}))
      return rc;
    if (!count || !state_n) return (int)MA_OK;
    const StepArgs a = step_args(*args);
    return on_device(who, stream, [&] {
      return each_type(count, tensors, copy != nullptr, [&](const Table &T, auto *p, auto *g, auto c) {
        using P = std::remove_pointer_t<decltype(p)>;
        using G = std::remove_pointer_t<decltype(g)>;
        hipLaunchKernelGGL((step_kernel<P, G, decltype(c)::value>), dim3(T.chunks), dim3(kThreads), 0, stream, T, a,
                           copy, m, v);
        return hipGetLastError();
      });
    });
  });
}

int ma_adamw8_many_step(int64_t count, const ma_tensor *tensors, const ma_adamw_args *args, float *copy, int8_t *cm, uint8_t *cv,
                        float *sm, float *sr, int64_t state_n, hipStream_t stream) {
  const char *who = "ma_adamw8_many_step";
  return guarded(who, [&] {
    if (count > 0 && state_n > 0 &&
        (!cm || !cv || !sm || !sr || (((uintptr_t)cm | (uintptr_t)cv) & 15u) || (((uintptr_t)sm | (uintptr_t)sr) & 3u)))
      return fail(MA_EINVAL, "%s: null or misaligned moments", who);
    const uint64_t codes = (uint64_t)state_n, scales = codes / kBlock * 4;
    if (const int rc = check_step(who, count, tensors, args, copy, state_n,
                                  {{copy, copy ? 4 * codes : 0}, {cm, codes}, {cv, codes}, {sm, scales}, {sr, scales}}))
      return rc;
    if (!count || !state_n) return (int)MA_OK;
    const StepArgs a = step_args(*args);
    return on_device(who, stream, [&] {
      return each_type(count, tensors, copy != nullptr, [&](const Table &T, auto *p, auto *g, auto c) {
        using P = std::remove_pointer_t<decltype(p)>;
        using G = std::remove_pointer_t<decltype(g)>;
        hipLaunchKernelGGL((step8_kernel<P, G, decltype(c)::value>), dim3(T.chunks), dim3(kThreads), 0, stream, T, a,
                           copy, cm, cv, sm, sr);
        return hipGetLastError();
      });
    });
  });
}

int ma_adamw8_many_values(int64_t state_n, const int8_t *cm, const uint8_t *cv, const float *sm, const float *sr, float *m, float *v,
                          hipStream_t stream) {
  const char *who = "ma_adamw8_many_values";
  return guarded(who, [&] {
    if (state_n < 0 || state_n % kBlock) return fail(MA_EINVAL, "%s: the states' size must be a multiple of %d", who, kBlock);
    if (state_n > kMost) return fail(MA_EUNSUPPORTED, "%s: states of more than 2^40 elements", who);
    if (!state_n) return (int)MA_OK;
    if (!cm || !cv || !sm || !sr || !m || !v || (((uintptr_t)cm | (uintptr_t)cv | (uintptr_t)m | (uintptr_t)v) & 15u) ||
        (((uintptr_t)sm | (uintptr_t)sr) & 3u))
      return fail(MA_EINVAL, "%s: null or misaligned pointer", who);
    return on_device(who, stream, [&] {
      constexpr int64_t most = int64_t(kMostChunks) * kChunk;
      for (int64_t at = 0; at < state_n; at += most) {
        const int64_t n = std::min(state_n - at, most), b = at / kBlock;
        hipLaunchKernelGGL(values8_kernel, dim3((unsigned)((n + kChunk - 1) / kChunk)), dim3(kThreads), 0, stream, cm + at, cv + at,
                           sm + b, sr + b, m + at, v + at, n / kBlock);
        if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
      }
      return hipSuccess;
    });
  });
}

}  // extern "C"
