// The global L2 norm of many gradient tensors, and clipping by it:
//
//   norm = sqrt(sum over all tensors and elements of g^2)
//   out  = g * min(1, max_norm / (norm + 1e-6))
//
// Two kernels, whatever the number of tensors (up to kMost per launch): the
// tensors are one list of chunks, split evenly over the blocks, and the
// table of addresses, sizes and types travels in the kernels' parameters, so
// that nothing is kept between calls and a captured graph holds its own
// copy.  Pass 1 writes each block's sum of squares; pass 2 adds those sums
// in a fixed order in every block (bitwise reproducible, no atomics), and
// scales.  In place with norm <= max_norm it has nothing to do and returns.
//
// Sums: eight squares in fp32, then fp64.  Groups whose fp32 sum leaves
// [2^-80, 2^120] are summed again in fp64, so the norm neither overflows nor
// loses small gradients over the whole range of fp32.
//
// What bounds it: memory, one read for the norm, one read and one write for
// the scaling.  Pass 2 walks each block's range backwards, so that it begins
// with what pass 1 has left in L2; its stores are marked for early eviction.
// Measured: 354 M bf16 values in 217 tensors: 387 us (130 + 228 us of device
// time, 5.4 and 6.2 TB/s); 19 tensors of 0.5 M fp32 values: 5.4 us in a graph.
#include <cuda_bf16.h>
#include <math.h>

#include <algorithm>
#include <new>

#include "sa.h"
#include "sa_internal.h"
#include "sa_operators.cuh"

namespace sa {
namespace {

constexpr int kClipThreads = 256;
constexpr int64_t kChunk = 2048;   // elements; whole 16-byte units of either type
// Table sizes: the parameters are copied at every launch, so a short list
// gets a small table (48 entries: 1.5 KB, 256: 8 KB, 896: 28 KB).
constexpr int kFew = 48, kSome = 256, kMost = 896;
constexpr int kMaxClipBlocks = 8 * 148;

struct GradEntry {
  const void* src;
  void* dst;
  int64_t n;        // elements, the sign bit set for bf16
  int64_t chunk0;   // chunks of the entries before it
};

template <int MAX>
struct GradTable {
  GradEntry e[MAX];
  int count;
  int64_t chunks;
};
static_assert(sizeof(GradTable<kMost>) < 30000, "kernel parameter space");

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

__device__ __forceinline__ double squares(const float (&v)[8]) {
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) s = fmaf(v[i], v[i], s);
  if (s >= 0x1p-80f && s <= 0x1p120f) return s;
  double t = 0.0;
#pragma unroll
  for (int i = 0; i < 8; ++i) t = fma(static_cast<double>(v[i]), static_cast<double>(v[i]), t);
  return t;
}

// Sum of `v` over the block in a fixed order (all threads get it).
__device__ __forceinline__ double block_sum(double v, double* buf) {
#pragma unroll
  for (int m = 16; m > 0; m >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, m);
  if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = v;
  __syncthreads();
  double s = 0.0;
#pragma unroll
  for (int w = 0; w < kClipThreads / 32; ++w) s += buf[w];
  return s;
}

template <int MAX>
__device__ __forceinline__ int entry_of(const GradTable<MAX>& t, int64_t chunk) {
  int lo = 0, hi = t.count - 1;  // largest i with chunk0 <= chunk
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (t.e[mid].chunk0 <= chunk) lo = mid; else hi = mid - 1;
  }
  return lo;
}

template <int MAX>
__global__ void __launch_bounds__(kClipThreads)
    grad_squares_kernel(const __grid_constant__ GradTable<MAX> t, double* part) {
  __shared__ double buf[kClipThreads / 32];
  const int64_t c0 = t.chunks * blockIdx.x / gridDim.x;
  const int64_t c1 = t.chunks * (blockIdx.x + 1) / gridDim.x;
  double sum = 0.0;
  int i = c0 < c1 ? entry_of(t, c0) : 0;
  for (int64_t c = c0; c < c1; ++i) {
    const GradEntry& g = t.e[i];
    const int64_t n = g.n & INT64_MAX;
    const int64_t last = (n + kChunk - 1) / kChunk + g.chunk0;  // one past the entry's chunks
    const int64_t lo = (c - g.chunk0) * kChunk;
    const int64_t hi = c1 < last ? (c1 - g.chunk0) * kChunk : n;
    c = c1 < last ? c1 : last;
    const bool bf = g.n < 0, vec = (reinterpret_cast<uintptr_t>(g.src) & 15u) == 0;
    int64_t done = lo;
    if (vec) {
      const int64_t units = (hi - lo) / 8;
      done = lo + units * 8;
      if (bf) {
        const uint4* p = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(g.src) + lo);
#pragma unroll 4
        for (int64_t u = threadIdx.x; u < units; u += kClipThreads) {
          const uint4 w = __ldg(p + u);
          const float v[8] = {bf_lo(w.x), bf_hi(w.x), bf_lo(w.y), bf_hi(w.y),
                              bf_lo(w.z), bf_hi(w.z), bf_lo(w.w), bf_hi(w.w)};
          sum += squares(v);
        }
      } else {
        const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(g.src) + lo);
#pragma unroll 4
        for (int64_t u = threadIdx.x; u < units; u += kClipThreads) {
          const float4 w0 = __ldg(p + 2 * u), w1 = __ldg(p + 2 * u + 1);
          const float v[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
          sum += squares(v);
        }
      }
    }
    for (int64_t e = done + threadIdx.x; e < hi; e += kClipThreads) {
      const double v = bf ? __uint_as_float(
                                static_cast<uint32_t>(static_cast<const uint16_t*>(g.src)[e]) << 16)
                          : static_cast<const float*>(g.src)[e];
      sum = fma(v, v, sum);
    }
  }
  sum = block_sum(sum, buf);
  if (threadIdx.x == 0) part[blockIdx.x] = sum;
}

__device__ __forceinline__ double total_norm(const double* part, int parts, double* buf) {
  double s = 0.0;
  for (int i = threadIdx.x; i < parts; i += kClipThreads) s += part[i];
  return sqrt(block_sum(s, buf));
}

__global__ void __launch_bounds__(kClipThreads)
    grad_norm_kernel(const double* part, int parts, float* norm) {
  __shared__ double buf[kClipThreads / 32];
  grid_dependency_wait();
  const double n = total_norm(part, parts, buf);
  if (threadIdx.x == 0) *norm = static_cast<float>(n);
}

__device__ __forceinline__ uint32_t scale2(uint32_t w, float m) {
  return pack_bf16x2(bf_lo(w) * m, bf_hi(w) * m);
}

template <int MAX>
__global__ void __launch_bounds__(kClipThreads)
    grad_scale_kernel(const __grid_constant__ GradTable<MAX> t, const double* part, int parts,
                      double max_norm, float* norm) {
  __shared__ double buf[kClipThreads / 32];
  grid_dependency_wait();
  const double n = total_norm(part, parts, buf);
  const float told = static_cast<float>(n);
  if (norm != nullptr && blockIdx.x == 0 && threadIdx.x == 0) *norm = told;
  // A norm that is not finite in fp32, as the caller sees it, leaves the
  // values as they are.
  const double factor = max_norm / (n + 1e-6);
  const float m = isfinite(told) && factor < 1.0 ? static_cast<float>(factor) : 1.f;
  // A factor below the smallest normal fp32 has fewer bits there, or none:
  // products are then taken in 64 bits, element by element (a call on 354 M
  // bf16 values: 852 us instead of 379).
  const bool fine = isfinite(told) && factor < 0x1p-126 && factor != 0.0;
  const int64_t c0 = t.chunks * blockIdx.x / gridDim.x;
  const int64_t c1 = t.chunks * (blockIdx.x + 1) / gridDim.x;
  if (c0 >= c1) return;
  int i = entry_of(t, c1 - 1);
  for (int64_t c = c1; c > c0; --i) {
    const GradEntry& g = t.e[i];
    const int64_t size = g.n & INT64_MAX;
    const int64_t first = c0 > g.chunk0 ? c0 : g.chunk0;
    const int64_t lo = (first - g.chunk0) * kChunk;
    const int64_t end = (c - g.chunk0) * kChunk, hi = end < size ? end : size;
    c = first;
    if (m == 1.f && g.dst == g.src) continue;
    const bool bf = g.n < 0;
    if (fine) {
      for (int64_t e = lo + threadIdx.x; e < hi; e += kClipThreads) {
        if (bf)
          static_cast<__nv_bfloat16*>(g.dst)[e] = __float2bfloat16_rn(static_cast<float>(
              static_cast<double>(__bfloat162float(static_cast<const __nv_bfloat16*>(g.src)[e])) * factor));
        else
          static_cast<float*>(g.dst)[e] =
              static_cast<float>(static_cast<double>(static_cast<const float*>(g.src)[e]) * factor);
      }
      continue;
    }
    const bool vec = ((reinterpret_cast<uintptr_t>(g.src) | reinterpret_cast<uintptr_t>(g.dst)) & 15u) == 0;
    const int64_t units = vec ? (hi - lo) / (bf ? 8 : 4) : 0;
    const int64_t done = lo + units * (bf ? 8 : 4);
    for (int64_t e = done + threadIdx.x; e < hi; e += kClipThreads) {
      if (bf)
        static_cast<__nv_bfloat16*>(g.dst)[e] =
            m == 1.f ? static_cast<const __nv_bfloat16*>(g.src)[e]
                     : __float2bfloat16_rn(__bfloat162float(static_cast<const __nv_bfloat16*>(g.src)[e]) * m);
      else
        static_cast<float*>(g.dst)[e] = static_cast<const float*>(g.src)[e] * m;
    }
    const uint4* p = reinterpret_cast<const uint4*>(static_cast<const char*>(g.src) + lo * (bf ? 2 : 4));
    uint4* o = reinterpret_cast<uint4*>(static_cast<char*>(g.dst) + lo * (bf ? 2 : 4));
#pragma unroll 4
    for (int64_t u = threadIdx.x; u < units; u += kClipThreads) {
      const int64_t r = units - 1 - u;
      uint4 w = p[r];
      if (bf) {
        w = make_uint4(scale2(w.x, m), scale2(w.y, m), scale2(w.z, m), scale2(w.w, m));
      } else {
        w = make_uint4(__float_as_uint(__uint_as_float(w.x) * m), __float_as_uint(__uint_as_float(w.y) * m),
                       __float_as_uint(__uint_as_float(w.z) * m), __float_as_uint(__uint_as_float(w.w) * m));
      }
      __stcs(o + r, w);
    }
  }
}

bool al(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) % n) == 0; }

struct Span {
  uintptr_t lo, hi;
  bool written;
};

// True if no written range meets another range (a tensor scaled in place is
// one written range).  False too when the host has no memory for the list.
bool ranges_apart(const void* const* src, void* const* dst, const int64_t* numel,
                  const sa_dtype* dtypes, int64_t tensors) {
  Span* s = new (std::nothrow) Span[2 * tensors];
  if (s == nullptr) return false;
  int64_t n = 0;
  for (int64_t i = 0; i < tensors; ++i) {
    const uintptr_t bytes = static_cast<uintptr_t>(numel[i]) * (dtypes[i] == SA_BF16 ? 2 : 4);
    if (bytes == 0) continue;
    const uintptr_t a = reinterpret_cast<uintptr_t>(src[i]);
    const uintptr_t b = dst != nullptr ? reinterpret_cast<uintptr_t>(dst[i]) : a;
    if (b != a) s[n++] = {a, a + bytes, false};
    s[n++] = {b, b + bytes, true};
  }
  std::sort(s, s + n, [](const Span& x, const Span& y) { return x.lo < y.lo; });
  uintptr_t any = 0, written = 0;
  bool ok = true;
  for (int64_t i = 0; i < n && ok; ++i) {
    ok = s[i].lo >= (s[i].written ? any : written);
    if (s[i].hi > any) any = s[i].hi;
    if (s[i].written && s[i].hi > written) written = s[i].hi;
  }
  delete[] s;
  return ok;
}

struct Group {
  int64_t first, last;  // tensors
  int blocks;
};

// The next launch's tensors from `first`, filled into `t`.
template <int MAX>
Group fill(GradTable<MAX>& t, const void* const* src, void* const* dst, const int64_t* numel,
           const sa_dtype* dtypes, int64_t tensors, int64_t first) {
  t.count = 0;
  t.chunks = 0;
  int64_t i = first;
  for (; i < tensors && t.count < MAX; ++i) {
    if (numel[i] == 0) continue;
    GradEntry& e = t.e[t.count++];
    e.src = src[i];
    e.dst = dst != nullptr ? dst[i] : const_cast<void*>(src[i]);
    e.n = numel[i] | (dtypes[i] == SA_BF16 ? INT64_MIN : 0);
    e.chunk0 = t.chunks;
    t.chunks += (numel[i] + kChunk - 1) / kChunk;
  }
  const int blocks = static_cast<int>(t.chunks < kMaxClipBlocks ? t.chunks : kMaxClipBlocks);
  return {first, i, blocks};
}

template <class... P, class... A>
cudaError_t launch_after(void (*kernel)(P...), int blocks, cudaStream_t st, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks));
  cfg.blockDim = dim3(kClipThreads);
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <int MAX>
sa_status run_clip(const void* const* src, void* const* dst, const int64_t* numel,
                   const sa_dtype* dtypes, int64_t tensors, bool scale, double max_norm,
                   float* norm, double* part, cudaStream_t st) {
  GradTable<MAX>* t = new (std::nothrow) GradTable<MAX>;
  if (t == nullptr) return SA_ERR_CUDA;
  cudaError_t err = cudaSuccess;
  int parts = 0;
  bool wrote = false;
  for (int64_t i = 0; i < tensors && err == cudaSuccess;) {
    const Group g = fill(*t, src, dst, numel, dtypes, tensors, i);
    i = g.last;
    if (g.blocks == 0) continue;
    grad_squares_kernel<MAX><<<g.blocks, kClipThreads, 0, st>>>(*t, part + parts);
    err = cudaGetLastError();
    parts += g.blocks;
  }
  // Later launches of pass 2 need not wait for earlier ones: only the first
  // follows pass 1, and each waits for the launch before it to complete.
  for (int64_t i = 0; scale && i < tensors && err == cudaSuccess;) {
    const Group g = fill(*t, src, dst, numel, dtypes, tensors, i);
    i = g.last;
    if (g.blocks == 0) continue;
    err = launch_after(grad_scale_kernel<MAX>, g.blocks, st, *t, static_cast<const double*>(part),
                       parts, max_norm, wrote ? static_cast<float*>(nullptr) : norm);
    wrote = true;
  }
  if (!wrote && err == cudaSuccess)
    err = launch_after(grad_norm_kernel, 1, st, static_cast<const double*>(part), parts, norm);
  delete t;
  return err == cudaSuccess ? SA_OK : SA_ERR_CUDA;
}

sa_status clip(const void* const* src, void* const* dst, const int64_t* numel,
               const sa_dtype* dtypes, int64_t tensors, bool scale, double max_norm, float* norm,
               void* workspace, size_t workspace_bytes, void* stream) {
  if (tensors < 0 || tensors > (int64_t{1} << 20) || norm == nullptr || !al(norm, 4) ||
      workspace == nullptr || !al(workspace, 8))
    return SA_ERR_INVALID_ARG;
  if (tensors > 0 && (src == nullptr || numel == nullptr || dtypes == nullptr))
    return SA_ERR_INVALID_ARG;
  for (int64_t i = 0; i < tensors; ++i) {
    if (dtypes[i] != SA_BF16 && dtypes[i] != SA_FP32) return SA_ERR_INVALID_ARG;
    const size_t e = dtypes[i] == SA_BF16 ? 2 : 4;
    if (numel[i] < 0 || numel[i] >= (int64_t{1} << 44)) return SA_ERR_INVALID_ARG;
    if (numel[i] > 0 && (src[i] == nullptr || !al(src[i], e) ||
                         (dst != nullptr && (dst[i] == nullptr || !al(dst[i], e)))))
      return SA_ERR_INVALID_ARG;
  }
  if (scale && !ranges_apart(src, dst, numel, dtypes, tensors)) return SA_ERR_INVALID_ARG;
  int dev = 0, major = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess)
    return SA_ERR_CUDA;
  if (major != 10) return SA_ERR_UNSUPPORTED;
  if (workspace_bytes < sa_workspace_bytes_grad_norm(tensors)) return SA_ERR_WORKSPACE;
  double* part = static_cast<double*>(workspace);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  auto run = tensors <= kFew ? run_clip<kFew> : tensors <= kSome ? run_clip<kSome> : run_clip<kMost>;
  return run(src, dst, numel, dtypes, tensors, scale, max_norm, norm, part, st);
}

}  // namespace
}  // namespace sa

extern "C" {

size_t sa_workspace_bytes_grad_norm(int64_t tensors) {
  if (tensors < 0) return 0;
  const int64_t launches = tensors <= sa::kMost ? 1 : (tensors + sa::kMost - 1) / sa::kMost;
  return static_cast<size_t>(launches) * sa::kMaxClipBlocks * sizeof(double);
}

sa_status sa_grad_norm(const void* const* grads, const int64_t* numel, const sa_dtype* dtypes,
                       int64_t tensors, float* norm, void* workspace, size_t workspace_bytes,
                       void* stream) {
  return sa::clip(grads, nullptr, numel, dtypes, tensors, false, 1.0, norm, workspace,
                  workspace_bytes, stream);
}

sa_status sa_clip_grad_norm(void* const* grads, void* const* out, const int64_t* numel,
                            const sa_dtype* dtypes, int64_t tensors, float max_norm, float* norm,
                            void* workspace, size_t workspace_bytes, void* stream) {
  if (!(max_norm >= 0.f) || !(max_norm < INFINITY)) return SA_ERR_INVALID_ARG;
  return sa::clip(const_cast<const void* const*>(grads), out, numel, dtypes, tensors, true,
                  max_norm, norm, workspace, workspace_bytes, stream);
}

}  // extern "C"
