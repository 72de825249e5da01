// Linear attention with a decay per head on the CUDA cores, in fp32
// arithmetic: for fp32 inputs, which the tensor cores cannot multiply without
// losing bits, and for bf16 inputs whose addresses or strides TMA cannot take.
// The scans and their formulas are in sa_linear_attention.h.
//
// One block of 256 threads walks one segment in chunks of 64 rows, with a, b,
// c and the weighted P of the chunk in shared memory and the state in
// registers (a da/16 x dc/16 tile per thread) and, for the products that read
// it, in shared memory.  Every product is a register-tiled one: 16 x 16
// threads, operands read as 16-byte vectors.
//
// A chunk costs 64 da 64 (P) + half of 64 64 dc (P c, the other half is zero
// and skipped) + 2 * 64 da dc multiply-adds.  Tiles of 64 rows: P's cost grows
// with the tile, the number of passes over the state with its inverse, and at
// da = dc = 128 the five arrays fill 183 KB.
// What bounds it: latency.  The eight warps of an SM's one block wait for the
// chunk's operands, which are loaded element by element between two barriers
// with nothing in flight meanwhile, and for shared memory: 148 histories of
// 2048 rows at da = dc = 64 keep the fp32 pipe busy for 35 % of its cycles,
// the issue slots for 48 %, DRAM for 8 %.  Measured: 16 x 100K rows, two heads
// of 64, forward: 6.9-8.6 ms; 48 ragged histories of up to 4099 rows, eight
// heads of 128: 2.8-3.3 ms; backward of 16 x 10K rows, eight heads of 128:
// 14-16 ms.
#include <cuda_bf16.h>

#include "sa.h"
#include "sa_internal.h"
#include "sa_linear_attention.h"
#include "sa_operators.cuh"

namespace sa {
namespace {

constexpr int kThreads = 256, kRows = 64, kPadP = kRows + 4;

template <int DA, int DC>
struct SimtPlan {
  static constexpr int kPad = DA + 4;               // conflict-free 16-byte reads of 8 rows
  static constexpr int kA = 0, kB = kA + kRows * kPad, kC = kB + kRows * kPad;
  static constexpr int kP = kC + kRows * DC, kS = kP + kRows * kPadP;
  static constexpr int kPow = kS + DA * DC;         // l^0 .. l^64, then l^64's rounding error
  static constexpr int kFloats = kPow + kRows + 4;
  static constexpr int kSmem = kFloats * 4;
  static_assert(kSmem <= 232448, "shared memory budget");
};

__device__ __forceinline__ float load_f(const float* p) { return *p; }
__device__ __forceinline__ float load_f(const uint16_t* p) {
  return __uint_as_float(static_cast<uint32_t>(*p) << 16);
}
__device__ __forceinline__ void store4(float* p, float4 v) { *reinterpret_cast<float4*>(p) = v; }
__device__ __forceinline__ void store4(uint16_t* p, float4 v) {
  *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
}
__device__ __forceinline__ float4 ld4(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ void axpy(float a, const float4& x, float4& y) {
  y.x = fmaf(a, x.x, y.x);
  y.y = fmaf(a, x.y, y.y);
  y.z = fmaf(a, x.z, y.z);
  y.w = fmaf(a, x.w, y.w);
}

// kRows rows of one operand into shared memory, zeros behind row n.
template <class T, int D, int PAD>
__device__ __forceinline__ void load_rows(float* dst, const ScanInput& in, int64_t row0, int head,
                                          int n) {
  const T* p = static_cast<const T*>(in.p) + row0 * in.row + static_cast<int64_t>(head) * in.head;
#pragma unroll 8
  for (int e = threadIdx.x; e < kRows * D; e += kThreads) {
    const int r = e / D, c = e % D;
    dst[r * PAD + c] = r < n ? load_f(p + r * in.row + c) : 0.f;
  }
}

template <class T, int DA, int DC, bool STATE>
__global__ void __launch_bounds__(kThreads, 1) scan_simt_kernel(const __grid_constant__ ScanArgs t) {
  using Pl = SimtPlan<DA, DC>;
  constexpr int RS = DA / 16, CS = DC / 64;  // state rows, groups of four columns per thread
  extern __shared__ __align__(16) float smem_f[];
  __shared__ uint32_t check_flags;
  float *sa = smem_f + Pl::kA, *sb = smem_f + Pl::kB, *sc = smem_f + Pl::kC, *sp = smem_f + Pl::kP,
        *ss = smem_f + Pl::kS, *pw = smem_f + Pl::kPow;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  if (t.check && blockIdx.x == 0) check_inputs(t.s, &check_flags);
  for (int64_t x = blockIdx.x; x < t.items; x += gridDim.x) {
    ScanItem it;
    if (!item_of(t, x, threadIdx.x & 31, STATE, it)) continue;
    const ScanPass& p = t.p[it.pass];
    const bool rev = p.reverse != 0;
    __syncthreads();  // the item before has been read out
    const double g = static_cast<double>(usable_decay(t.s.log_decay[it.head]));
    if (threadIdx.x <= kRows) {
      const double w = exp(g * threadIdx.x);
      pw[threadIdx.x] = static_cast<float>(w);
      if (threadIdx.x == kRows) pw[kRows + 1] = static_cast<float>(w - static_cast<float>(w));
    }
    float4 S[RS][CS];
    {
      const bool seg = !STATE && it.from >= 0;
      const float* src = STATE ? nullptr : seg ? p.bound : p.ends;
      const float m = seg ? 1.f : p.ends_mul;
      const int64_t o = (seg ? it.from : it.state) * (DA * DC);
#pragma unroll
      for (int r = 0; r < RS; ++r)
#pragma unroll
        for (int c = 0; c < CS; ++c) {
          const int row = ty * RS + r, col = c * 64 + tx * 4;
          if (src == nullptr) {
            S[r][c] = make_float4(0.f, 0.f, 0.f, 0.f);
          } else if (p.transposed) {
            const float* q = src + o + col * DA + row;
            S[r][c] = make_float4(m * q[0], m * q[DA], m * q[2 * DA], m * q[3 * DA]);
          } else {
            const float4 v = ld4(src + o + row * DC + col);
            S[r][c] = make_float4(m * v.x, m * v.y, m * v.z, m * v.w);
          }
        }
    }
    const int64_t chunks = (it.hi - it.lo + kRows - 1) / kRows;
    for (int64_t k = 0; k < chunks; ++k) {
      const int64_t r0 = it.lo + kRows * (rev ? chunks - 1 - k : k);
      const int L = static_cast<int>(it.hi - r0 < kRows ? it.hi - r0 : kRows);
      // A reverse scan's first rows of a user take the start state undecayed.
      const int skip = rev && it.first && k == 0 ? 1 : 0;
      __syncthreads();
      if (!STATE) {
        load_rows<T, DA, Pl::kPad>(sa, p.a, r0, it.head, L);
#pragma unroll
        for (int r = 0; r < RS; ++r)
#pragma unroll
          for (int c = 0; c < CS; ++c)
            *reinterpret_cast<float4*>(ss + (ty * RS + r) * DC + c * 64 + tx * 4) = S[r][c];
      }
      load_rows<T, DA, Pl::kPad>(sb, p.b, r0, it.head, L);
      load_rows<T, DC, DC>(sc, p.c, r0, it.head, L);
      __syncthreads();
      if (!STATE) {
        // P: rows 4 ty + r, columns tx + 16 c.
        float acc[4][4] = {};
#pragma unroll 4
        for (int d = 0; d < DA; d += 4) {
          float4 u[4], v[4];
#pragma unroll
          for (int r = 0; r < 4; ++r) u[r] = ld4(sa + (ty * 4 + r) * Pl::kPad + d);
#pragma unroll
          for (int c = 0; c < 4; ++c) v[c] = ld4(sb + (tx + 16 * c) * Pl::kPad + d);
#pragma unroll
          for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int c = 0; c < 4; ++c)
              acc[r][c] = fmaf(u[r].w, v[c].w, fmaf(u[r].z, v[c].z,
                               fmaf(u[r].y, v[c].y, fmaf(u[r].x, v[c].x, acc[r][c]))));
        }
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const int i = ty * 4 + r, j = tx + 16 * c, dist = rev ? j - i : i - j;
            sp[i * kPadP + j] = dist >= 0 ? acc[r][c] * pw[dist] : 0.f;
          }
        // a S, weighted, while P is written.
        float4 o[4][CS];
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
          for (int c = 0; c < CS; ++c) o[r][c] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
        for (int d = 0; d < DA; d += 4) {
          float4 u[4];
#pragma unroll
          for (int r = 0; r < 4; ++r) u[r] = ld4(sa + (ty * 4 + r) * Pl::kPad + d);
#pragma unroll
          for (int e = 0; e < 4; ++e)
#pragma unroll
            for (int c = 0; c < CS; ++c) {
              const float4 v = ld4(ss + (d + e) * DC + c * 64 + tx * 4);
#pragma unroll
              for (int r = 0; r < 4; ++r) axpy((&u[r].x)[e], v, o[r][c]);
            }
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int i = ty * 4 + r;
          const float w = i < L ? pw[rev ? L - i - skip : i + 1] : 0.f;
#pragma unroll
          for (int c = 0; c < CS; ++c) {
            o[r][c].x *= w;
            o[r][c].y *= w;
            o[r][c].z *= w;
            o[r][c].w *= w;
          }
        }
        __syncthreads();
        // P c: the row group's own four columns of P one by one (a row that
        // the scan has not reached must not be multiplied, whatever c holds
        // there), then the groups it covers whole.
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
          for (int c = 0; c < CS; ++c) {
            const float4 v = ld4(sc + (ty * 4 + e) * DC + c * 64 + tx * 4);
#pragma unroll
            for (int r = 0; r < 4; ++r)
              if (rev ? e >= r : e <= r) axpy(sp[(ty * 4 + r) * kPadP + ty * 4 + e], v, o[r][c]);
          }
        const int j0 = rev ? ty * 4 + 4 : 0, j1 = rev ? kRows : ty * 4;
        for (int j = j0; j < j1; j += 4) {
          float4 u[4];
#pragma unroll
          for (int r = 0; r < 4; ++r) u[r] = ld4(sp + (ty * 4 + r) * kPadP + j);
#pragma unroll
          for (int e = 0; e < 4; ++e)
#pragma unroll
            for (int c = 0; c < CS; ++c) {
              const float4 v = ld4(sc + (j + e) * DC + c * 64 + tx * 4);
#pragma unroll
              for (int r = 0; r < 4; ++r) axpy((&u[r].x)[e], v, o[r][c]);
            }
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          if (ty * 4 + r >= L) continue;
          T* q = static_cast<T*>(p.out) + ((r0 + ty * 4 + r) * t.s.heads + it.head) * DC + tx * 4;
#pragma unroll
          for (int c = 0; c < CS; ++c)
            store4(q + c * 64, make_float4(o[r][c].x * p.out_mul, o[r][c].y * p.out_mul,
                                           o[r][c].z * p.out_mul, o[r][c].w * p.out_mul));
        }
      }
      // The state: the chunk's sum from zero, then one addition to S.
      float4 D[RS][CS];
#pragma unroll
      for (int r = 0; r < RS; ++r)
#pragma unroll
        for (int c = 0; c < CS; ++c) D[r][c] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
      for (int j = 0; j < L; ++j) {
        const float w = pw[rev ? j : L - 1 - j];
        float4 v[CS], u[RS / 4];
#pragma unroll
        for (int c = 0; c < CS; ++c) v[c] = ld4(sc + j * DC + c * 64 + tx * 4);
#pragma unroll
        for (int r = 0; r < RS / 4; ++r) u[r] = ld4(sb + j * Pl::kPad + ty * RS + r * 4);
#pragma unroll
        for (int r = 0; r < RS; ++r)
#pragma unroll
          for (int c = 0; c < CS; ++c) axpy(w * (&u[r / 4].x)[r % 4], v[c], D[r][c]);
      }
      const float f = pw[L - skip], fl = L - skip == kRows ? pw[kRows + 1] : 0.f;
#pragma unroll
      for (int r = 0; r < RS; ++r)
#pragma unroll
        for (int c = 0; c < CS; ++c) {
          axpy(fl, S[r][c], D[r][c]);
          axpy(f, S[r][c], D[r][c]);
          S[r][c] = D[r][c];
        }
    }
    // The state behind the last row.
    float* dst = nullptr;
    float m = 1.f;
    if (STATE) {
      dst = p.bound + it.to * (DA * DC);
    } else if (it.last && p.fin != nullptr) {
      dst = p.fin + it.state * (DA * DC);
      m = p.fin_mul * (rev && chunks > 0 ? pw[1] : 1.f);
    }
    if (dst == nullptr) continue;
#pragma unroll
    for (int r = 0; r < RS; ++r)
#pragma unroll
      for (int c = 0; c < CS; ++c)
        store4(dst + (ty * RS + r) * DC + c * 64 + tx * 4,
               make_float4(m * S[r][c].x, m * S[r][c].y, m * S[r][c].z, m * S[r][c].w));
  }
}

template <class T, int DA, int DC, bool STATE>
cudaError_t launch(const ScanArgs& t, cudaStream_t st) {
  constexpr int smem = SimtPlan<DA, DC>::kSmem;
  static std::atomic<uint64_t> allowed{0};
  const cudaError_t err = allow_smem(scan_simt_kernel<T, DA, DC, STATE>, smem, allowed);
  if (err != cudaSuccess) return err;
  const int64_t most = int64_t{1} << 30;
  scan_simt_kernel<T, DA, DC, STATE>
      <<<static_cast<unsigned>(t.items < most ? t.items : most), kThreads, smem, st>>>(t);
  return cudaGetLastError();
}

template <class T, bool STATE>
cudaError_t launch_any(const ScanArgs& t, cudaStream_t st) {
  if (t.p[0].da == 64)
    return t.p[0].dc == 64 ? launch<T, 64, 64, STATE>(t, st) : launch<T, 64, 128, STATE>(t, st);
  return t.p[0].dc == 64 ? launch<T, 128, 64, STATE>(t, st) : launch<T, 128, 128, STATE>(t, st);
}

}  // namespace

cudaError_t launch_scan_simt(const ScanArgs& t, bool bf16, bool states_only, cudaStream_t st) {
  if (states_only) return bf16 ? launch_any<uint16_t, true>(t, st) : launch_any<float, true>(t, st);
  return bf16 ? launch_any<uint16_t, false>(t, st) : launch_any<float, false>(t, st);
}

}  // namespace sa
