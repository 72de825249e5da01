// The norms before and after a block, fused with the block's gate and
// residual scale (the residual stream around a mixing block such as linear
// attention or the FFN), forward and backward:
//
//   n = norm(y; g1, b1)              norm after the block (n = y without g1)
//   r = x + rs * act(z) * n          residual scale rs, gate act(z)
//   u = norm(r; g2, b2)              norm before the next block
//
// norm(x; g, b) = g (x - mean) rstd + b (layer) or g x rstd + b (root mean
// square, mean = 0), rstd = 1 / sqrt(var + eps).  Backward, from r, y, z and
// the upstream gradients dr, du (x^ the normalised value):
//
//   h   = du g2;   dx = dr + rstd_r (h - mean(h) - r^ mean(h r^))
//   dn  = dx rs act(z);   dz = dx rs n act'(z);   drs = sum dx act(z) n
//   p   = dn g1;   dy = rstd_y (p - mean(p) - y^ mean(p y^))
//   dg2 = sum du r^, db2 = sum du, dg1 = sum dn y^, db1 = sum dn   (over rows)
//
// (mean(h) and mean(p) only in the layer form).  All arithmetic is fp32; an
// output is rounded once, when it is stored, and u is taken from the
// unrounded r.  Statistics are two-pass (mean, then squared deviations): the
// row is in registers, so the second pass costs no memory access and large
// means lose nothing.
//
// What bounds it: memory; each input is read once and each output written
// once.  A row is held by R threads, 8 columns (one or two 16-byte loads)
// per thread and operand, so that gains, biases and the backward's five
// column sums stay in registers over the rows of a persistent block.  R is
// the power of two that covers d: up to 32, several rows share a warp or
// block and reduce by shuffles; above, one block holds one row and reduces
// through shared memory with one barrier per reduction.  Rows whose width or
// address does not allow 16-byte accesses use the same code with
// single-element loads at columns R apart, so that neighbouring threads read
// neighbouring elements.
// Measured: forward over 200K x 1024 bf16 with both norms, SiLU gate and
// scale: 390-419 us (5.0 TB/s; 68 % of the issue slots); backward over 400K x
// 128, fp32 residual: 242-261 us (4.4 TB/s; 50 % of the issue slots, with
// three blocks of 128 threads per SM, by registers).
// Far from memory's time: rows without 16-byte accesses, which are bound by
// instructions (backward over 100K x 300 bf16: 626 us, 65 % of the issue slots,
// where its bytes take 73), and the backward above 4096 columns, whose two
// groups per thread do not fit its registers (20K x 8192: 1.4 ms, where its
// bytes take 0.40; a launch over 5000 rows moves 2.2 GB to and from local
// memory, beside 0.7 GB of DRAM).  The column sums add up to some hundreds of
// rows per thread in fp32, then the blocks' sums in fp64.
#include <cuda_bf16.h>

#include <atomic>

#include "sa.h"
#include "sa_internal.h"
#include "sa_operators.cuh"

namespace sa {
namespace {

constexpr int kMaxNormWidth = 8192;
constexpr int kMaxDevices = 64;
constexpr int kCols = 8;         // columns per thread and group
constexpr int kPairs = kCols / 2;  // as pairs, for packed fp32 arithmetic

struct NormArgs {
  const void *x, *y, *z;        // forward: residual, block, gate; backward: r, block, gate
  int64_t ldx, ldy, ldz;
  const float *g1, *b1, *rs, *g2, *b2;
  const void *dr, *du;          // backward only
  int64_t lddr, lddu;
  void *o1, *o2, *o3;           // forward: r, u; backward: dx, dy, dz
  float* part;                  // backward: [grid][5][d] column sums
  int64_t rows;
  int d, layer, gate_kind, sums;
  float eps, inv_d;
};

// Rows in flight.  A thread copies its 8 neighbouring columns of every operand
// of its next D rows into slots of shared memory that it alone reads (16-byte
// asynchronous copies, no barrier), so that the bytes in flight, which the
// bandwidth follows here, do not cost registers: 36 KB per SM in registers
// gave 304 us for the backward over 400K x 128, see the kernels.  Rows that
// do not allow 16-byte accesses go through registers, one row ahead.
template <class T>
__host__ __device__ constexpr int units() { return kCols * static_cast<int>(sizeof(T)) / 16; }

__device__ __forceinline__ void copy_async(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(uint16_t v) { return __uint_as_float(static_cast<uint32_t>(v) << 16); }

// Two bf16 as a pair of fp32.
__device__ __forceinline__ uint64_t widen(uint32_t w) {
  return f2_pack(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
__device__ __forceinline__ uint64_t both(float v) { return f2_pack(v, v); }
__device__ __forceinline__ float f2_sum(uint64_t v) {
  float a, b;
  f2_unpack(v, a, b);
  return a + b;
}

template <class T, int R, int NV, int TT, bool VEC>
struct Operand {
  T v[VEC ? 1 : NV][VEC ? 1 : kCols];  // the register path's next row
  // Starts the copy of a row into the slots at `slot` (stride: 16 bytes per
  // thread of the block), or loads it.
  __device__ __forceinline__ void fetch(const void* base, int64_t offset, uint32_t slot, int l, int d) {
    const T* row = static_cast<const T*>(base) + offset;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if constexpr (VEC) {
        const int c = (l + j * R) * kCols;
        if (c < d) {
#pragma unroll
          for (int i = 0; i < units<T>(); ++i)
            copy_async(slot + (j * units<T>() + i) * TT * 16, row + c + i * (16 / static_cast<int>(sizeof(T))));
        }
      } else {
#pragma unroll
        for (int e = 0; e < kCols; ++e) {
          const int c = l + R * (j * kCols + e);
          v[j][e] = c < d ? row[c] : T(0);
        }
      }
    }
  }
  __device__ __forceinline__ void take(bool use, uint32_t slot, int l, int d, uint64_t (&out)[NV][kPairs]) const {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if constexpr (VEC) {
        if (use && (l + j * R) * kCols < d) {
#pragma unroll
          for (int i = 0; i < units<T>(); ++i) {
            const uint4 w = ld_shared_v4u(slot + (j * units<T>() + i) * TT * 16);
            if constexpr (sizeof(T) == 2) {
              out[j][0] = widen(w.x), out[j][1] = widen(w.y), out[j][2] = widen(w.z), out[j][3] = widen(w.w);
            } else {
              out[j][2 * i] = f2_pack(__uint_as_float(w.x), __uint_as_float(w.y));
              out[j][2 * i + 1] = f2_pack(__uint_as_float(w.z), __uint_as_float(w.w));
            }
          }
        } else {
#pragma unroll
          for (int e = 0; e < kPairs; ++e) out[j][e] = 0ull;
        }
      } else {
#pragma unroll
        for (int e = 0; e < kPairs; ++e)
          out[j][e] = use ? f2_pack(to_f(v[j][2 * e]), to_f(v[j][2 * e + 1])) : 0ull;
      }
    }
  }
};

__device__ __forceinline__ void put8(float* row, const uint64_t (&v)[kPairs]) {
  ulonglong2* p = reinterpret_cast<ulonglong2*>(row);
  p[0] = make_ulonglong2(v[0], v[1]);
  p[1] = make_ulonglong2(v[2], v[3]);
}
__device__ __forceinline__ uint32_t narrow(uint64_t v) {
  float a, b;
  f2_unpack(v, a, b);
  return pack_bf16x2(a, b);
}
__device__ __forceinline__ void put8(uint16_t* row, const uint64_t (&v)[kPairs]) {
  *reinterpret_cast<uint4*>(row) = make_uint4(narrow(v[0]), narrow(v[1]), narrow(v[2]), narrow(v[3]));
}
__device__ __forceinline__ void put1(float* p, float v) { *p = v; }
__device__ __forceinline__ void put1(uint16_t* p, float v) {
  *p = __bfloat16_as_ushort(__float2bfloat16_rn(v));
}

template <class T, int R, int NV, bool VEC>
__device__ __forceinline__ void put_row(void* base, int64_t row, const uint64_t (&v)[NV][kPairs], int l,
                                        int d) {
  T* p = static_cast<T*>(base) + row * d;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    if constexpr (VEC) {
      const int c = (l + j * R) * kCols;
      if (c < d) put8(p + c, v[j]);
    } else {
#pragma unroll
      for (int e = 0; e < kCols; ++e) {
        const int c = l + R * (j * kCols + e);
        float f[2];
        f2_unpack(v[j][e / 2], f[0], f[1]);
        if (c < d) put1(p + c, f[e % 2]);
      }
    }
  }
}

// Column of element e of group j (VEC: 8 neighbours; else R apart).
template <bool VEC>
__device__ __forceinline__ int column(int l, int j, int e, int R) {
  return VEC ? (l + j * R) * kCols + e : l + R * (j * kCols + e);
}

template <bool VEC, int NV>
__device__ __forceinline__ void load_params(const float* p, float fill, int l, int R, int d,
                                            uint64_t (&out)[NV][kPairs]) {
  auto at = [&](int c) { return c >= d ? 0.f : p != nullptr ? __ldg(p + c) : fill; };
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int e = 0; e < kPairs; ++e)
      out[j][e] = f2_pack(at(column<VEC>(l, j, 2 * e, R)), at(column<VEC>(l, j, 2 * e + 1, R)));
}

// Sums of K values over the R threads of a row (R <= 32: within the warp; R
// > 32: the whole block, one barrier, two buffers in turn).  The order of
// the additions is fixed.
template <int R, int K>
__device__ __forceinline__ void row_sum(float (&v)[K], float* buf, int& phase) {
#pragma unroll
  for (int m = (R < 32 ? R : 32) / 2; m > 0; m >>= 1)
#pragma unroll
    for (int i = 0; i < K; ++i) v[i] += __shfl_xor_sync(0xFFFFFFFFu, v[i], m);
  if constexpr (R > 32) {
    constexpr int W = R / 32;
    float* b = buf + phase * 2 * W;
    phase ^= 1;
    if ((threadIdx.x & 31) == 0) {
#pragma unroll
      for (int i = 0; i < K; ++i) b[i * W + (threadIdx.x >> 5)] = v[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < K; ++i) {
      float s = 0.f;
#pragma unroll
      for (int w = 0; w < W; ++w) s += b[i * W + w];
      v[i] = s;
    }
  }
}

// 1 / (1 + exp(-z)) of a pair.  The exponential and the reciprocal are the
// approximate ones: a relative error of some (|z| + 8) 2^-24, most of it from
// rounding z log2(e).  With expf and a division the forward over 200K x 1024
// takes 540 us instead of 394.
__device__ __forceinline__ uint64_t sigmoid2(uint64_t z) {
  float a, b;
  f2_unpack(f2_mul(z, both(-1.4426950408889634f)), a, b);
  f2_unpack(f2_add(f2_pack(ex2_approx(a), ex2_approx(b)), both(1.f)), a, b);
  return f2_pack(rcp_approx(a), rcp_approx(b));
}
// act(z) in place.  kind 0: z, 1: sigmoid(z), 2: z sigmoid(z).
template <int NV>
__device__ __forceinline__ void gate_values(uint64_t (&z)[NV][kPairs], int kind) {
  if (kind == 0) return;
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int e = 0; e < kPairs; ++e) {
      const uint64_t s = sigmoid2(z[j][e]);
      z[j][e] = kind == 1 ? s : f2_mul(z[j][e], s);
    }
}
// act'(z), and act(z) in `act`.  With t = exp(-|z|) and r = 1 / (1 + t) the
// factors s and 1 - s of the slope are r and t r, swapped by the sign of z: 1
// minus a rounded s would lose all of the slope's bits by z = 17.
__device__ __forceinline__ uint64_t gate_slope(uint64_t z, int kind, uint64_t& act) {
  const uint64_t one = both(1.f);
  if (kind == 0) {
    act = z;
    return one;
  }
  float a, b, za, zb;
  f2_unpack(z, za, zb);
  f2_unpack(f2_mul(f2_pack(fabsf(za), fabsf(zb)), both(-1.4426950408889634f)), a, b);
  const uint64_t t = f2_pack(ex2_approx(a), ex2_approx(b));
  f2_unpack(f2_add(t, one), a, b);
  const float r0 = rcp_approx(a), r1 = rcp_approx(b);
  f2_unpack(f2_mul(t, f2_pack(r0, r1)), a, b);
  const uint64_t s = f2_pack(za < 0.f ? a : r0, zb < 0.f ? b : r1);
  const uint64_t rest = f2_pack(za < 0.f ? r0 : a, zb < 0.f ? r1 : b);  // 1 - s
  if (kind == 1) {
    act = s;
    return f2_mul(s, rest);
  }
  act = f2_mul(z, s);
  return f2_mul(s, f2_fma(z, rest, one));
}

// v - mean in the row's columns; the columns behind them hold 0 and keep it.
template <bool VEC, int R, int NV>
__device__ __forceinline__ void subtract(uint64_t (&v)[NV][kPairs], float mean, const NormArgs& a, int l) {
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    if constexpr (VEC) {
      const uint64_t m = both((l + j * R) * kCols < a.d ? -mean : 0.f);
#pragma unroll
      for (int e = 0; e < kPairs; ++e) v[j][e] = f2_add(v[j][e], m);
    } else {
#pragma unroll
      for (int e = 0; e < kPairs; ++e)
        v[j][e] = f2_add(v[j][e], f2_pack(column<VEC>(l, j, 2 * e, R) < a.d ? -mean : 0.f,
                                          column<VEC>(l, j, 2 * e + 1, R) < a.d ? -mean : 0.f));
    }
  }
}

template <int NV>
__device__ __forceinline__ float total(const uint64_t (&v)[NV][kPairs]) {
  uint64_t s = 0ull;
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int e = 0; e < kPairs; ++e) s = f2_add(s, v[j][e]);
  return f2_sum(s);
}
template <int NV>
__device__ __forceinline__ float total_squares(const uint64_t (&v)[NV][kPairs]) {
  uint64_t s = 0ull;
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int e = 0; e < kPairs; ++e) s = f2_fma(v[j][e], v[j][e], s);
  return f2_sum(s);
}

// In place: v -> (v - mean) with mean the row's (layer form); returns rstd.
template <bool VEC, int R, int NV>
__device__ __forceinline__ float centre(uint64_t (&v)[NV][kPairs], const NormArgs& a, int l, float* buf,
                                        int& phase) {
  if (a.layer) {
    float s[1] = {total(v)};
    row_sum<R, 1>(s, buf, phase);
    subtract<VEC, R, NV>(v, s[0] * a.inv_d, a, l);
  }
  float q[1] = {total_squares(v)};
  row_sum<R, 1>(q, buf, phase);
  return rsqrtf(fmaf(q[0], a.inv_d, a.eps));
}

// The same for two rows of values at once, with half as many reductions.
template <bool VEC, int R, int NV>
__device__ __forceinline__ void centre2(uint64_t (&v)[NV][kPairs], uint64_t (&w)[NV][kPairs],
                                        const NormArgs& a, int l, float* buf, int& phase, float& rv,
                                        float& rw) {
  if (a.layer) {
    float s[2] = {total(v), total(w)};
    row_sum<R, 2>(s, buf, phase);
    subtract<VEC, R, NV>(v, s[0] * a.inv_d, a, l);
    subtract<VEC, R, NV>(w, s[1] * a.inv_d, a, l);
  }
  float q[2] = {total_squares(v), total_squares(w)};
  row_sum<R, 2>(q, buf, phase);
  rv = rsqrtf(fmaf(q[0], a.inv_d, a.eps));
  rw = rsqrtf(fmaf(q[1], a.inv_d, a.eps));
}

template <int R>
__host__ __device__ constexpr int norm_threads() { return R <= 256 ? (R <= 128 ? 128 : 256) : R; }

// Stages of the ring: up to `most`, within 200 KB for a block.
template <int SLOTS, int T, bool VEC>
__host__ __device__ constexpr int ring_stages(int most) {
  const int fit = 200 * 1024 / (SLOTS * T * 16);
  return !VEC ? 1 : fit < 1 ? 1 : fit < most ? fit : most;
}
template <class TB, class TR, int R, int NV, bool VEC, bool BACK>
struct NormPlan {
  static constexpr int T = norm_threads<R>();
  static constexpr int G = R > 32 ? 1 : T / R;  // rows per block (R > 32: R == T)
  static constexpr int kSlots = NV * (BACK ? 2 * units<TR>() + 3 * units<TB>() : units<TR>() + 2 * units<TB>());
  static constexpr int D = ring_stages<kSlots, T, VEC>(BACK ? 3 : 4);
  static constexpr int kSmem = VEC ? D * kSlots * T * 16 : 0;
  static_assert(kSmem <= 227 * 1024, "shared memory budget");
  static_assert(R <= 32 || R == T, "one row per block above a warp");
};

template <class TB, class TR, int R, int NV, bool VEC>
__global__ void __launch_bounds__(norm_threads<R>())
    block_norm_forward_kernel(const NormArgs a) {
  using Pl = NormPlan<TB, TR, R, NV, VEC, false>;
  constexpr int T = Pl::T, G = Pl::G, D = Pl::D;
  extern __shared__ __align__(16) uint8_t ring[];
  __shared__ float buf[4 * (T / 32)];
  const int l = R > 32 ? threadIdx.x : threadIdx.x % R;
  const int grp = R > 32 ? 0 : threadIdx.x / R;
  int phase = 0;
  uint64_t g1[NV][kPairs], b1[NV][kPairs], rs[NV][kPairs], g2[NV][kPairs], b2[NV][kPairs];
  load_params<VEC, NV>(a.g1, 1.f, l, R, a.d, g1);
  load_params<VEC, NV>(a.b1, 0.f, l, R, a.d, b1);
  load_params<VEC, NV>(a.rs, 1.f, l, R, a.d, rs);
  load_params<VEC, NV>(a.g2, 1.f, l, R, a.d, g2);
  load_params<VEC, NV>(a.b2, 0.f, l, R, a.d, b2);
  const int64_t step = static_cast<int64_t>(gridDim.x) * G;
  Operand<TR, R, NV, T, VEC> ox;
  Operand<TB, R, NV, T, VEC> oy, oz;
  constexpr int kY = NV * units<TR>() * T * 16, kZ = kY + NV * units<TB>() * T * 16;
  const uint32_t mine = smem_u32(ring) + threadIdx.x * 16;
  auto fetch = [&](int stage, int64_t row) {
    if (row < a.rows) {
      const uint32_t slot = mine + stage * (Pl::kSlots * T * 16);
      ox.fetch(a.x, row * a.ldx, slot, l, a.d);
      if (a.y != nullptr) oy.fetch(a.y, row * a.ldy, slot + kY, l, a.d);
      if (a.z != nullptr) oz.fetch(a.z, row * a.ldz, slot + kZ, l, a.d);
    }
    if (VEC) copy_commit();
  };
  int64_t row = static_cast<int64_t>(blockIdx.x) * G + grp;
#pragma unroll
  for (int i = 0; i < D; ++i) fetch(i, row + i * step);
  int stage = 0;
  // Groups past the last row go through the same reductions on zeros and
  // store nothing.
  for (int64_t row0 = static_cast<int64_t>(blockIdx.x) * G; row0 < a.rows; row0 += step, row += step) {
    const bool live = row < a.rows;
    uint64_t x[NV][kPairs], y[NV][kPairs], z[NV][kPairs];
    if (VEC) copy_wait<D - 1>();
    const uint32_t slot = mine + stage * (Pl::kSlots * T * 16);
    ox.take(live, slot, l, a.d, x);
    oy.take(live && a.y != nullptr, slot + kY, l, a.d, y);
    oz.take(live && a.z != nullptr, slot + kZ, l, a.d, z);
    fetch(stage, row + D * step);
    stage = stage + 1 == D ? 0 : stage + 1;
    if (a.y != nullptr) {
      if (a.z != nullptr) gate_values(z, a.gate_kind);
      if (a.g1 != nullptr) {
        const uint64_t ry = both(centre<VEC, R, NV>(y, a, l, buf, phase));
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
          for (int e = 0; e < kPairs; ++e) y[j][e] = f2_fma(f2_mul(y[j][e], ry), g1[j][e], b1[j][e]);
      }
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int e = 0; e < kPairs; ++e)
          x[j][e] = f2_fma(a.z != nullptr ? f2_mul(rs[j][e], z[j][e]) : rs[j][e], y[j][e], x[j][e]);
      if (a.o1 != nullptr && live) put_row<TR, R, NV, VEC>(a.o1, row, x, l, a.d);
    }
    if (a.o2 != nullptr) {
      const uint64_t rr = both(centre<VEC, R, NV>(x, a, l, buf, phase));
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int e = 0; e < kPairs; ++e) x[j][e] = f2_fma(f2_mul(x[j][e], rr), g2[j][e], b2[j][e]);
      if (live) put_row<TB, R, NV, VEC>(a.o2, row, x, l, a.d);
    }
  }
}

// At 128 threads the backward takes the registers it wants (162, three blocks
// per SM: 254 us over 400K x 128; cut to 128 for four blocks it spills and
// takes 317); a block of 512 threads is alone on its SM.
template <int R>
__host__ __device__ constexpr int norm_blocks() { return R == 512 ? 1 : 0; }

template <class TB, class TR, int R, int NV, bool VEC>
__global__ void __launch_bounds__(norm_threads<R>(), norm_blocks<R>())
    block_norm_backward_kernel(const NormArgs a) {
  using Pl = NormPlan<TB, TR, R, NV, VEC, true>;
  constexpr int T = Pl::T, G = Pl::G, D = Pl::D;
  extern __shared__ __align__(16) uint8_t ring[];
  __shared__ float buf[4 * (T / 32)];
  __shared__ float red[G > 1 ? T * kCols : 1];
  const int l = R > 32 ? threadIdx.x : threadIdx.x % R;
  const int grp = R > 32 ? 0 : threadIdx.x / R;
  int phase = 0;
  uint64_t g1[NV][kPairs], b1[NV][kPairs], rs[NV][kPairs], g2[NV][kPairs];
  load_params<VEC, NV>(a.g1, 1.f, l, R, a.d, g1);
  load_params<VEC, NV>(a.b1, 0.f, l, R, a.d, b1);
  load_params<VEC, NV>(a.rs, 1.f, l, R, a.d, rs);
  load_params<VEC, NV>(a.g2, 1.f, l, R, a.d, g2);
  uint64_t acc[5][NV][kPairs];  // dg1, db1, drs, dg2, db2
#pragma unroll
  for (int i = 0; i < 5; ++i)
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int e = 0; e < kPairs; ++e) acc[i][j][e] = 0ull;
  const int64_t step = static_cast<int64_t>(gridDim.x) * G;
  Operand<TR, R, NV, T, VEC> ox, odr;
  Operand<TB, R, NV, T, VEC> oy, oz, odu;
  constexpr int kDr = NV * units<TR>() * T * 16, kY = 2 * kDr, kZ = kY + NV * units<TB>() * T * 16,
                kDu = kZ + NV * units<TB>() * T * 16;
  const uint32_t mine = smem_u32(ring) + threadIdx.x * 16;
  auto fetch = [&](int stage, int64_t row) {
    if (row < a.rows) {
      const uint32_t slot = mine + stage * (Pl::kSlots * T * 16);
      if (a.du != nullptr) {
        ox.fetch(a.x, row * a.ldx, slot, l, a.d);
        odu.fetch(a.du, row * a.lddu, slot + kDu, l, a.d);
      }
      if (a.y != nullptr) oy.fetch(a.y, row * a.ldy, slot + kY, l, a.d);
      if (a.z != nullptr) oz.fetch(a.z, row * a.ldz, slot + kZ, l, a.d);
      if (a.dr != nullptr) odr.fetch(a.dr, row * a.lddr, slot + kDr, l, a.d);
    }
    if (VEC) copy_commit();
  };
  int64_t row = static_cast<int64_t>(blockIdx.x) * G + grp;
#pragma unroll
  for (int i = 0; i < D; ++i) fetch(i, row + i * step);
  int stage = 0;
  // Groups past the last row go through the same reductions on zeros, which
  // add nothing to the sums, and store nothing.
  for (int64_t row0 = static_cast<int64_t>(blockIdx.x) * G; row0 < a.rows; row0 += step, row += step) {
    const bool live = row < a.rows;
    uint64_t x[NV][kPairs], dx[NV][kPairs], y[NV][kPairs], z[NV][kPairs], h[NV][kPairs];
    if (VEC) copy_wait<D - 1>();
    const uint32_t slot = mine + stage * (Pl::kSlots * T * 16);
    ox.take(live && a.du != nullptr, slot, l, a.d, x);
    odu.take(live && a.du != nullptr, slot + kDu, l, a.d, h);
    oy.take(live && a.y != nullptr, slot + kY, l, a.d, y);
    oz.take(live && a.z != nullptr, slot + kZ, l, a.d, z);
    odr.take(live && a.dr != nullptr, slot + kDr, l, a.d, dx);
    fetch(stage, row + D * step);
    stage = stage + 1 == D ? 0 : stage + 1;
    float rr = 1.f, ry = 1.f;
    if (a.du != nullptr && a.g1 != nullptr)
      centre2<VEC, R, NV>(x, y, a, l, buf, phase, rr, ry);
    else if (a.du != nullptr)
      rr = centre<VEC, R, NV>(x, a, l, buf, phase);
    else if (a.g1 != nullptr)
      ry = centre<VEC, R, NV>(y, a, l, buf, phase);
    if (a.du != nullptr) {
      const uint64_t r2 = both(rr);
      uint64_t s0 = 0ull, s1 = 0ull;
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int e = 0; e < kPairs; ++e) {
          const uint64_t xh = f2_mul(x[j][e], r2), du = h[j][e];
          acc[3][j][e] = f2_fma(du, xh, acc[3][j][e]);
          acc[4][j][e] = f2_add(acc[4][j][e], du);
          x[j][e] = xh;
          h[j][e] = f2_mul(du, g2[j][e]);
          s0 = f2_fma(h[j][e], xh, s0);
          s1 = f2_add(s1, h[j][e]);
        }
      float s[2] = {f2_sum(s0), f2_sum(s1)};
      row_sum<R, 2>(s, buf, phase);
      const uint64_t c1 = both(-s[0] * a.inv_d), c2 = both(a.layer ? -s[1] * a.inv_d : 0.f);
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int e = 0; e < kPairs; ++e)
          dx[j][e] = f2_fma(r2, f2_fma(x[j][e], c1, f2_add(h[j][e], c2)), dx[j][e]);
    }
    if (a.o1 != nullptr && live) put_row<TR, R, NV, VEC>(a.o1, row, dx, l, a.d);
    if (a.y == nullptr) continue;
    const uint64_t r1 = both(ry);
    uint64_t s0 = 0ull, s1 = 0ull;
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int e = 0; e < kPairs; ++e) {
        const uint64_t yh = f2_mul(y[j][e], r1);
        const uint64_t n = f2_fma(yh, g1[j][e], b1[j][e]);
        const uint64_t ds = f2_mul(dx[j][e], rs[j][e]);
        uint64_t dn = ds, n2 = n;  // n2: act n
        if (a.z != nullptr) {
          uint64_t act;
          const uint64_t slope = gate_slope(z[j][e], a.gate_kind, act);
          z[j][e] = f2_mul(f2_mul(ds, n), slope);  // dz
          dn = f2_mul(ds, act);
          n2 = f2_mul(act, n);
        }
        acc[2][j][e] = f2_fma(dx[j][e], n2, acc[2][j][e]);
        acc[0][j][e] = f2_fma(dn, yh, acc[0][j][e]);
        acc[1][j][e] = f2_add(acc[1][j][e], dn);
        const uint64_t p = f2_mul(dn, g1[j][e]);
        y[j][e] = yh;
        dx[j][e] = p;
        s0 = f2_fma(p, yh, s0);
        s1 = f2_add(s1, p);
      }
    if (a.o3 != nullptr && live) put_row<TB, R, NV, VEC>(a.o3, row, z, l, a.d);
    if (a.g1 != nullptr) {
      float s[2] = {f2_sum(s0), f2_sum(s1)};
      row_sum<R, 2>(s, buf, phase);
      const uint64_t c1 = both(-s[0] * a.inv_d), c2 = both(a.layer ? -s[1] * a.inv_d : 0.f);
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int e = 0; e < kPairs; ++e)
          dx[j][e] = f2_mul(r1, f2_fma(y[j][e], c1, f2_add(dx[j][e], c2)));
    }
    if (a.o2 != nullptr && live) put_row<TB, R, NV, VEC>(a.o2, row, dx, l, a.d);
  }
  if (!a.sums) return;
  // The block's column sums: its row groups in ascending order.
  float* part = a.part + static_cast<int64_t>(blockIdx.x) * 5 * a.d;
#pragma unroll
  for (int i = 0; i < 5; ++i)
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if constexpr (G > 1) {
        __syncthreads();
#pragma unroll
        for (int e = 0; e < kPairs; ++e) {
          float lo, hi;
          f2_unpack(acc[i][j][e], lo, hi);
          red[2 * e * T + threadIdx.x] = lo;
          red[(2 * e + 1) * T + threadIdx.x] = hi;
        }
        __syncthreads();
        if (grp == 0) {
#pragma unroll
          for (int e = 0; e < kCols; ++e) {
            float s = 0.f;
            for (int g = 0; g < G; ++g) s += red[e * T + g * R + l];
            const int c = column<VEC>(l, j, e, R);
            if (c < a.d) part[i * a.d + c] = s;
          }
        }
      } else {
#pragma unroll
        for (int e = 0; e < kCols; ++e) {
          const int c = column<VEC>(l, j, e, R);
          float v[2];
          f2_unpack(acc[i][j][e / 2], v[0], v[1]);
          if (c < a.d) part[i * a.d + c] = v[e % 2];
        }
      }
    }
}

struct NormSums {
  float* out[5];
};

// out[i][c] = the blocks' column sums in ascending order (16 interleaved runs
// per column in fp64, joined in a fixed order): bitwise reproducible.
constexpr int kRuns = 16;
__global__ void __launch_bounds__(32 * kRuns) block_norm_sums_kernel(const float* part, int blocks, int d,
                                                                     NormSums o) {
  __shared__ double red[kRuns][32];
  const int lane = threadIdx.x & 31, run = threadIdx.x >> 5;
  const int e = blockIdx.x * 32 + lane, n = 5 * d;
  grid_dependency_wait();
  double s = 0.0;
  if (e < n) {
#pragma unroll 8
    for (int b = run; b < blocks; b += kRuns) s += part[static_cast<int64_t>(b) * n + e];
  }
  red[run][lane] = s;
  __syncthreads();
  if (run == 0 && e < n) {
    for (int r = 1; r < kRuns; ++r) s += red[r][lane];
    float* out = o.out[e / d];
    if (out != nullptr) out[e % d] = static_cast<float>(s);
  }
}

// Threads per row: the power of two that covers d with one group of 8
// columns per thread, 4 to 512; above 4096 columns two groups.
int row_threads(int d) {
  int r = 4;
  while (r * kCols < d && r < 512) r *= 2;
  return r == 64 ? 128 : r;  // a block of one row has at least 128 threads
}

template <class TB, class TR, int R, int NV, bool VEC, bool BACK>
cudaError_t launch_norm(const NormArgs& a, int sms, int* blocks, cudaStream_t st) {
  using Pl = NormPlan<TB, TR, R, NV, VEC, BACK>;
  void (*kernel)(NormArgs);
  if constexpr (BACK) kernel = block_norm_backward_kernel<TB, TR, R, NV, VEC>;
  else kernel = block_norm_forward_kernel<TB, TR, R, NV, VEC>;
  // Set and asked once per device: blocks that fit an SM.
  static std::atomic<int> resident[kMaxDevices];
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  int per_sm = dev < kMaxDevices ? resident[dev].load(std::memory_order_relaxed) : 0;
  if (per_sm == 0) {
    if (Pl::kSmem > 0)
      err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Pl::kSmem);
    if (err == cudaSuccess)
      err = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, Pl::T, Pl::kSmem);
    if (err != cudaSuccess) return err;
    if (per_sm < 1) per_sm = 1;
    if (dev < kMaxDevices) resident[dev].store(per_sm, std::memory_order_relaxed);
  }
  const int64_t need = (a.rows + Pl::G - 1) / Pl::G;
  const int64_t most = static_cast<int64_t>(sms) * per_sm;
  *blocks = static_cast<int>(need < most ? need : most);
  kernel<<<static_cast<unsigned>(*blocks), Pl::T, Pl::kSmem, st>>>(a);
  return cudaGetLastError();
}

template <class TB, class TR, bool VEC, bool BACK>
cudaError_t dispatch_width(const NormArgs& a, int sms, int* blocks, cudaStream_t st) {
  switch (row_threads(a.d)) {
    case 4: return launch_norm<TB, TR, 4, 1, VEC, BACK>(a, sms, blocks, st);
    case 8: return launch_norm<TB, TR, 8, 1, VEC, BACK>(a, sms, blocks, st);
    case 16: return launch_norm<TB, TR, 16, 1, VEC, BACK>(a, sms, blocks, st);
    case 32: return launch_norm<TB, TR, 32, 1, VEC, BACK>(a, sms, blocks, st);
    case 128: return launch_norm<TB, TR, 128, 1, VEC, BACK>(a, sms, blocks, st);
    case 256: return launch_norm<TB, TR, 256, 1, VEC, BACK>(a, sms, blocks, st);
    default: break;
  }
  return a.d <= 4096 ? launch_norm<TB, TR, 512, 1, VEC, BACK>(a, sms, blocks, st)
                     : launch_norm<TB, TR, 512, 2, VEC, BACK>(a, sms, blocks, st);
}

bool al(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) % n) == 0; }

// 16-byte accesses: every row of every operand starts on a 16-byte boundary
// and holds whole groups of 8 columns.
bool vector_rows(const NormArgs& a, size_t er, size_t eb) {
  if (a.d % 8 != 0) return false;
  const void* rp[] = {a.x, a.dr, a.o1};
  const int64_t rl[] = {a.x ? a.ldx : 0, a.dr ? a.lddr : 0, 0};
  for (int i = 0; i < 3; ++i)
    if (!al(rp[i], 16) || rl[i] * er % 16 != 0) return false;
  const void* bp[] = {a.y, a.z, a.du, a.o2, a.o3};
  const int64_t bl[] = {a.y ? a.ldy : 0, a.z ? a.ldz : 0, a.du ? a.lddu : 0, 0, 0};
  for (int i = 0; i < 5; ++i)
    if (!al(bp[i], 16) || bl[i] * eb % 16 != 0) return false;
  return true;
}

template <class TB, class TR>
cudaError_t dispatch_types(const NormArgs& a, bool vec, bool backward, int sms, int* blocks,
                           cudaStream_t st) {
  if (backward)
    return vec ? dispatch_width<TB, TR, true, true>(a, sms, blocks, st)
               : dispatch_width<TB, TR, false, true>(a, sms, blocks, st);
  return vec ? dispatch_width<TB, TR, true, false>(a, sms, blocks, st)
             : dispatch_width<TB, TR, false, false>(a, sms, blocks, st);
}

cudaError_t dispatch(const NormArgs& a, sa_dtype tr, sa_dtype tb, bool backward, int sms,
                     int* blocks, cudaStream_t st) {
  const bool vec = vector_rows(a, tr == SA_BF16 ? 2 : 4, tb == SA_BF16 ? 2 : 4);
  if (tb == SA_FP32) return dispatch_types<float, float>(a, vec, backward, sms, blocks, st);
  if (tr == SA_FP32) return dispatch_types<uint16_t, float>(a, vec, backward, sms, blocks, st);
  return dispatch_types<uint16_t, uint16_t>(a, vec, backward, sms, blocks, st);
}

// Most blocks the backward pass may launch on a device of `sms` SMs (its
// partial sums are sized for them): 16 blocks of 128 threads fill an SM.
int64_t most_blocks(int sms, int d) {
  const int r = row_threads(d);
  const int t = r <= 128 ? 128 : r;
  return static_cast<int64_t>(sms) * (2048 / t);
}

sa_status device_sms(int* sms) {
  int dev = 0, major = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
      cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return SA_ERR_CUDA;
  return major == 10 ? SA_OK : SA_ERR_UNSUPPORTED;
}

bool norm_args_ok(const NormArgs& a, sa_dtype tr, sa_dtype tb, int kind, int gate_kind) {
  if (a.rows < 0 || a.rows >= (int64_t{1} << 40) || a.d < 1 || a.d > kMaxNormWidth) return false;
  if ((tr != SA_BF16 && tr != SA_FP32) || (tb != SA_BF16 && tb != SA_FP32) ||
      (tb == SA_FP32 && tr != SA_FP32))
    return false;
  if (kind < 0 || kind > 1 || gate_kind < 0 || gate_kind > 2) return false;
  if (!(a.eps > 0.f) || !(a.eps < 3.0e38f)) return false;
  const size_t er = tr == SA_BF16 ? 2 : 4, eb = tb == SA_BF16 ? 2 : 4;
  if (!al(a.x, er) || !al(a.y, eb) || !al(a.z, eb) || !al(a.dr, er) || !al(a.du, eb) ||
      !al(a.o1, er) || !al(a.g1, 4) || !al(a.b1, 4) || !al(a.rs, 4) || !al(a.g2, 4) ||
      !al(a.b2, 4) || !al(a.o2, eb) || !al(a.o3, eb))
    return false;
  const int64_t ld[] = {a.ldx, a.y ? a.ldy : a.d, a.z ? a.ldz : a.d, a.dr ? a.lddr : a.d,
                        a.du ? a.lddu : a.d};
  for (int64_t l : ld)
    if (l < a.d || l >= (int64_t{1} << 40)) return false;
  // What applies to the block's output needs a block, a bias its gain.
  if (a.y == nullptr && (a.z || a.g1 || a.rs)) return false;
  if ((a.b1 && !a.g1) || (a.b2 && !a.g2)) return false;
  return true;
}

}  // namespace
}  // namespace sa

extern "C" {

sa_status sa_block_norm_forward(const void* residual, int64_t ld_residual, const void* block,
                                int64_t ld_block, const void* gate, int64_t ld_gate,
                                const float* post_gain, const float* post_bias,
                                const float* res_scale, const float* pre_gain,
                                const float* pre_bias, int64_t rows, int d,
                                sa_dtype residual_dtype, sa_dtype dtype, sa_norm_kind kind,
                                sa_gate_kind gate_kind, float eps, void* residual_out,
                                void* normed, void* stream) {
  sa::NormArgs a = {};
  a.x = residual, a.y = block, a.z = gate;
  a.ldx = ld_residual, a.ldy = ld_block, a.ldz = ld_gate;
  a.g1 = post_gain, a.b1 = post_bias, a.rs = res_scale, a.g2 = pre_gain, a.b2 = pre_bias;
  a.o1 = residual_out, a.o2 = normed;
  a.rows = rows, a.d = d, a.layer = kind == SA_NORM_LAYER, a.gate_kind = gate_kind;
  a.eps = eps, a.inv_d = d > 0 ? 1.f / static_cast<float>(d) : 0.f;
  if (!sa::norm_args_ok(a, residual_dtype, dtype, kind, gate_kind)) return SA_ERR_INVALID_ARG;
  // u needs its gain; r is written if and only if there is a block to add.
  if ((normed == nullptr) != (pre_gain == nullptr) || (residual_out == nullptr) != (block == nullptr) ||
      (normed == nullptr && residual_out == nullptr))
    return SA_ERR_INVALID_ARG;
  if (rows == 0) return SA_OK;
  if (residual == nullptr) return SA_ERR_INVALID_ARG;
  int sms = 0, blocks = 0;
  const sa_status s = sa::device_sms(&sms);
  if (s != SA_OK) return s;
  return sa::dispatch(a, residual_dtype, dtype, false, sms, &blocks,
                      static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? SA_OK
             : SA_ERR_CUDA;
}

size_t sa_workspace_bytes_block_norm(int64_t rows, int d) {
  int sms = 0;
  if (rows < 0 || d < 1 || d > sa::kMaxNormWidth || sa::device_sms(&sms) != SA_OK) return 0;
  const int64_t most = sa::most_blocks(sms, d);
  const int64_t blocks = rows < 1 ? 1 : rows < most ? rows : most;
  return static_cast<size_t>(blocks) * 5 * d * sizeof(float);
}

sa_status sa_block_norm_backward(const void* residual_out, int64_t ld_residual, const void* block,
                                 int64_t ld_block, const void* gate, int64_t ld_gate,
                                 const float* post_gain, const float* post_bias,
                                 const float* res_scale, const float* pre_gain, int64_t rows,
                                 int d, sa_dtype residual_dtype, sa_dtype dtype,
                                 sa_norm_kind kind, sa_gate_kind gate_kind, float eps,
                                 const void* d_residual_out, int64_t ld_d_residual,
                                 const void* d_normed, int64_t ld_d_normed, void* d_residual,
                                 void* d_block, void* d_gate, float* d_post_gain,
                                 float* d_post_bias, float* d_res_scale, float* d_pre_gain,
                                 float* d_pre_bias, void* workspace, size_t workspace_bytes,
                                 void* stream) {
  sa::NormArgs a = {};
  a.x = residual_out, a.y = block, a.z = gate;
  a.ldx = d_normed != nullptr ? ld_residual : d, a.ldy = ld_block, a.ldz = ld_gate;
  a.g1 = post_gain, a.b1 = post_bias, a.rs = res_scale, a.g2 = pre_gain;
  a.dr = d_residual_out, a.du = d_normed, a.lddr = ld_d_residual, a.lddu = ld_d_normed;
  a.o1 = d_residual, a.o2 = d_block, a.o3 = d_gate;
  a.rows = rows, a.d = d, a.layer = kind == SA_NORM_LAYER, a.gate_kind = gate_kind;
  a.eps = eps, a.inv_d = d > 0 ? 1.f / static_cast<float>(d) : 0.f;
  a.part = static_cast<float*>(workspace);
  const sa::NormSums sums = {{d_post_gain, d_post_bias, d_res_scale, d_pre_gain, d_pre_bias}};
  for (float* p : sums.out) {
    if (!sa::al(p, 4)) return SA_ERR_INVALID_ARG;
    a.sums |= p != nullptr;
  }
  if (!sa::norm_args_ok(a, residual_dtype, dtype, kind, gate_kind)) return SA_ERR_INVALID_ARG;
  if ((d_normed == nullptr) != (pre_gain == nullptr) ||
      (d_normed == nullptr && d_residual_out == nullptr) || d_residual == nullptr ||
      (block == nullptr) != (d_block == nullptr) || (gate == nullptr) != (d_gate == nullptr) ||
      ((d_post_gain || d_post_bias) && !post_gain) || (d_res_scale && !block) ||
      ((d_pre_gain || d_pre_bias) && !pre_gain))
    return SA_ERR_INVALID_ARG;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (rows == 0) {
    for (float* p : sums.out)
      if (p != nullptr && cudaMemsetAsync(p, 0, sizeof(float) * d, st) != cudaSuccess)
        return SA_ERR_CUDA;
    return SA_OK;
  }
  if (d_normed != nullptr && residual_out == nullptr) return SA_ERR_INVALID_ARG;
  int sms = 0, blocks = 0;
  const sa_status s = sa::device_sms(&sms);
  if (s != SA_OK) return s;
  if (a.sums) {
    if (workspace == nullptr || !sa::al(workspace, 16)) return SA_ERR_INVALID_ARG;
    if (workspace_bytes < sa_workspace_bytes_block_norm(rows, d)) return SA_ERR_WORKSPACE;
  }
  if (sa::dispatch(a, residual_dtype, dtype, true, sms, &blocks, st) != cudaSuccess)
    return SA_ERR_CUDA;
  if (!a.sums) return SA_OK;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((5 * d + 31) / 32);
  cfg.blockDim = dim3(32 * sa::kRuns);
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, sa::block_norm_sums_kernel,
                            static_cast<const float*>(workspace), blocks, d, sums) == cudaSuccess
             ? SA_OK
             : SA_ERR_CUDA;
}

}  // extern "C"
