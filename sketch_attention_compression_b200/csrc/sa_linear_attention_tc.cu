// Linear attention with a decay per head on the tensor cores (bf16 inputs).
// The scans and their formulas are in sa_linear_attention.h.  Chunks have 128
// rows; per chunk, with all operands in shared memory:
//
//   M1  P   = a b^T                   M 128, N 128, K da
//       P~  = mul P, weighted and masked   (bf16, TMEM)
//   M2  O2  = a S~                    M 128, N dc,  K da   (S~: S in bf16)
//   M3  O1  = P~ c                    M 128, N dc,  K 128  (A from TMEM)
//   M4  D^T = c^T (w b)               M dc,  N da,  K 128, w_j = l^(L-1-r_j)
//       out = O1 + mul l^(r+1) O2;  S <- l^L S + D
//
// Roundings to bf16: P~ and S~, the operands of an output that is bf16
// itself.  They take its error from 1.7e-3 (its own rounding) to 2.3e-3 of its
// 2-norm; second parts would double M2 and M3, and at da = dc = 128 there is
// no shared memory for S~'s.  S^T is kept in fp32 registers: w b is split into bf16 parts whose
// products are all accumulated, three parts (24 significant bits) where the
// state itself is an answer, two (16 bits) where only S~ is taken from it;
// each chunk's D starts from zero and is added to S in registers, so that
// long sums are not left to the accumulator's rounding.
//
// One persistent CTA per SM: warp 0 fetches work items and loads tiles (TMA,
// two or three stages), warp 1 issues the MMAs.  Warps 4-11 hold the state, two warps
// per TMEM lane quarter, each with half of the columns; per chunk they
//   s1  add D of the chunk before to S and store S~
//   s3  split w b: into a place of its own (da = dc = 64), the first part
//       over b once M1 has read it (da = 64), or also the others over a and
//       in S~'s place once M2 has read those
// and warps 12-15, one row of the chunk per thread,
//   s2  turn P into P~ (TMEM to TMEM), while M2 and s3 run
//   s4  store out, while M4 runs.
// (Warps 4-11 that stored a part of out too were slower, and so were eight
// warps for the output: backward of 16 x 10K rows at eight heads of 128: 857
// us, with 96 of 128 columns stored by warps 4-11 932, with 20 warps 969.)
// What bounds it: the chain s1, M2, s3, M4 from chunk to chunk, some 7000
// cycles at da = dc = 128 (8500 with three parts) against 5500 for the chunk's
// share of DRAM.  No unit is full (148 histories of 4096 rows at da = dc =
// 128: tensor pipe 38 % of its cycles, issue slots 40 %, shared-memory pipe
// 38 %, DRAM 49 %), but the products read 8 KB of shared memory every 64
// cycles, all that it has, so that they and s3 slow each other down where they
// meet: M4 by halves of the rows, to start during s3, made a chunk 8 % longer.
// Code size counts too: unrolling s2's loop made it 40 % longer.  With da = 64
// the parts of w b lie side by side, and one product of N = 128 or 192 reads c
// once for all of them.
// Measured: 16 x 100K rows, two heads of 64: 0.72-0.80 ms (2.1-2.3 TB/s of its
// own bytes), of which the segments' states take 0.22; 48 ragged histories of
// up to 4099 rows, eight heads of 128: 0.16-0.18 ms (3.3-3.7 TB/s), 0.14
// without final states (two parts); backward of 16 x 10K rows, eight heads of
// 128: 0.89-1.04 ms (2.2-2.6 TB/s).
// TMEM: P and P~ at 0, O1 at 128, O2 at 256, D behind it.  Shared memory at
// da = dc = 128: two stages of three 32 KB tiles and 32 KB for S~: 224 KB.
//
// A product of P~ = 0 with a c that is not finite is NaN, so a row could see
// such a value in its future.  An output whose O1 is not finite although the
// state's share is no NaN is summed again over the rows that it may see
// (sum_again): in the first chunk of a user and head that holds such a value,
// and in later ones only for columns that the state has not made NaN by then.
#include <cuda_bf16.h>

#include "sa.h"
#include "sa_internal.h"
#include "sa_linear_attention.h"
#include "sa_operators.cuh"

namespace sa {
namespace {

constexpr int kThreads = 512;
constexpr int kStateThreads = 256;  // warps 4-11
constexpr int kRing = 4;
constexpr int kBox = 128 * 128;  // 128 rows x 64 bf16
constexpr int kTable = 132;         // l^0 .. l^128, then l^128's rounding error

template <int DA, int DC, bool STATE>
struct TcPlan {
  // The parts of w b.  da = dc = 64: a place of their own (two in turn for
  // the states alone), and three stages of tiles; da = 64: the first one over
  // b, the others behind it; else over b, over a and in S~'s place.
  static constexpr bool kApart = DA == 64 && DC == 64, kOwn = DA == 64 && !kApart;
  static constexpr int kStages = kApart ? 3 : 2;
  static constexpr int kA = 0;                          // within a stage
  static constexpr int kB = STATE && kApart ? 0 : kA + (DA / 64) * kBox;
  static constexpr int kC = kB + (kOwn ? 3 : DA / 64) * kBox;
  static constexpr int kStage = kC + (DC / 64) * kBox;
  static constexpr int kParts = kStages * kStage;       // (kApart)
  static constexpr int kS = kParts + (kApart ? (STATE ? 6 : 3) * kBox : 0);  // S~^T: da / 64 boxes of dc rows
  static constexpr int kSBox = DC * 128;
  static constexpr int kTab = kS + (DA == 64 ? kSBox : 2 * kBox);  // four tables of powers
  static constexpr int kItems = kTab + 4 * kTable * 4;
  static constexpr int kBars = kItems + kRing * 64;
  static constexpr int kUsed = kBars + 256;
  // M4 with dc = 64 reads a second box behind c's: those rows of D are never
  // used, and the reads stay inside the allocation.  At least 116 KB, so
  // that one CTA holds an SM (it allocates all of TMEM).
  static constexpr int kNeed = kUsed > kS + kBox ? kUsed : kS + kBox;
  static constexpr int kSmem = kNeed > 118784 ? kNeed : 118784;
  static_assert(kSmem <= 232448, "shared memory budget");
  static_assert(kItems % 16 == 0 && kBars % 8 == 0, "alignment");
  static constexpr int kColD = DC == 64 ? 320 : 384;
};

static_assert(sizeof(ScanItem) <= 64, "ring entry");

constexpr uint32_t kColP = 0, kColO1 = 128, kColO2 = 256;

__device__ __forceinline__ uint32_t swz(int r, int u) {
  return (r >> 3) * 1024 + (r & 7) * 128 + ((u ^ (r & 7)) << 4);
}

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// The pairs of eight bf16.
__device__ __forceinline__ void widen8(uint4 w, float (&v)[8]) {
  v[0] = bf_lo(w.x), v[1] = bf_hi(w.x), v[2] = bf_lo(w.y), v[3] = bf_hi(w.y);
  v[4] = bf_lo(w.z), v[5] = bf_hi(w.z), v[6] = bf_lo(w.w), v[7] = bf_hi(w.w);
}

// Sums the outputs of a warp's 32 rows again, in fp32 and over the rows that
// the scan has reached only, where O1 is not finite and O2 is no NaN
// (`batches`: a bit per 16 columns of this thread's row with such an O1).  A
// row's weights are taken once and kept where O1 was: 128 columns of TMEM
// that this warp's lanes own until o_read.  Bound by the latency of loads
// from L2: about 150 us for a chunk at da = dc = 128, against 4 of any other
// chunk (64 users of 512 rows with a row of NaN each, four heads, forward and
// backward: 180 us without, 1200 to 1400 with).  Four weights at a time: 16
// take a third less here, but that much code, though never run, made scans
// without such values 1 to 2 % slower.
template <int DC>
__device__ __forceinline__ void sum_again(const ScanPass& p, int heads, int head, int64_t r0, int L, int row,
                                       uint32_t batches, float w1, uint32_t lane_base, uint32_t powers) {
  __syncwarp();  // the pair's other lane has stored half of this row
  uint32_t todo = 0u;
#pragma unroll 1
  for (int b = 0; b < DC / 16; ++b) {
    if (!__any_sync(0xFFFFFFFFu, (batches >> b) & 1u)) continue;
    uint32_t x[16], y[16];
    tmem_ld16(lane_base + kColO1 + b * 16, x);
    tmem_ld16(lane_base + kColO2 + b * 16, y);
    tmem_wait_ld();
    tmem_pin16(x);
    tmem_pin16(y);
#pragma unroll
    for (int e = 0; e < 16; ++e)
      if (!isfinite(__uint_as_float(x[e])) && !isnan(__uint_as_float(y[e]))) todo |= 1u << b;
  }
  if (row >= L) todo = 0u;
  if (!__any_sync(0xFFFFFFFFu, todo)) return;
  auto line = [&](const ScanInput& in, int r) {  // a row of the chunk (16-byte aligned)
    return reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(in.p) + (r0 + r) * in.row +
                                          static_cast<int64_t>(head) * in.head);
  };
  const bool rev = p.reverse != 0;
  const int base = row & ~31;  // the warp's rows
  const int j0 = rev ? base : 0, j1 = rev ? L : (base + 32 < L ? base + 32 : L);
  const uint4* a = line(p.a, row < L ? row : L - 1);
#pragma unroll 1
  for (int j = j0; j < j1; j += 4) {
    float x[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
    for (int d = 0; d < p.da / 8; ++d) {
      float u[8], v[8];
      widen8(__ldg(a + d), u);
      const uint4* b = line(p.b, j) + d;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        widen8(j + e < L ? __ldg(b) : make_uint4(0u, 0u, 0u, 0u), v);
        b += p.b.row / 8;
#pragma unroll
        for (int i = 0; i < 8; ++i) x[e] = fmaf(u[i], v[i], x[e]);
      }
    }
    // A row that sees a NaN weight is NaN in every column, as it was stored.
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int dist = rev ? j + e - row : row - j - e;
      if (dist >= 0 && isnan(x[e])) todo = 0u;
      tmem_st1(lane_base + kColO1 + j + e,
               dist >= 0 && j + e < L
                   ? __float_as_uint(x[e] * (p.out_mul * ld_shared_f32(powers + dist * 4)))
                   : 0u);
    }
  }
  tmem_wait_st();
  uint16_t* out = static_cast<uint16_t*>(p.out) +
                  ((r0 + row) * static_cast<int64_t>(heads) + head) * DC;
#pragma unroll 1
  for (int b = 0; b < DC / 16; ++b) {
    const bool mine = (todo >> b) & 1u;
    if (!__any_sync(0xFFFFFFFFu, mine)) continue;
    float o[16];
    uint32_t y[16];
    tmem_ld16(lane_base + kColO2 + b * 16, y);
    tmem_wait_ld();
    tmem_pin16(y);
#pragma unroll
    for (int e = 0; e < 16; ++e) o[e] = w1 * __uint_as_float(y[e]);
#pragma unroll 1
    for (int j = j0; j < j1; ++j) {
      const uint4* c = line(p.c, j) + b * 2;  // j < L
      uint4 lo = __ldg(c), hi = __ldg(c + 1);
      uint32_t w;
      tmem_ld1(lane_base + kColO1 + j, w);
      tmem_wait_ld();
      tmem_pin1(w);
      // A weight of 0 would not keep out what is not finite.
      if (rev ? j < row : j > row) lo = hi = make_uint4(0u, 0u, 0u, 0u);
      float v[8];
      widen8(lo, v);
#pragma unroll
      for (int e = 0; e < 8; ++e) o[e] = fmaf(__uint_as_float(w), v[e], o[e]);
      widen8(hi, v);
#pragma unroll
      for (int e = 0; e < 8; ++e) o[8 + e] = fmaf(__uint_as_float(w), v[e], o[8 + e]);
    }
    if (mine) {
      uint32_t z[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) z[e] = pack_bf16x2(o[2 * e], o[2 * e + 1]);
      uint4* q = reinterpret_cast<uint4*>(out + b * 16);
      q[0] = make_uint4(z[0], z[1], z[2], z[3]);
      q[1] = make_uint4(z[4], z[5], z[6], z[7]);
    }
  }
}

// The powers of exp(*log_decay) that one thread of a table's takes.
__device__ __forceinline__ void store_powers(float* table, const float* log_decay, int e) {
  if (e > 128) return;
  const double w = exp(static_cast<double>(usable_decay(__ldg(log_decay))) * e);
  table[e] = static_cast<float>(w);
  if (e == 128) table[129] = static_cast<float>(w - static_cast<float>(w));
}

__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity,
                                          volatile uint32_t* abort_flag, uint32_t* sticky) {
  const bool ok = mbar_wait(bar, parity, abort_flag, sticky);
  return __all_sync(0xFFFFFFFFu, ok);
}

__device__ __forceinline__ void warp_arrive(uint64_t* bar, int lane) {
  __syncwarp();
  if (lane == 0) mbar_arrive(bar);
  __syncwarp();  // the other lanes' next wait must not hold the arrival up
}

// One row of out, from TMEM: O1 + w1 O2.
template <int DC>
__device__ __forceinline__ void store_out(const ScanPass& p, int heads, int head, int64_t r0, int L,
                                          int row, float w1, uint32_t lane_base, uint32_t powers) {
  const bool odd = (row & 1) != 0;
  const uint64_t w2 = f2_pack(w1, w1);
  const int64_t stride = static_cast<int64_t>(heads) * DC;
  uint16_t* o = static_cast<uint16_t*>(p.out) + (r0 + (row & ~1)) * stride + head * DC + (odd ? 8 : 0);
  const bool even_row = (row & ~1) < L, odd_row = (row | 1) < L;
  uint32_t spoiled = 0u;
#pragma unroll 1
  for (int b = 0; b < DC / 16; ++b, o += 16) {
    const int col = b * 16;
    uint32_t x[16], y[16], z[8];
    tmem_ld16(lane_base + kColO1 + col, x);
    tmem_ld16(lane_base + kColO2 + col, y);
    tmem_wait_ld();
    tmem_pin16(x);
    tmem_pin16(y);
    uint64_t finite = 0ull;  // NaN if some O1 is not finite
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint64_t x2 = f2_pack(__uint_as_float(x[2 * e]), __uint_as_float(x[2 * e + 1]));
      const uint64_t y2 = f2_pack(__uint_as_float(y[2 * e]), __uint_as_float(y[2 * e + 1]));
      finite = f2_fma(x2, 0ull, finite);
      float u, v;
      f2_unpack(f2_fma(w2, y2, x2), u, v);
      z[e] = pack_bf16x2(u, v);
    }
    float f0, f1;
    f2_unpack(finite, f0, f1);
    // A thread holds 32 bytes of its row; two threads exchange halves so that
    // their stores cover 32 bytes of one row together.
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t got = __shfl_xor_sync(0xFFFFFFFFu, odd ? z[i] : z[i + 4], 1);
      if (odd) z[i] = got; else z[i + 4] = got;
    }
    if (even_row) *reinterpret_cast<uint4*>(o) = make_uint4(z[0], z[1], z[2], z[3]);
    if (odd_row) *reinterpret_cast<uint4*>(o + stride) = make_uint4(z[4], z[5], z[6], z[7]);
    if (f0 != 0.f || f1 != 0.f) spoiled |= 1u << b;
  }
  if (__any_sync(0xFFFFFFFFu, spoiled))
    sum_again<DC>(p, heads, head, r0, L, row, spoiled, w1, lane_base, powers);
}

template <int DA, int DC, bool STATE>
__global__ void __launch_bounds__(kThreads, 1)
    scan_tc_kernel(const __grid_constant__ ScanMaps maps, const __grid_constant__ ScanArgs t) {
  using Pl = TcPlan<DA, DC, STATE>;
  extern __shared__ __align__(1024) uint8_t smem[];
  constexpr int kStages = Pl::kStages;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if ((smem_u32(smem) & 1023u) != 0u) {
    if (blockIdx.x == 0 && tid == 0) {
      t.s.header->flags = 0u;
      t.s.header->timeout_flags = DEVFLAG_SMEM_ALIGN;
    }
    return;
  }
  // The scans of one call's other shape may start beside this launch; this
  // one ends after the launch that it was started beside.
  grid_dependency_launch();
  if (t.check && blockIdx.x == 0) check_inputs(t.s, reinterpret_cast<uint32_t*>(smem));
  const uint32_t sbase = smem_u32(smem);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + Pl::kBars);
  uint64_t* full = bars;                   // [3] a stage's tiles have landed
  uint64_t* empty = bars + 3;              // [3] a stage's products are done
  uint64_t* item_full = bars + 6;          // [4]
  uint64_t* item_empty = bars + 10;        // [4]
  uint64_t* p_full = bars + 14;            // M1 done
  uint64_t* s_ready = bars + 15;           // S~ stored, D read
  uint64_t* a_free = bars + 16;            // M2 done (and M1)
  uint64_t* p_ready = bars + 17;           // P~ stored
  uint64_t* b_ready = bars + 18;           // w b stored
  uint64_t* o_full = bars + 19;            // M3 done (and M2)
  uint64_t* d_full = bars + 20;            // [2] M4 done (chunks in turn)
  uint64_t* o_read = bars + 22;            // warps 12-15 have read O1, O2
  uint64_t* tab_ready = bars + 23;         // [2] a table of powers stored (state, weight warps)
  uint64_t* drain = bars + 25;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 26);
  volatile uint32_t* abort_flag = tmem_slot + 1;
  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(full + i, 1);
      mbar_init(empty + i, 1);
    }
    for (int i = 0; i < kRing; ++i) {
      mbar_init(item_full + i, 1);
      mbar_init(item_empty + i, STATE ? 9 : 13);
    }
    mbar_init(p_full, 1);
    mbar_init(s_ready, 8);
    mbar_init(a_free, 1);
    mbar_init(p_ready, 4);
    mbar_init(b_ready, 8);
    mbar_init(o_full, 1);
    mbar_init(d_full, 1);
    mbar_init(d_full + 1, 1);
    mbar_init(o_read, 4);
    mbar_init(tab_ready, 8);
    mbar_init(tab_ready + 1, 4);
    mbar_init(drain, 1);
    *abort_flag = 0u;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  uint32_t* sticky = &t.s.header->timeout_flags;
  const uint32_t tmem = *tmem_slot;

  // The next item from the ring; false at the end (hi < lo) or on abort.
  uint32_t ri = 0;  // ring entries taken
  auto take = [&](ScanItem& it, bool& ok) -> bool {
    ok = ok && warp_wait(item_full + ri % kRing, (ri / kRing) & 1u, abort_flag, sticky);
    if (!ok) return false;
    const volatile ScanItem* e = reinterpret_cast<const volatile ScanItem*>(smem + Pl::kItems + (ri % kRing) * 64);
    it.lo = e->lo, it.hi = e->hi, it.state = e->state, it.from = e->from, it.to = e->to;
    it.head = e->head, it.pass = e->pass, it.first = e->first, it.last = e->last;
    warp_arrive(item_empty + ri % kRing, lane);
    ++ri;
    return it.hi >= it.lo;
  };

  if (warp == 0) {
    // ------------------------------------------------------------ items and TMA loads
    bool ok = true;
    uint32_t n = 0;  // chunks loaded
    int64_t next = blockIdx.x;
    while (ok) {
      if (t.counter != nullptr) {
        unsigned long long x = 0;
        if (lane == 0) x = atomicAdd(t.counter, 1ull);
        next = static_cast<int64_t>(__shfl_sync(0xFFFFFFFFu, x, 0));
      }
      ScanItem it;
      const bool end = next >= t.items;
      const bool some = !end && item_of(t, next, lane, STATE, it);
      next += gridDim.x;
      if (!end && !some) continue;
      if (end) it.lo = 0, it.hi = -1;
      if (ri >= kRing) ok = warp_wait(item_empty + ri % kRing, (ri / kRing + 1) & 1u, abort_flag, sticky);
      if (!ok) break;
      if (lane == 0) {
        volatile ScanItem* e = reinterpret_cast<volatile ScanItem*>(smem + Pl::kItems + (ri % kRing) * 64);
        e->lo = it.lo, e->hi = it.hi;
        if (!end) {
          e->state = it.state, e->from = it.from, e->to = it.to;
          e->head = it.head, e->pass = it.pass, e->first = it.first, e->last = it.last;
        }
        mbar_arrive(item_full + ri % kRing);
      }
      ++ri;
      if (end) break;
      const ScanPass& p = t.p[it.pass];
      const int64_t chunks = (it.hi - it.lo + 127) / 128;
      for (int64_t c = 0; c < chunks && ok; ++c, ++n) {
        const uint32_t st = n % kStages;
        if (n >= kStages) ok = warp_wait(empty + st, (n / kStages + 1) & 1u, abort_flag, sticky);
        if (!ok) break;
        if (lane == 0) {
          const int32_t y = it.head;
          const int32_t z = static_cast<int32_t>(it.lo + 128 * (p.reverse ? chunks - 1 - c : c));
          uint8_t* d = smem + st * Pl::kStage;
          mbar_arrive_expect_tx(full + st, ((STATE ? 1 : 2) * (DA / 64) + DC / 64) * kBox);
#pragma unroll
          for (int b = 0; b < DA / 64; ++b) {
            if (!STATE) tma_load_3d(d + Pl::kA + b * kBox, &maps.m[p.map_a], full + st, b * 64, y, z);
            tma_load_3d(d + Pl::kB + b * kBox, &maps.m[p.map_b], full + st, b * 64, y, z);
          }
#pragma unroll
          for (int b = 0; b < DC / 64; ++b)
            tma_load_3d(d + Pl::kC + b * kBox, &maps.m[p.map_c], full + st, b * 64, y, z);
        }
        __syncwarp();
      }
    }
    if (!ok && lane == 0) {
      // Let the copies in flight land before the CTA releases its memory.
      for (uint32_t k = (n >= kStages ? n - kStages : 0); k < n; ++k)
        mbar_wait_bounded(full + k % kStages, (k / kStages) & 1u);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    bool ok = true;
    constexpr uint32_t id_p = idesc_bf16_f32(128, 128, 0, 0);
    constexpr uint32_t id_o2 = idesc_bf16_f32(128, DC, 0, 0);
    constexpr uint32_t id_o1 = idesc_bf16_f32(128, DC, 0, 1);
    constexpr uint32_t id_64 = idesc_bf16_f32(128, 64, 1, 1);
    constexpr uint32_t id_128 = idesc_bf16_f32(128, 128, 1, 1);
    constexpr uint32_t id_192 = idesc_bf16_f32(128, 192, 1, 1);
    uint32_t n = 0;
    // Every lane waits for the issuing one: lanes that ran ahead would poll
    // the next barrier in turns with its instructions.  Products are issued
    // in groups of four steps of K (64 columns of a K-major operand, 64 rows
    // of an MN-major one).
    auto d_col = [&](uint32_t c) { return tmem + (STATE ? (c & 1u) * 256u : Pl::kColD); };
    auto group = [&](uint32_t acc, uint64_t da, int step_a, uint64_t db, int step_b, uint32_t id,
                     bool first) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        mma_bf16_ss(acc, da + i * step_a, db + i * step_b, id, first && i == 0 ? 0u : 1u);
    };
    constexpr int kStepK = 32 >> 4, kStepMn = 2048 >> 4;
    auto m1 = [&](uint32_t c) {
      const uint32_t d = sbase + (c % kStages) * Pl::kStage;
      const uint64_t da = smem_desc(d + Pl::kA, 16, 1024, 2), db = smem_desc(d + Pl::kB, 16, 1024, 2);
#pragma unroll
      for (int g = 0; g < DA / 64; ++g)
        group(tmem + kColP, da + g * (kBox >> 4), kStepK, db + g * (kBox >> 4), kStepK, id_p, g == 0);
      mma_commit(p_full);
    };
    ScanItem it;
    while (take(it, ok)) {
      const int64_t chunks = (it.hi - it.lo + 127) / 128;
      bool ahead = false;  // M1 of this chunk already issued
      for (int64_t c = 0; c < chunks && ok; ++c, ++n) {
        const uint32_t st = n % kStages, ph = n & 1u;
        const uint32_t d = sbase + st * Pl::kStage;
        const uint64_t cm = smem_desc(d + Pl::kC, kBox, 1024, 2);  // c, MN-major
        bool next = false;
        auto ahead_m1 = [&]() {
          if (c + 1 >= chunks) return;
          next = __all_sync(0xFFFFFFFFu,
                            mbar_test_wait(full + (n + 1) % kStages, ((n + 1) / kStages) & 1u));
          if (!next) return;
          tc_fence_after();
          if (lane == 0) m1(n + 1);
          __syncwarp();
        };
        if (!STATE) {
          if (!ahead) {
            if (!warp_wait(full + st, (n / kStages) & 1u, abort_flag, sticky)) { ok = false; break; }
            tc_fence_after();
            if (lane == 0) m1(n);
            __syncwarp();
          }
          if (!warp_wait(s_ready, ph, abort_flag, sticky) ||
              (n > 0 && !warp_wait(o_read, (n - 1) & 1u, abort_flag, sticky))) {
            ok = false;
            break;
          }
          tc_fence_after();
          if (lane == 0) {
            const uint64_t da = smem_desc(d + Pl::kA, 16, 1024, 2);
            const uint64_t sm = smem_desc(sbase + Pl::kS, 16, 1024, 2);
#pragma unroll
            for (int g = 0; g < DA / 64; ++g)
              group(tmem + kColO2, da + g * (kBox >> 4), kStepK, sm + g * (Pl::kSBox >> 4), kStepK, id_o2, g == 0);
            mma_commit(a_free);
          }
          __syncwarp();
          if (!warp_wait(p_ready, ph, abort_flag, sticky)) { ok = false; break; }
          tc_fence_after();
          if (lane == 0) {
#pragma unroll
            for (int g = 0; g < 2; ++g) {
#pragma unroll
              for (int i = 0; i < 4; ++i)
                mma_bf16_ts(tmem + kColO1, tmem + kColP + (g * 4 + i) * 8, cm + (g * 4 + i) * kStepMn, id_o1,
                            g + i > 0 ? 1u : 0u);
            }
            mma_commit(o_full);
          }
          __syncwarp();
          // The next chunk's M1 goes before this chunk's M4 where s3 waits for
          // it, if its tiles are there.
          if (DA == 64) ahead_m1();
        }
        if (!warp_wait(b_ready, ph, abort_flag, sticky)) { ok = false; break; }
        tc_fence_after();
        if (lane == 0) {
          // c^T times the parts of w b, both MN-major.
          const bool three = t.p[it.pass].parts == 3;
          const uint64_t hi = smem_desc(
              Pl::kApart ? sbase + Pl::kParts + (STATE ? (n & 1u) * (3 * kBox) : 0) : d + Pl::kB, kBox, 1024, 2);
          auto product = [&](uint64_t part, uint32_t id, bool first) {
#pragma unroll
            for (int g = 0; g < 2; ++g)
              group(d_col(n), cm + g * 4 * kStepMn, kStepMn, part + g * 4 * kStepMn, kStepMn, id,
                    first && g == 0);
          };
          if (DA == 64) {
            // One product for the parts side by side, 64 columns of D each;
            // with dc = 128 TMEM has room for two of them.
            product(hi, DC == 64 && three ? id_192 : id_128, true);
            if (DC == 128 && three) product(smem_desc(d + Pl::kB + 2 * kBox, kBox, 1024, 2), id_64, false);
          } else {
            product(hi, id_128, true);
            product(smem_desc(d + Pl::kA, kBox, 1024, 2), id_128, false);
            if (three) product(smem_desc(sbase + Pl::kS, kBox, 1024, 2), id_128, false);
          }
          mma_commit(empty + st);
          mma_commit(d_full + (n & 1u));
        }
        __syncwarp();
        if (!STATE && DA != 64) ahead_m1();
        ahead = next;
      }
    }
    if (!ok && lane == 0) {
      mma_commit(drain);
      mbar_wait_bounded(drain, 0);
    }
  } else if (warp >= 4 && warp < 12) {
    // ------------------------------------------------------------ state
    bool ok = true;
    const int q = warp & 3, hf = (warp - 4) >> 2, ctid = tid - 128;
    const int row = q * 32 + lane;  // TMEM lane: column of the state (row of S^T), row of out
    const uint32_t lane_base = tmem + (static_cast<uint32_t>(q * 32) << 16);
    uint32_t tab = 0, items = 0, n = 0;
    constexpr int HA = DA / 2;
    const bool state_row = DC == 128 || q < 2;
    uint64_t S[HA / 2];  // pairs of rows of the state
    ScanItem it;
    auto power = [&](int e) { return ld_shared_f32(tab + e * 4); };
    // S <- (f + fl) S + D of chunk `of`, once its M4 is done.
    auto add_d = [&](uint32_t of, float f, float fl, bool three) {
      if (!ok || !warp_wait(d_full + (of & 1u), (of >> 1) & 1u, abort_flag, sticky)) {
        ok = false;
        return;
      }
      tc_fence_after();
      if (state_row) {
        const uint64_t f2 = f2_pack(f, f), fl2 = f2_pack(fl, fl);
        const uint32_t d = lane_base + (STATE ? (of & 1u) * 256u : Pl::kColD) + hf * HA;
#pragma unroll
        for (int j = 0; j < HA / 16; ++j) {
          uint32_t v[16], lo[16];
          tmem_ld16(d + j * 16, v);
          if (DA == 64) tmem_ld16(d + 64 + j * 16, lo);
          tmem_wait_ld();
          tmem_pin16(v);
          if (DA == 64) {
            tmem_pin16(lo);
            if (DC == 64 && three) {
              uint32_t low[16];
              tmem_ld16(d + 128 + j * 16, low);
              tmem_wait_ld();
              tmem_pin16(low);
#pragma unroll
              for (int e = 0; e < 16; ++e)
                lo[e] = __float_as_uint(__uint_as_float(lo[e]) + __uint_as_float(low[e]));
            }
#pragma unroll
            for (int e = 0; e < 16; ++e)
              v[e] = __float_as_uint(__uint_as_float(v[e]) + __uint_as_float(lo[e]));
          }
#pragma unroll
          for (int e = 0; e < 8; ++e)
            S[j * 8 + e] = f2_fma(f2, S[j * 8 + e],
                                  f2_fma(fl2, S[j * 8 + e],
                                         f2_pack(__uint_as_float(v[2 * e]), __uint_as_float(v[2 * e + 1]))));
        }
      }
      tc_fence_before();
    };
    while (take(it, ok)) {
      const ScanPass& p = t.p[it.pass];
      const bool rev = p.reverse != 0;
      // The decay's powers, in one of two tables: a warp that writes a table
      // has seen tab_ready of the item before, so every warp has left the
      // item before that one, which used the same table.
      tab = sbase + Pl::kTab + (items & 1u) * (kTable * 4);
      store_powers(reinterpret_cast<float*>(smem + Pl::kTab) + (items & 1u) * kTable,
                   t.s.log_decay + it.head, ctid);
      warp_arrive(tab_ready, lane);
      // The state to start from.
      if (state_row) {
        const bool seg = !STATE && it.from >= 0;
        const float* src = STATE ? nullptr : seg ? p.bound : p.ends;
        const float m = seg ? 1.f : p.ends_mul;
        const int64_t o = (seg ? it.from : it.state) * (DA * DC);
        const int step = p.transposed ? 1 : DC;
        const int64_t first = o + (p.transposed ? row * DA + hf * HA : hf * HA * DC + row);
#pragma unroll
        for (int j = 0; j < HA / 2; ++j)
          S[j] = src == nullptr ? 0ull
                                : f2_pack(m * src[first + (2 * j) * step], m * src[first + (2 * j + 1) * step]);
      }
      if (!warp_wait(tab_ready, items & 1u, abort_flag, sticky)) break;
      ++items;
      const int64_t chunks = (it.hi - it.lo + 127) / 128;
      float f = 0.f, fl = 0.f;  // decay of S over the chunk before
      // s3 comes before s1 where its places are free by then.
      const bool early = STATE ? DA == 64 || p.parts == 2 : Pl::kOwn;
      // s3: w b in two or three bf16 parts, for a chunk of L rows at d.
      auto split = [&](uint32_t d, int L, uint32_t m) {
        constexpr int kRowStep = kStateThreads / (DA / 8);  // a multiple of 8
        const int u = ctid % (DA / 8), first = ctid / (DA / 8);
        const uint32_t o = (u >> 3) * kBox + swz(first, u & 7);
        uint32_t src = d + Pl::kB + o;
        uint32_t hi_dst = Pl::kApart ? sbase + Pl::kParts + (STATE ? (m & 1u) * (3 * kBox) : 0) + o : src;
        uint32_t dst = DA == 64 ? hi_dst + kBox : d + Pl::kA + o;
        uint32_t third = DA == 64 ? hi_dst + 2 * kBox : sbase + Pl::kS + o;
        const bool three = p.parts == 3;
        const uint64_t minus = f2_pack(-1.f, -1.f);
#pragma unroll 2
        for (int r = first; r < 128; r += kRowStep) {
          const float w1 = r < L ? power(rev ? r : L - 1 - r) : 0.f;
          const uint64_t w = f2_pack(w1, w1);
          const uint4 x = ld_shared_v4u(src);
          uint32_t v[4] = {x.x, x.y, x.z, x.w};
          if (r >= L) v[0] = v[1] = v[2] = v[3] = 0u;
          uint64_t y[4];
          uint32_t hi[4], lo[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            y[i] = f2_mul(w, f2_pack(bf_lo(v[i]), bf_hi(v[i])));
            float y0, y1;
            f2_unpack(y[i], y0, y1);
            hi[i] = pack_bf16x2(y0, y1);
            y[i] = f2_fma(minus, f2_pack(bf_lo(hi[i]), bf_hi(hi[i])), y[i]);
            f2_unpack(y[i], y0, y1);
            lo[i] = pack_bf16x2(y0, y1);
          }
          st_shared_v4(hi_dst, hi[0], hi[1], hi[2], hi[3]);
          st_shared_v4(dst, lo[0], lo[1], lo[2], lo[3]);
          if (three) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              float y0, y1;
              f2_unpack(f2_fma(minus, f2_pack(bf_lo(lo[i]), bf_hi(lo[i])), y[i]), y0, y1);
              hi[i] = pack_bf16x2(y0, y1);
            }
            st_shared_v4(third, hi[0], hi[1], hi[2], hi[3]);
          }
          src += kRowStep * 128, hi_dst += kRowStep * 128, dst += kRowStep * 128, third += kRowStep * 128;
        }
      };
      // Waits for the tiles of chunk c, number m; s3 too where its places do
      // not depend on M2.
      auto tiles = [&](int64_t c, uint32_t m) {
        const uint32_t d = sbase + (m % kStages) * Pl::kStage;
        const int64_t r0 = it.lo + 128 * (rev ? chunks - 1 - c : c);
        const int L = static_cast<int>(it.hi - r0 < 128 ? it.hi - r0 : 128);
        if (!warp_wait(full + m % kStages, (m / kStages) & 1u, abort_flag, sticky)) return false;
        if (L < 128) {
          // Rows behind the end belong to another user or to nobody: c's must
          // not reach the sums, whatever they hold.
          for (int e = ctid; e < (128 - L) * (DC / 8); e += kStateThreads) {
            const int r = L + e / (DC / 8), u = e % (DC / 8);
            st_shared_v4(d + Pl::kC + (u >> 3) * kBox + swz(r, u & 7), 0u, 0u, 0u, 0u);
          }
        }
        if (early) {
          if (!STATE && !warp_wait(p_full, m & 1u, abort_flag, sticky)) return false;
          split(d, L, m);
        }
        return true;
      };
      for (int64_t c = 0; c < chunks; ++c, ++n) {
        const uint32_t st = n % kStages, ph = n & 1u;
        const uint32_t d = sbase + st * Pl::kStage;
        const int64_t r0 = it.lo + 128 * (rev ? chunks - 1 - c : c);
        const int L = static_cast<int>(it.hi - r0 < 128 ? it.hi - r0 : 128);
        // A reverse scan's first chunk of a user takes the start state undecayed.
        const int skip = rev && it.first && c == 0 ? 1 : 0;
        if (!tiles(c, n)) { ok = false; break; }
        if (STATE && early) {
          // Two places for D: the chunk before is added while M4 runs.
          fence_proxy_async_smem();
          warp_arrive(b_ready, lane);
        }
        // s1
        if (c > 0) add_d(n - 1, f, fl, p.parts == 3);
        if (!ok) break;
        f = power(L - skip);
        fl = L - skip == 128 ? power(129) : 0.f;
        if (!STATE) {
          if (state_row) {
#pragma unroll
            for (int u = 0; u < HA / 8; ++u) {
              const int col = hf * HA + u * 8;
              uint32_t w[4];
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                float x, y;
                f2_unpack(S[u * 4 + i], x, y);
                w[i] = pack_bf16x2(x, y);
              }
              st_shared_v4(sbase + Pl::kS + (col >> 6) * Pl::kSBox + swz(row, (col & 63) >> 3), w[0], w[1],
                           w[2], w[3]);
            }
          }
          fence_proxy_async_smem();
          tc_fence_before();
          warp_arrive(s_ready, lane);
        }
        if (!early) {
          if (!STATE && !Pl::kApart && !warp_wait(a_free, ph, abort_flag, sticky)) { ok = false; break; }
          split(d, L, n);
        }
        if (!STATE || !early) {
          fence_proxy_async_smem();
          warp_arrive(b_ready, lane);
        }
      }
      if (!ok) break;
      if (chunks > 0) add_d(n - 1, f, fl, p.parts == 3);
      if (!ok) break;
      // The state behind the last row.
      float* dst = nullptr;
      float m = 1.f;
      int64_t o = 0;
      if (STATE) {
        dst = p.bound;
        o = it.to * (DA * DC);
      } else if (it.last && p.fin != nullptr) {
        dst = p.fin;
        o = it.state * (DA * DC);
        m = p.fin_mul * (rev && chunks > 0 ? power(1) : 1.f);
      }
      if (dst != nullptr && state_row) {
#pragma unroll
        for (int j = 0; j < HA / 2; ++j) {
          float x, y;
          f2_unpack(S[j], x, y);
          dst[o + (hf * HA + 2 * j) * DC + row] = m * x;
          dst[o + (hf * HA + 2 * j + 1) * DC + row] = m * y;
        }
      }
    }
  } else if (!STATE && warp >= 12) {
    // ------------------------------------------------------------ weights
    bool ok = true;
    const int q = warp & 3, ctid = tid - 384;
    const int row = q * 32 + lane;  // TMEM lane: row of the chunk
    const uint32_t lane_base = tmem + (static_cast<uint32_t>(q * 32) << 16);
    uint32_t items = 0, n = 0;
    ScanItem it;
    while (take(it, ok)) {
      const ScanPass& p = t.p[it.pass];
      const bool rev = p.reverse != 0;
      const uint32_t tab = sbase + Pl::kTab + (2 + (items & 1u)) * (kTable * 4);
      float* table = reinterpret_cast<float*>(smem + Pl::kTab) + (2 + (items & 1u)) * kTable;
      auto power = [&](int e) { return ld_shared_f32(tab + e * 4); };
      store_powers(table, t.s.log_decay + it.head, ctid);
      if (ctid == 0) store_powers(table, t.s.log_decay + it.head, 128);
      warp_arrive(tab_ready + 1, lane);
      if (!warp_wait(tab_ready + 1, items & 1u, abort_flag, sticky)) break;
      ++items;
      const int64_t chunks = (it.hi - it.lo + 127) / 128;
      for (int64_t c = 0; c < chunks; ++c, ++n) {
        const uint32_t ph = n & 1u;
        const int64_t r0 = it.lo + 128 * (rev ? chunks - 1 - c : c);
        const int L = static_cast<int>(it.hi - r0 < 128 ? it.hi - r0 : 128);
        const int skip = rev && it.first && c == 0 ? 1 : 0;
        // s2: 32 columns of P at a time; their 16 columns of P~ go where
        // columns lay that have been read.  A block of 32 x 32 that the scan
        // covers whole has the weight E F_j, both powers with exponents >= 0;
        // the one on the diagonal is masked.
        if (!warp_wait(p_full, ph, abort_flag, sticky)) { ok = false; break; }
        tc_fence_after();
#pragma unroll 1
        for (int jb = 0; jb < 4; ++jb) {
          uint32_t o[16];
          if (rev ? jb < q : jb > q) {
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] = 0u;
          } else {
            uint32_t v[32];
            tmem_ld32(lane_base + kColP + jb * 32, v);
            tmem_wait_ld();
            tmem_pin32(v);
            if (jb == q) {
#pragma unroll
              for (int e = 0; e < 32; ++e) {
                const int dist = rev ? e - lane : lane - e;
                const float w = p.out_mul * power(dist >= 0 ? dist : 0);
                v[e] = dist >= 0 ? __float_as_uint(__uint_as_float(v[e]) * w) : 0u;
              }
#pragma unroll
              for (int e = 0; e < 16; ++e)
                o[e] = pack_bf16x2(__uint_as_float(v[2 * e]), __uint_as_float(v[2 * e + 1]));
            } else {
              const float E1 = p.out_mul * power(rev ? jb * 32 - row : row - jb * 32 - 31);
              const uint64_t E = f2_pack(E1, E1);
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                const uint64_t w = f2_mul(E, f2_pack(power(rev ? 2 * e : 31 - 2 * e),
                                                     power(rev ? 2 * e + 1 : 30 - 2 * e)));
                float x, y;
                f2_unpack(f2_mul(w, f2_pack(__uint_as_float(v[2 * e]), __uint_as_float(v[2 * e + 1]))),
                          x, y);
                o[e] = pack_bf16x2(x, y);
              }
            }
            if (L < jb * 32 + 32) {
              // Columns behind the user's end.
#pragma unroll
              for (int e = 0; e < 16; ++e)
                o[e] &= (jb * 32 + 2 * e < L ? 0xFFFFu : 0u) | (jb * 32 + 2 * e + 1 < L ? 0xFFFF0000u : 0u);
            }
          }
          tmem_st16(lane_base + kColP + jb * 16, o);
        }
        tmem_wait_st();
        tc_fence_before();
        warp_arrive(p_ready, lane);
        // s4
        if (!warp_wait(o_full, ph, abort_flag, sticky)) { ok = false; break; }
        tc_fence_after();
        const float w1 = p.out_mul * power(row < L ? (rev ? L - row : row + 1) - skip : 0);
        store_out<DC>(p, t.s.heads, it.head, r0, L, row, w1, lane_base, tab);
        tc_fence_before();
        warp_arrive(o_read, lane);
      }
      if (!ok) break;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  grid_dependency_wait();
}

template <int DA, int DC, bool STATE>
cudaError_t launch(const ScanMaps& m, const ScanArgs& t, bool beside, int sms, cudaStream_t st) {
  using Pl = TcPlan<DA, DC, STATE>;
  static std::atomic<uint64_t> allowed{0};
  const cudaError_t err = allow_smem(scan_tc_kernel<DA, DC, STATE>, Pl::kSmem, allowed);
  if (err != cudaSuccess) return err;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(t.items < sms ? t.items : sms));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = Pl::kSmem;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = beside ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, scan_tc_kernel<DA, DC, STATE>, m, t);
}

template <bool STATE>
cudaError_t launch_any(const ScanMaps& m, const ScanArgs& t, bool beside, int sms, cudaStream_t st) {
  if (t.p[0].da == 64)
    return t.p[0].dc == 64 ? launch<64, 64, STATE>(m, t, beside, sms, st)
                           : launch<64, 128, STATE>(m, t, beside, sms, st);
  return t.p[0].dc == 64 ? launch<128, 64, STATE>(m, t, beside, sms, st)
                         : launch<128, 128, STATE>(m, t, beside, sms, st);
}

}  // namespace

bool scan_tc_usable(const ScanInput& in) {
  return (reinterpret_cast<uintptr_t>(in.p) & 15u) == 0 && in.row > 0 && in.row % 8 == 0 &&
         in.head > 0 && in.head % 8 == 0;
}

cudaError_t launch_scan_tc(const ScanArgs& t, const ScanMaps& maps, bool states_only, bool beside,
                           int sms, cudaStream_t st) {
  return states_only ? launch_any<true>(maps, t, beside, sms, st)
                     : launch_any<false>(maps, t, beside, sms, st);
}

}  // namespace sa
