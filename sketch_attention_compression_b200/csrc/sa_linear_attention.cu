// Linear attention with a decay per head: the C entry points, the CUDA-core
// scan and the single-step kernel.  The formulas are in sa_linear_attention.h.
#include <cuda_bf16.h>
#include <math.h>

#include "sa.h"
#include "sa_internal.h"
#include "sa_linear_attention.h"
#include "sa_operators.cuh"

namespace sa {
namespace {

__device__ __forceinline__ float load_f(const float* p) { return *p; }
__device__ __forceinline__ float load_f(const uint16_t* p) {
  return __uint_as_float(static_cast<uint32_t>(*p) << 16);
}
__device__ __forceinline__ void store4(float* p, const float (&v)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) p[i] = v[i];
}
__device__ __forceinline__ void store4(uint16_t* p, const float (&v)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) p[i] = __bfloat16_as_ushort(__float2bfloat16_rn(v[i]));
}

// ---------------------------------------------------------------- states between segments
// Boundary j receives the state (gradient of the state) behind (before) it,
// from the segments' own sums.  One thread per four state elements, segment
// after segment.  Bound by latency, one load after the other: 16 sums are
// loaded ahead (8 us for 32 states of 64 x 64 over 37 segments).
struct ChainArgs {
  int reverse;
  const float* ends;
  float ends_mul;
  float* bound;
};

__global__ void __launch_bounds__(256)
    state_chain_kernel(const ScanCommon s, int64_t segment, int elems, const ChainArgs f,
                       const ChainArgs r) {
  const ChainArgs& a = blockIdx.z == 0 ? f : r;
  const int64_t b = blockIdx.x / s.heads;
  const int head = static_cast<int>(blockIdx.x % s.heads);
  int64_t lo, hi;
  user_rows(s, b, lo, hi);
  const int64_t n = hi - lo, count = n > 0 ? (n + segment - 1) / segment : 1;
  const int e = (blockIdx.y * 256 + threadIdx.x) * 4;
  if (count < 2 || e >= elems) return;
  const double g = static_cast<double>(usable_decay(s.log_decay[head]));
  const int64_t step = static_cast<int64_t>(s.heads) * elems;
  float* p = a.bound + ((lo / segment) * s.heads + head) * static_cast<int64_t>(elems) + e;
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
  if (a.ends != nullptr) {
    v = *reinterpret_cast<const float4*>(a.ends + (b * s.heads + head) * static_cast<int64_t>(elems) + e);
    v.x *= a.ends_mul, v.y *= a.ends_mul, v.z *= a.ends_mul, v.w *= a.ends_mul;
  }
  const float whole = static_cast<float>(exp(g * static_cast<double>(segment)));
  const int64_t tail = n - (count - 1) * segment - 1;  // the last segment's rows but one
  const float first = a.reverse ? static_cast<float>(exp(g * static_cast<double>(tail))) : whole;
  constexpr int kAhead = 16;
  float4 x[kAhead];
  auto at = [&](int64_t j) {
    return reinterpret_cast<float4*>(p + (a.reverse ? count - 2 - j : j) * step);
  };
#pragma unroll
  for (int k = 0; k < kAhead; ++k)
    if (k < count - 1) x[k] = *at(k);
  for (int64_t j = 0; j < count - 1; j += kAhead) {
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      if (j + k >= count - 1) break;
      const float m = j + k == 0 ? first : whole;
      v.x = fmaf(m, v.x, x[k].x);
      v.y = fmaf(m, v.y, x[k].y);
      v.z = fmaf(m, v.z, x[k].z);
      v.w = fmaf(m, v.w, x[k].w);
      if (j + k + kAhead < count - 1) x[k] = *at(j + k + kAhead);
      *at(j + k) = v;
    }
  }
}

// ---------------------------------------------------------------- order of the users
// Clears the header, checks the inputs and ranks the users by length, longest
// first, so that a ragged batch does not end with its longest history on one
// SM (48 users of up to 4099 rows at eight heads: 230 -> 182 us).  One block;
// every user counts the longer ones.
constexpr int kMostOrdered = 1024;

__global__ void __launch_bounds__(kMostOrdered) order_kernel(const ScanCommon s, int32_t* order) {
  __shared__ int64_t lens[kMostOrdered];
  __shared__ uint32_t flags;
  const int tid = threadIdx.x, n = static_cast<int>(s.batch);
  if (tid < static_cast<int>(sizeof(WsHeader) / 4)) reinterpret_cast<uint32_t*>(s.header)[tid] = 0u;
  int64_t mine = -1;
  if (tid < n) {
    int64_t lo, hi;
    user_rows(s, tid, lo, hi);
    mine = hi - lo;
  }
  lens[tid] = mine;
  __syncthreads();
  check_inputs(s, &flags);
  if (tid >= n) return;
  int rank = 0;
  for (int i = 0; i < n; ++i) rank += lens[i] > mine || (lens[i] == mine && i < tid);
  order[rank] = tid;
}

// ---------------------------------------------------------------- one step
// S <- l S + k v^T, o = mul S^T q for one row of each listed state.  Bound
// by reading and writing the state once: a thread takes four columns of
// every (threads / column groups)-th state row, its loads issued in batches
// before they are used, and the partial outputs are joined in shared memory
// in a fixed order.  1000 states of eight heads of 128 x 128: 160 us, 6.6
// TB/s; one state of two heads of 64 x 64: 2.5 us in a graph.
struct StepArgs {
  ScanInput q, k, v;       // strides: row = batch entry
  const float* log_decay;
  const int64_t* slots;    // may be null: entry b uses state b
  int64_t batch, states;
  float* state;            // [states][H][dk][dv]
  void* out;               // [batch][H][dv]
  int heads, dk, dv;
  int cols4;               // four-column groups per block
  float mul;
  uint32_t* flags;         // may be null
  int marked;              // mark_kernel has gone before
};

constexpr int kStepThreads = 256, kStepBatch = 8, kStepMaxWidth = 256;
// Of entries with equal slots the first is taken, a later one raises the
// flag.  Up to this many blocks, each looks through the earlier entries' slots
// while its state arrives; above, mark_kernel does so once per entry, not per
// head, and leaves the answer where the entry's output goes.  Eight heads of
// 64 x 64: 2000 entries 127 us (comparing) and 129 (marked), 4000: 260 and 240,
// 10000: 696 and 592; one head, 10000: 100 and 105.
constexpr int64_t kMostComparing = 16384;

__device__ __forceinline__ void store_mark(float* p, bool m) { *p = m ? 1.f : 0.f; }
__device__ __forceinline__ void store_mark(uint16_t* p, bool m) { *p = m ? 1 : 0; }

// Thirty-two entries per block, a lane each; its eight warps share the earlier
// entries, 512 at a time.
template <class T>
__global__ void __launch_bounds__(256) mark_kernel(const StepArgs a) {
  constexpr int kTile = 512;
  __shared__ longlong2 tile[kTile / 2];
  __shared__ uint32_t found[8];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t b0 = static_cast<int64_t>(blockIdx.x) * 32, b = b0 + lane;
  const int64_t slot = b < a.batch ? a.slots[b] : -1;
  const int64_t end = b0 + 32 < a.batch ? b0 + 32 : a.batch;
  auto fetch = [&](int64_t i) { return i < end ? a.slots[i] : -1; };
  int64_t next0 = fetch(tid), next1 = fetch(tid + 256);
  bool twice = false;
  for (int64_t i0 = 0; i0 < end; i0 += kTile) {
    __syncthreads();
    int64_t* t = reinterpret_cast<int64_t*>(tile);
    t[tid] = next0;
    t[tid + 256] = next1;
    __syncthreads();
    next0 = fetch(i0 + kTile + tid);
    next1 = fetch(i0 + kTile + 256 + tid);
    if (i0 + kTile <= b0) {  // all of them earlier than all of the block's
#pragma unroll 8
      for (int j = warp; j < kTile / 2; j += 8) {
        const longlong2 s = tile[j];
        twice |= s.x == slot || s.y == slot;
      }
    } else {
      for (int j = warp; j < kTile / 2; j += 8) {
        const longlong2 s = tile[j];
        twice |= (s.x == slot && i0 + 2 * j < b) || (s.y == slot && i0 + 2 * j + 1 < b);
      }
    }
  }
  const uint32_t m = __ballot_sync(0xFFFFFFFFu, twice);
  if (lane == 0) found[warp] = m;
  __syncthreads();
  uint32_t all = 0u;
#pragma unroll
  for (int w = 0; w < 8; ++w) all |= found[w];
  for (int e = tid; e < 32 * a.heads; e += 256) {
    const int64_t c = b0 + e / a.heads;
    if (c < a.batch)
      store_mark(static_cast<T*>(a.out) + (c * a.heads + e % a.heads) * a.dv, (all >> (e / a.heads)) & 1u);
  }
}

template <class T>
__global__ void __launch_bounds__(kStepThreads) step_kernel(const StepArgs a) {
  __shared__ float sq[kStepMaxWidth], sk[kStepMaxWidth];
  __shared__ float4 red[kStepThreads];
  const int tid = threadIdx.x;
  const int64_t b = blockIdx.x / a.heads;
  const int h = static_cast<int>(blockIdx.x % a.heads);
  const int groups = kStepThreads / a.cols4;         // state rows taken at a time
  const int c4 = tid % a.cols4, g = tid / a.cols4;
  const int col = (blockIdx.y * a.cols4 + c4) * 4;   // first column
  const bool live = g < groups && col < a.dv;
  // A negative slot marks a padded entry, one past the pool raises the flag.
  const int64_t slot = a.slots != nullptr ? a.slots[b] : b;
  const bool padded = slot < 0, past = slot >= a.states, in_pool = !padded && !past;
  const float gd = a.log_decay[h];
  float* st = a.state + (((in_pool ? slot : 0) * a.heads + h) * a.dk) * a.dv + col;
  const T* vp = static_cast<const T*>(a.v.p) + b * a.v.row + h * a.v.head + col;
  float v[4] = {0.f, 0.f, 0.f, 0.f}, o[4] = {0.f, 0.f, 0.f, 0.f};
  float4 s[kStepBatch];
  auto fetch = [&](int r0) {
#pragma unroll
    for (int i = 0; i < kStepBatch; ++i) {
      const int r = r0 + i * groups;
      if (live && r < a.dk) s[i] = *reinterpret_cast<const float4*>(st + static_cast<int64_t>(r) * a.dv);
    }
  };
  if (in_pool) fetch(g);
  static_assert(kStepMaxWidth <= kStepThreads, "an element of q and k per thread");
  float qt = 0.f, kt = 0.f;
  if (tid < a.dk) {
    qt = load_f(static_cast<const T*>(a.q.p) + b * a.q.row + h * a.q.head + tid);
    kt = load_f(static_cast<const T*>(a.k.p) + b * a.k.row + h * a.k.head + tid);
  }
  if (live) {
#pragma unroll
    for (int c = 0; c < 4; ++c) v[c] = load_f(vp + c);
  }
  sq[tid] = qt;
  sk[tid] = kt;
  bool twice = false;
  if (a.marked) {
    twice = static_cast<const T*>(a.out)[(b * a.heads + h) * a.dv] != T(0);
  } else if (a.slots != nullptr && in_pool) {
#pragma unroll 4
    for (int64_t i = tid; i < b; i += kStepThreads) twice |= a.slots[i] == slot;
  }
  // The decay with its rounding error, which has one sign at every step and
  // would add up over the horizon of a state that is advanced row by row: 1 +
  // expm1 as a sum of two where the horizon is longer than two rows.  Rounded
  // down, so that the error's share of an infinite state has its sign, and
  // never 0 while the decay is not.  Taken while the loads are under way.
  const float gu = usable_decay(gd), m = expm1f(gu);
  float e = expf(gu);
  asm("" : "+f"(e));
  const float l1 = __fadd_rd(1.f, m);
  const float l = gu > -0.5f ? l1 : e;
  const float ll = fmaxf(gu > -0.5f ? m - (l1 - 1.f) : 0.f, __fmul_ru(l, 0x1p-100f));
  twice = __syncthreads_or(twice) != 0;
  T* out = static_cast<T*>(a.out) + (b * a.heads + h) * a.dv + col;
  if (padded || past || twice) {
    if (!padded && tid == 0 && a.flags != nullptr) atomicOr(a.flags, SA_DEVFLAG_SLOT);
    const float zero[4] = {0.f, 0.f, 0.f, 0.f};
    if (g == 0 && col < a.dv) store4(out, zero);
    return;
  }
  if (!(gd <= 0.f) && tid == 0 && a.flags != nullptr) atomicOr(a.flags, SA_DEVFLAG_DECAY);
  auto next = [&](float x, float kv) { return fmaf(l, x, fmaf(ll, x, kv)); };
  for (int r0 = g; r0 < a.dk; r0 += kStepBatch * groups) {
    if (r0 != g) fetch(r0);
#pragma unroll
    for (int i = 0; i < kStepBatch; ++i) {
      const int r = r0 + i * groups;
      if (!live || r >= a.dk) continue;
      const float kv = sk[r], qv = sq[r];
      float4 x = s[i];
      x.x = next(x.x, kv * v[0]);
      x.y = next(x.y, kv * v[1]);
      x.z = next(x.z, kv * v[2]);
      x.w = next(x.w, kv * v[3]);
      *reinterpret_cast<float4*>(st + static_cast<int64_t>(r) * a.dv) = x;
      o[0] = fmaf(qv, x.x, o[0]);
      o[1] = fmaf(qv, x.y, o[1]);
      o[2] = fmaf(qv, x.z, o[2]);
      o[3] = fmaf(qv, x.w, o[3]);
    }
  }
  red[tid] = make_float4(o[0], o[1], o[2], o[3]);
  __syncthreads();
  if (g == 0 && col < a.dv) {
    for (int i = 1; i < groups; ++i) {
      const float4 x = red[i * a.cols4 + c4];
      o[0] += x.x;
      o[1] += x.y;
      o[2] += x.z;
      o[3] += x.w;
    }
#pragma unroll
    for (int c = 0; c < 4; ++c) o[c] *= a.mul;
    store4(out, o);
  }
}

bool al(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) % n) == 0; }

bool width_ok(int d) { return d == 64 || d == 128; }

bool input_ok(const ScanInput& in, int heads, int d, size_t elem) {
  const int64_t most = int64_t{1} << 40;
  return al(in.p, elem) && in.row >= 0 && in.row < most && in.head >= 0 && in.head < most &&
         (heads == 1 || in.head >= d);
}

// True if the rows of `in` may meet [out, out + bytes).
bool may_meet(const ScanInput& in, int64_t rows, int heads, int d, size_t elem, const void* out,
              size_t bytes) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(in.p), o = reinterpret_cast<uintptr_t>(out);
  const int64_t last = (rows - 1) * in.row + (heads - 1) * in.head + d;  // elements
  return a < o + bytes && o < a + static_cast<uintptr_t>(last) * elem;
}

// A stride that no element needs (one head, one row) as a dense tensor has it.
ScanInput dense_where_free(ScanInput in, int64_t rows, int heads, int d) {
  if (heads == 1) in.head = d;
  if (rows == 1) in.row = static_cast<int64_t>(heads) * d;
  return in;
}

bool common_ok(const ScanCommon& s, int dk, int dv, sa_dtype dtype, float scale) {
  return s.batch >= 0 && s.batch < (int64_t{1} << 31) / 1024 && s.rows >= 0 &&
         s.rows < (int64_t{1} << 31) - 256 && s.heads >= 1 && s.heads <= 1024 && width_ok(dk) &&
         width_ok(dv) && (dtype == SA_BF16 || dtype == SA_FP32) && isfinite(scale) &&
         fabsf(scale) >= 1e-20f && fabsf(scale) <= 1e20f && s.log_decay != nullptr &&
         s.offsets != nullptr && al(s.log_decay, 4) && al(s.offsets, 8);
}

sa_status on_sm100() {
  int dev = 0, major = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess)
    return SA_ERR_CUDA;
  return major == 10 ? SA_OK : SA_ERR_UNSUPPORTED;
}

// Rows per segment, or 0 where histories stay whole, for `scans` scans of the
// batch.  In rows of one head on one SM: whole, they take their share of all
// rows or the longest history (equal histories in rounds, unequal ones end
// with the longest), whichever is more; split, the share, the states' sums
// (about half as much again), one segment and the extra launches.  Four
// segments per SM even out the segments' ends where the share is long; a
// short share is one segment, so that there are no more of them than SMs.
struct SplitRule {
  int64_t tile, least, even, launches;  // rows: chunk, shortest segment, shortest of four per
                                        // SM, the extra launches' worth
};
// Tensor cores, us: 1 history x 1500 rows, 4 heads of 128: 29 split, 55
// whole; 1 x 20000, 2 heads of 64: 34 in segments of the share, 45 in shorter
// ones.
constexpr SplitRule kSplitSimt = {64, 64, 64, 32}, kSplitTc = {128, 256, 1024, 384};

int64_t split_rows(const SplitRule& rule, int64_t batch, int64_t rows, int64_t max_rows, int heads,
                   int scans, int sms) {
  const int64_t longest = max_rows > 0 && max_rows < rows ? max_rows : rows;
  const int64_t share = rows * heads * scans / sms;
  auto tiles = [&](int64_t x) { return (x + rule.tile - 1) / rule.tile * rule.tile; };
  int64_t segment = tiles(share / 4);
  if (segment < rule.even) segment = tiles(share) < rule.even ? tiles(share) : rule.even;
  if (segment < rule.least) segment = rule.least;
  if (longest < 2 * segment) return 0;
  const int64_t waves = (batch * heads * scans + sms - 1) / sms;
  int64_t whole = share > longest ? share : longest;
  if (batch * longest <= rows + rows / 8 && waves * longest > whole) whole = waves * longest;
  return whole > share + share / 2 + segment + rule.launches ? segment : 0;
}

constexpr size_t kOrderBytes = kMostOrdered * sizeof(int32_t);

size_t up256(size_t x) { return (x + 255) / 256 * 256; }

// The states between segments, one direction.
size_t bound_bytes(int64_t rows, int64_t segment, int heads, int elems) {
  return segment == 0 ? 0 : up256(static_cast<size_t>(rows / segment) * heads * elems * 4);
}

size_t state_bytes(int64_t batch, int heads, int elems) {
  return up256(static_cast<size_t>(batch) * heads * elems * 4);
}

int device_sms() {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return 0;
  return sms;
}

// Runs n scans (n = 1: the forward; n = 3: dq, dk, dv) of one batch.  The
// workspace: header | order of the users | states between segments, forward,
// reverse | a copy of the initial states (forward scans whose final states
// replace them).
// `inputs` are q, k, v and, for the gradients, d_out.
cudaError_t run_scans(ScanPass* passes, int n, const ScanInput* inputs, const ScanCommon& s,
                      int64_t max_rows, int d_k, int d_v, bool bf16, int sms, cudaStream_t st) {
  const int elems = d_k * d_v, operands = n == 3 ? 4 : 3;
  bool tc = bf16 && s.rows > 0;
  ScanMaps maps = {};
  for (int i = 0; i < operands; ++i) tc = tc && scan_tc_usable(inputs[i]);
  for (int i = 0; tc && i < operands; ++i)
    tc = make_tmap_bf16_heads(&maps.m[i], inputs[i].p, s.rows, s.heads, i < 2 ? d_k : d_v,
                              inputs[i].row, inputs[i].head, 128);
  const int64_t segment = split_rows(tc ? kSplitTc : kSplitSimt, s.batch, s.rows, max_rows, s.heads,
                                     n, sms);
  int32_t* order = reinterpret_cast<int32_t*>(reinterpret_cast<uint8_t*>(s.header) + kWsHeaderBytes);
  uint8_t* ws = reinterpret_cast<uint8_t*>(order) + kOrderBytes;
  const size_t half = bound_bytes(s.rows, segment, s.heads, elems);
  for (int i = 0; i < n; ++i) passes[i].bound = reinterpret_cast<float*>(ws + passes[i].reverse * half);
  ScanArgs t = {};
  t.s = s;
  t.check = 1;
  t.segment = segment == 0 ? s.rows + 1 : segment;
  const int64_t slots = s.batch + (segment == 0 ? 0 : s.rows / segment);
  // The tensor-core scan's item counters live in the header, behind its flag
  // words; they are needed where an SM takes more than one item.
  unsigned long long* counter = nullptr;
  cudaError_t err = cudaSuccess;
  if (tc && slots * s.heads * n > sms) {
    counter = reinterpret_cast<unsigned long long*>(s.header) + 8;
    const int64_t longest = max_rows > 0 && max_rows < s.rows ? max_rows : s.rows;
    if (segment == 0 && s.batch <= kMostOrdered && s.batch * longest > s.rows + s.rows / 8) {
      order_kernel<<<1, kMostOrdered, 0, st>>>(s, order);
      err = cudaGetLastError();
      t.order = order;
      t.check = 0;
    } else {
      err = cudaMemsetAsync(s.header, 0, kWsHeaderBytes, st);
    }
  }
  auto launch = [&](ScanArgs& u, bool states_only, bool beside) {
    u.items = slots * s.heads * u.passes;
    if (!tc) return launch_scan_simt(u, bf16, states_only, st);
    if (counter != nullptr) u.counter = counter++;
    return launch_scan_tc(u, maps, states_only, beside, sms, st);
  };
  if (segment != 0) {
    if (n == 1 && passes[0].ends != nullptr && passes[0].ends == passes[0].fin) {
      // The last segment's final state must not meet the first one's start.
      void* copy = ws + 2 * half;
      if (err == cudaSuccess)
        err = cudaMemcpyAsync(copy, passes[0].ends, static_cast<size_t>(s.batch) * s.heads * elems * 4,
                              cudaMemcpyDeviceToDevice, st);
      passes[0].ends = static_cast<const float*>(copy);
    }
    // The states of the forward direction are sums over k and v, those of
    // the reverse one over q and d_out (dv's b and c), each stored once.
    ScanArgs u = t;
    ChainArgs chain[2] = {};
    for (int i = 0; i < n; ++i) {
      const ScanPass& p = passes[i];
      if (n == 3 && i == 1) continue;  // dk shares dv's
      ScanPass& o = u.p[u.passes++] = p;
      if (n == 3 && i == 0) {          // dq's (a, b, c) = (do, v, k)
        o.b = p.c, o.c = p.b;
        o.map_b = p.map_c, o.map_c = p.map_b;
      }
      o.da = d_k, o.dc = d_v;
      chain[p.reverse] = {p.reverse, p.ends, p.ends_mul, p.bound};
    }
    if (err == cudaSuccess) err = launch(u, true, false);
    t.check = 0;
    if (err == cudaSuccess) {
      const dim3 grid(static_cast<unsigned>(s.batch * s.heads),
                      static_cast<unsigned>((elems / 4 + 255) / 256), static_cast<unsigned>(u.passes));
      state_chain_kernel<<<grid, 256, 0, st>>>(s, segment, elems, chain[0], chain[1]);
      err = cudaGetLastError();
    }
  }
  // Scans of one shape share a launch; those of the other shape run beside it.
  for (int i = 0; i < n && err == cudaSuccess;) {
    ScanArgs u = t;
    const int da = passes[i].da, dc = passes[i].dc;
    const bool beside = i > 0;
    for (; i < n && passes[i].da == da && passes[i].dc == dc; ++i) u.p[u.passes++] = passes[i];
    err = launch(u, false, beside);
    t.check = 0;
  }
  return err;
}

}  // namespace
}  // namespace sa

extern "C" {

size_t sa_workspace_bytes_linear_attention(int heads, int d_k, int d_v, int64_t batch,
                                           int64_t total_rows, int64_t max_rows) {
  if (heads < 1 || batch < 0 || total_rows < 0 || max_rows < 0 || !sa::width_ok(d_k) ||
      !sa::width_ok(d_v))
    return 0;
  const int sms = sa::device_sms(), elems = d_k * d_v;
  if (sms == 0) return 0;
  size_t most = 0;
  for (int i = 0; i < 4; ++i) {  // either kernel, either direction
    const int scans = i < 2 ? 1 : 3;
    const int64_t seg = sa::split_rows(i % 2 == 0 ? sa::kSplitSimt : sa::kSplitTc, batch, total_rows,
                                       max_rows, heads, scans, sms);
    const size_t n = seg == 0 ? 0
                     : scans == 1 ? 2 * sa::bound_bytes(total_rows, seg, heads, elems) +
                                        sa::state_bytes(batch, heads, elems)
                                  : 2 * sa::bound_bytes(total_rows, seg, heads, elems);
    if (n > most) most = n;
  }
  return sa::kWsHeaderBytes + sa::kOrderBytes + most;
}

sa_status sa_linear_attention_forward(const void* q, int64_t q_row, int64_t q_head, const void* k,
                                      int64_t k_row, int64_t k_head, const void* v, int64_t v_row,
                                      int64_t v_head, const float* log_decay,
                                      const int64_t* offsets, int64_t batch, int64_t total_rows,
                                      int64_t max_rows, int heads, int d_k, int d_v,
                                      sa_dtype dtype, float scale, const float* initial_state,
                                      void* out, float* final_state, void* workspace,
                                      size_t workspace_bytes, void* stream) {
  const sa::ScanInput iq = {q, q_row, q_head}, ik = {k, k_row, k_head}, iv = {v, v_row, v_head};
  const sa::ScanCommon s = {log_decay, offsets, batch, total_rows, heads,
                            static_cast<sa::WsHeader*>(workspace)};
  if (!sa::common_ok(s, d_k, d_v, dtype, scale) || max_rows < 0) return SA_ERR_INVALID_ARG;
  const size_t e = dtype == SA_BF16 ? 2 : 4;
  if (!sa::input_ok(iq, heads, d_k, e) || !sa::input_ok(ik, heads, d_k, e) ||
      !sa::input_ok(iv, heads, d_v, e) || !sa::al(out, 16) || !sa::al(initial_state, 16) ||
      !sa::al(final_state, 16) || workspace == nullptr || !sa::al(workspace, 256))
    return SA_ERR_INVALID_ARG;
  if (total_rows > 0 && (q == nullptr || k == nullptr || v == nullptr || out == nullptr))
    return SA_ERR_INVALID_ARG;
  if (batch == 0) return total_rows == 0 ? SA_OK : SA_ERR_INVALID_ARG;
  const sa_status dev = sa::on_sm100();
  if (dev != SA_OK) return dev;
  if (workspace_bytes <
      sa_workspace_bytes_linear_attention(heads, d_k, d_v, batch, total_rows, max_rows))
    return SA_ERR_WORKSPACE;
  sa::ScanPass p = {};
  p.da = d_k, p.dc = d_v;
  p.ends = initial_state, p.ends_mul = 1.f;
  p.out = out, p.out_mul = scale;
  p.fin = final_state, p.fin_mul = 1.f;
  p.map_a = 0, p.map_b = 1, p.map_c = 2;
  p.parts = final_state != nullptr ? 3 : 2;
  const sa::ScanInput inputs[3] = {sa::dense_where_free(iq, total_rows, heads, d_k),
                                   sa::dense_where_free(ik, total_rows, heads, d_k),
                                   sa::dense_where_free(iv, total_rows, heads, d_v)};
  p.a = inputs[0], p.b = inputs[1], p.c = inputs[2];
  return sa::run_scans(&p, 1, inputs, s, max_rows, d_k, d_v, dtype == SA_BF16, sa::device_sms(),
                       static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? SA_OK
             : SA_ERR_CUDA;
}

sa_status sa_linear_attention_backward(const void* q, int64_t q_row, int64_t q_head, const void* k,
                                       int64_t k_row, int64_t k_head, const void* v, int64_t v_row,
                                       int64_t v_head, const float* log_decay,
                                       const int64_t* offsets, int64_t batch, int64_t total_rows,
                                       int64_t max_rows, int heads, int d_k, int d_v,
                                       sa_dtype dtype, float scale, const float* initial_state,
                                       const void* d_out, int64_t d_out_row, int64_t d_out_head,
                                       const float* d_final_state, void* dq, void* dk, void* dv,
                                       float* d_initial_state, void* workspace,
                                       size_t workspace_bytes, void* stream) {
  const sa::ScanInput iq = {q, q_row, q_head}, ik = {k, k_row, k_head}, iv = {v, v_row, v_head};
  const sa::ScanInput ig = {d_out, d_out_row, d_out_head};
  const sa::ScanCommon s = {log_decay, offsets, batch, total_rows, heads,
                            static_cast<sa::WsHeader*>(workspace)};
  if (!sa::common_ok(s, d_k, d_v, dtype, scale) || max_rows < 0) return SA_ERR_INVALID_ARG;
  const size_t e = dtype == SA_BF16 ? 2 : 4;
  if (!sa::input_ok(iq, heads, d_k, e) || !sa::input_ok(ik, heads, d_k, e) ||
      !sa::input_ok(iv, heads, d_v, e) || !sa::input_ok(ig, heads, d_v, e) || !sa::al(dq, 16) ||
      !sa::al(dk, 16) || !sa::al(dv, 16) || !sa::al(initial_state, 16) ||
      !sa::al(d_final_state, 16) || !sa::al(d_initial_state, 16) || workspace == nullptr ||
      !sa::al(workspace, 256))
    return SA_ERR_INVALID_ARG;
  if (total_rows > 0 && (q == nullptr || k == nullptr || v == nullptr || d_out == nullptr ||
                         dq == nullptr || dk == nullptr || dv == nullptr))
    return SA_ERR_INVALID_ARG;
  if (batch == 0) return total_rows == 0 ? SA_OK : SA_ERR_INVALID_ARG;
  const sa_status dev = sa::on_sm100();
  if (dev != SA_OK) return dev;
  if (workspace_bytes <
      sa_workspace_bytes_linear_attention(heads, d_k, d_v, batch, total_rows, max_rows))
    return SA_ERR_WORKSPACE;
  const float inv = 1.f / scale;
  sa::ScanPass p[3] = {};
  const sa::ScanInput inputs[4] = {sa::dense_where_free(iq, total_rows, heads, d_k),
                                   sa::dense_where_free(ik, total_rows, heads, d_k),
                                   sa::dense_where_free(iv, total_rows, heads, d_v),
                                   sa::dense_where_free(ig, total_rows, heads, d_v)};
  const int which[3][3] = {{3, 2, 1}, {2, 3, 0}, {1, 0, 3}};  // dq, dk, dv
  void* const out[3] = {dq, dk, dv};
  p[0].ends = initial_state, p[0].ends_mul = 1.f;
  p[2].fin = d_initial_state, p[2].fin_mul = scale;
  for (int i = 0; i < 3; ++i) {
    p[i].map_a = which[i][0], p[i].map_b = which[i][1], p[i].map_c = which[i][2];
    p[i].a = inputs[p[i].map_a], p[i].b = inputs[p[i].map_b], p[i].c = inputs[p[i].map_c];
    p[i].out = out[i];
    p[i].parts = p[i].fin != nullptr ? 3 : 2;
    p[i].transposed = i < 2;
    p[i].da = i < 2 ? d_v : d_k, p[i].dc = i < 2 ? d_k : d_v;
    p[i].out_mul = scale;
    if (i > 0) p[i].reverse = 1, p[i].ends = d_final_state, p[i].ends_mul = inv;
  }
  return sa::run_scans(p, 3, inputs, s, max_rows, d_k, d_v, dtype == SA_BF16, sa::device_sms(),
                       static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? SA_OK
             : SA_ERR_CUDA;
}

sa_status sa_linear_attention_step(const void* q, int64_t q_row, int64_t q_head, const void* k,
                                   int64_t k_row, int64_t k_head, const void* v, int64_t v_row,
                                   int64_t v_head, const float* log_decay, const int64_t* slots,
                                   int64_t batch, int64_t states, int heads, int d_k, int d_v,
                                   sa_dtype dtype, float scale, float* state, void* out,
                                   uint32_t* device_flags, void* stream) {
  const sa::ScanInput iq = {q, q_row, q_head}, ik = {k, k_row, k_head}, iv = {v, v_row, v_head};
  if (batch < 0 || batch >= (int64_t{1} << 31) / 1024 || states < 0 || heads < 1 || heads > 1024 ||
      d_k < 1 || d_k > sa::kStepMaxWidth || d_v < 4 || d_v > sa::kStepMaxWidth || d_v % 4 != 0 ||
      (dtype != SA_BF16 && dtype != SA_FP32) || !isfinite(scale) ||
      (slots == nullptr && states < batch))
    return SA_ERR_INVALID_ARG;
  const size_t e = dtype == SA_BF16 ? 2 : 4;
  if (!sa::input_ok(iq, heads, d_k, e) || !sa::input_ok(ik, heads, d_k, e) ||
      !sa::input_ok(iv, heads, d_v, e) || !sa::al(slots, 8) || !sa::al(log_decay, 4) ||
      !sa::al(state, 16) || !sa::al(out, e) || !sa::al(device_flags, 4))
    return SA_ERR_INVALID_ARG;
  if (batch == 0) return SA_OK;
  if (q == nullptr || k == nullptr || v == nullptr || log_decay == nullptr || out == nullptr ||
      (states > 0 && state == nullptr))
    return SA_ERR_INVALID_ARG;
  const sa_status dev = sa::on_sm100();
  if (dev != SA_OK) return dev;
  sa::StepArgs a = {iq, ik, iv, log_decay, slots, batch, states, state, out, heads, d_k, d_v, 0,
                    scale, device_flags, 0};
  // Whole state rows per block when there are two blocks for every SM (of
  // 148); else 32 columns per block, which gives up to eight times as many.
  const int all4 = d_v / 4;
  a.cols4 = batch * heads >= 296 ? all4 : all4 < 8 ? all4 : 8;
  const dim3 grid(static_cast<unsigned>(batch * heads), static_cast<unsigned>((all4 + a.cols4 - 1) / a.cols4));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  // Marks need an output of their own (and whole rows per block: one a head).
  const size_t out_bytes = static_cast<size_t>(batch) * heads * d_v * e;
  if (slots != nullptr && batch * heads > sa::kMostComparing &&
      !sa::may_meet(iq, batch, heads, d_k, e, out, out_bytes) &&
      !sa::may_meet(ik, batch, heads, d_k, e, out, out_bytes) &&
      !sa::may_meet(iv, batch, heads, d_v, e, out, out_bytes)) {
    a.marked = 1;
    const unsigned blocks = static_cast<unsigned>((batch + 31) / 32);
    if (dtype == SA_BF16) sa::mark_kernel<uint16_t><<<blocks, 256, 0, st>>>(a);
    else sa::mark_kernel<float><<<blocks, 256, 0, st>>>(a);
    if (cudaGetLastError() != cudaSuccess) return SA_ERR_CUDA;
  }
  if (dtype == SA_BF16) sa::step_kernel<uint16_t><<<grid, sa::kStepThreads, 0, st>>>(a);
  else sa::step_kernel<float><<<grid, sa::kStepThreads, 0, st>>>(a);
  return cudaGetLastError() == cudaSuccess ? SA_OK : SA_ERR_CUDA;
}

}  // extern "C"
