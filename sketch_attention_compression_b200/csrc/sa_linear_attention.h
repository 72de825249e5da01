// Linear attention with a decay per head: what its kernels share.
//
// Every direction is one scan over a user's rows.  With l = exp(log_decay):
//
//   forward scan   out_i = mul * sum_{j <= i} l^(i-j) (a_i . b_j) c_j  + end term
//   reverse scan   out_i = mul * sum_{j >= i} l^(j-i) (a_i . b_j) c_j  + end term
//
// carried by the state S (da x dc), the decayed sum of b_j c_j^T:
//
//   S <- l S + b_i c_i^T;  out_i = mul S^T a_i        (in scan order)
//
// and the gradients of the forward (a, b, c) = (q, k, v) are scans too:
//
//   dq: forward scan of (do, v, k), started from S_0^T
//   dk: reverse scan of (v, do, q), started from (dS_n / mul)^T
//   dv: reverse scan of (k, q, do), started from  dS_n / mul
//   dS_0 = mul l S behind dv's last row (dS_n itself for a user without rows)
//
// A forward scan decays its start before the first row's product is added; a
// reverse scan starts with the gradient of the state behind the last row, so
// its first row adds to the undecayed start, and its result is decayed once
// more.
//
// The kernels walk chunks of rows.  With L the rows of a chunk and r a row's
// place in scan order (forward: its index i; reverse: L - 1 - i):
//
//   P   = a b^T weighted by l^(distance), 0 where the scan has not yet been
//   out = mul (P c + l^(r+1) a S)
//   S  <- l^L S + sum_j l^(L-1-r_j) b_j c_j^T
//
// Every decay factor is a power with an exponent >= 0, so none overflows.
// The powers are taken in 64 bits and rounded once; l^L of a whole chunk is
// kept with its rounding error, which would else add up over a long history.
//
// Few and long histories are split along the rows into segments, so that
// every SM has work: a first launch sums each segment's own state from b and
// c alone, a second carries the states from segment to segment, and the scan
// starts each segment from its own.
#pragma once

#include <atomic>

#include "sa_internal.h"

namespace sa {

struct ScanInput {
  const void* p;
  int64_t row, head;  // strides in elements
};

struct ScanPass {
  ScanInput a, b, c;     // [N][H][da], [N][H][da], [N][H][dc]
  int da, dc;
  int reverse;
  int transposed;        // start states are stored [dc][da]
  const float* ends;     // start states [B][H][..], may be null
  float ends_mul;
  float* bound;          // states between segments [..][H][..], already scaled
  void* out;             // [N][H][dc]
  float out_mul;
  float* fin;            // [B][H][da][dc], may be null
  float fin_mul;
  int map_a, map_b, map_c;  // tensor maps (tensor-core scan)
  int parts;             // bf16 parts of the weighted b (tensor-core scan)
};

struct ScanCommon {
  const float* log_decay;  // [H]
  const int64_t* offsets;  // [B + 1]
  int64_t batch, rows;
  int heads;
  WsHeader* header;
};

struct ScanArgs {
  ScanCommon s;
  ScanPass p[3];           // of one shape
  int passes;
  int check;               // this launch checks offsets and decays
  int64_t segment;         // rows per segment (> rows where nothing is split)
  int64_t items;           // segment slots * heads * passes
  unsigned long long* counter;  // next item (tensor-core scan), or null: every grid-th item
  const int32_t* order;    // users by length, longest first, or null: as they come (whole histories)
};

// One scan of one segment of a user's rows for one head.
struct ScanItem {
  int64_t lo, hi;          // rows
  int64_t state;           // user * heads + head
  int64_t from, to;        // boundary states to start from and to write, -1: none
  int32_t head, pass;
  int32_t first, last;     // the user's first (last) segment in scan order
};

// log_decay as the kernels use it: [-1e4, 0] (exp(-1e4) is 0, and -1e4
// times a distance of 0 is 0, which -inf would not be).
__device__ __forceinline__ float usable_decay(float g) { return fminf(fmaxf(g, -1e4f), 0.f); }

// The rows of user b, inside [0, rows] whatever the offsets hold.
__device__ __forceinline__ void user_rows(const ScanCommon& s, int64_t b, int64_t& lo, int64_t& hi) {
  lo = s.offsets[b];
  hi = s.offsets[b + 1];
  lo = lo < 0 ? 0 : lo > s.rows ? s.rows : lo;
  hi = hi < lo ? lo : hi > s.rows ? s.rows : hi;
}

// Segment slots: user b's segment i has slot floor(off_b / segment) + b + i,
// which leaves room for ceil(n_b / segment) (at least one) segments of every
// user without a prefix sum.  Boundary state j (behind segment j) of user b
// has index floor(off_b / segment) + j.
__device__ __forceinline__ int64_t slot_base(const ScanCommon& s, int64_t segment, int64_t b) {
  int64_t o = s.offsets[b];
  o = o < 0 ? 0 : o > s.rows ? s.rows : o;
  return o / segment + b;
}

// Fills `it` with item `x` (called by whole warps with one x); false if the
// slot holds nothing to do (states_only: a user's last segment either).
__device__ __forceinline__ bool item_of(const ScanArgs& t, int64_t x, int lane, bool states_only,
                                        ScanItem& it) {
  const int pass = static_cast<int>(x % t.passes);
  x /= t.passes;
  const int head = static_cast<int>(x % t.s.heads);
  const int64_t slot = x / t.s.heads;
  const bool whole = t.segment > t.s.rows;
  int64_t b = 0, base = slot;
  if (whole) {
    b = slot < t.s.batch ? slot : t.s.batch - 1;
    if (t.order != nullptr) b = t.order[b];
    base = slot;
  } else {
    // Largest b with slot_base(b) <= slot: a 32-way search.
    int64_t hi = t.s.batch - 1;
    while (b < hi) {
      const int64_t step = (hi - b + 32) / 32;
      const int64_t c = b + lane * step;
      const uint32_t m = __ballot_sync(0xFFFFFFFFu, c <= hi && slot_base(t.s, t.segment, c) <= slot);
      const int64_t next = b + (m ? 31 - __clz(static_cast<int>(m)) : 0) * step;
      hi = next + step - 1 < hi ? next + step - 1 : hi;
      b = next;
    }
    base = slot_base(t.s, t.segment, b);
  }
  const int64_t i = slot - base;
  int64_t r0, r1;
  user_rows(t.s, b, r0, r1);
  const int64_t n = r1 - r0;
  const int64_t count = n > 0 ? (n + t.segment - 1) / t.segment : 1;
  if (i < 0 || i >= count) return false;
  const bool rev = t.p[pass].reverse != 0;
  it.lo = r0 + i * t.segment;
  it.hi = it.lo + t.segment < r1 ? it.lo + t.segment : r1;
  it.state = b * t.s.heads + head;
  it.head = head;
  it.pass = pass;
  it.first = rev ? i == count - 1 : i == 0;
  it.last = rev ? i == 0 : i == count - 1;
  const int64_t bound = base - b;  // (unused where nothing is split)
  it.from = it.first ? -1 : (bound + (rev ? i : i - 1)) * t.s.heads + head;
  it.to = it.last ? -1 : (bound + (rev ? i - 1 : i)) * t.s.heads + head;
  return !states_only || !it.last;
}

// Checks the offsets and decays with one block and stores the header's flag
// word; the timeout word is cleared.
__device__ __forceinline__ void check_inputs(const ScanCommon& s, uint32_t* shared_flags) {
  if (threadIdx.x == 0) *shared_flags = 0u;
  __syncthreads();
  uint32_t f = 0;
  for (int64_t b = threadIdx.x; b < s.batch; b += blockDim.x)
    if (s.offsets[b] > s.offsets[b + 1]) f |= SA_DEVFLAG_OFFSETS_DECREASE;
  for (int h = threadIdx.x; h < s.heads; h += blockDim.x)
    if (!(s.log_decay[h] <= 0.f)) f |= SA_DEVFLAG_DECAY;
  if (threadIdx.x == 0) {
    if (s.offsets[0] != 0) f |= SA_DEVFLAG_OFFSET0_NONZERO;
    if (s.offsets[s.batch] > s.rows) f |= SA_DEVFLAG_OFFSET_LAST;
  }
  if (f != 0) atomicOr(shared_flags, f);
  __syncthreads();
  if (threadIdx.x == 0) {
    s.header->flags = *shared_flags;
    s.header->timeout_flags = 0u;
  }
}

// Lets `kernel` use `bytes` of shared memory on the current device; asked of
// the runtime once per device (`done`: a bit per device).
template <class K>
cudaError_t allow_smem(K kernel, int bytes, std::atomic<uint64_t>& done) {
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  const uint64_t bit = dev < 64 ? uint64_t{1} << dev : 0;
  if ((done.load(std::memory_order_relaxed) & bit) != 0) return cudaSuccess;
  err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (err == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
  return err;
}

// Launches one scan (or, with states_only, the sums of its segments' states,
// written to p[].bound) on the CUDA cores (sa_linear_attention_simt.cu).
cudaError_t launch_scan_simt(const ScanArgs& t, bool bf16, bool states_only, cudaStream_t st);

// The same on the tensor cores (sa_linear_attention_tc.cu), bf16 inputs whose
// tensor maps the passes name.  `beside`: the launch reads nothing that the
// one before it writes and may run beside it.
struct ScanMaps {
  CUtensorMap m[4];
};
cudaError_t launch_scan_tc(const ScanArgs& t, const ScanMaps& maps, bool states_only, bool beside,
                           int sms, cudaStream_t st);
bool scan_tc_usable(const ScanInput& in);  // addresses and strides that TMA takes

}  // namespace sa
