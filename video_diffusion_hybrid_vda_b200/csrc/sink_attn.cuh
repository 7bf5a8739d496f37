// Shared by the sink-window attention kernels: the mask, the packed sequences
// and the tiles they are cut into.
//
// A query of a sequence with n_q queries and n_k keys, local row i, has the
// position p = i + n_k - n_q (the last query stands at the last key).  It
// sees key j iff
//     j <= p + ahead  and  (p - j < window  or  j < sinks).
// p is negative for queries that stand before the first key; with
// p + ahead < 0 a query sees nothing.
#pragma once

#include <cuda.h>
#include <stdint.h>

#include "common.cuh"
#include "ptx.cuh"

namespace vdn {

// Everything is int32: lengths are below 2^30 and window, ahead and sinks are
// clamped to 2^30 - 1 on the host, so p + ahead and p - window stay in range.
constexpr int kSinkMax = (1 << 30) - 1;

struct SinkMask {
  int window, ahead, sinks;
};

struct SinkDims {
  int Lq, Lk, B, H, Hkv;
  const int32_t* cu_q;  // [B + 1] first row of each sequence, or null: one sequence
  const int32_t* cu_k;
  SinkMask m;
};

struct SinkSeq {
  int q0, q1, k0, k1;  // rows
  __device__ int nq() const { return q1 - q0; }
  __device__ int nk() const { return k1 - k0; }
  __device__ int shift() const { return nk() - nq(); }  // position of local query 0
};

// Boundary b of the packed rows, kept inside [0, L] whatever the array holds.
__device__ __forceinline__ int sink_bound(const int32_t* cu, int b, int L) {
  const int v = __ldg(cu + b);
  return v < 0 ? 0 : v > L ? L : v;
}

__device__ __forceinline__ SinkSeq sink_seq(const SinkDims& s, int b) {
  SinkSeq r{0, s.Lq, 0, s.Lk};
  if (s.cu_q != nullptr) {
    r.q0 = sink_bound(s.cu_q, b, s.Lq);
    r.q1 = max(r.q0, sink_bound(s.cu_q, b + 1, s.Lq));
  }
  if (s.cu_k != nullptr) {
    r.k0 = sink_bound(s.cu_k, b, s.Lk);
    r.k1 = max(r.k0, sink_bound(s.cu_k, b + 1, s.Lk));
  }
  return r;
}

// Tiles of packed sequences without a prefix sum over them: sequence b owns
// the slots from cu[b] / tile + b on.  That is at least as many as it has
// tiles (floor((c + n) / t) - floor(c / t) + 1 >= ceil(n / t)), so the grid
// is L / tile + B slots, and a slot finds its sequence by bisection over cu.
// Slots past a sequence's tiles have nothing to do, nor have those below the
// first sequence's (a tile of rows or more before it): their tile is negative.
__host__ __device__ __forceinline__ int sink_slots(int L, int B, int tile) {
  return L / tile + B;
}

__device__ __forceinline__ int sink_slot_base(const int32_t* cu, int b, int L, int tile) {
  return cu == nullptr ? 0 : sink_bound(cu, b, L) / tile + b;
}

__device__ __forceinline__ int sink_slot_seq(const int32_t* cu, int B, int L, int tile, int slot) {
  int lo = 0, hi = B;  // base(lo) <= slot < base(hi)
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (sink_slot_base(cu, mid, L, tile) <= slot)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

// The keys that queries at positions [pa, pb] see between them, cut into
// tiles of 128: the sinks' tiles [0, s_end) and then the window's [w_lo, hi),
// or one run [0, hi) where they meet.
struct SinkKeyTiles {
  int s_end, w_lo, hi, n_sink, n;
  __device__ void init(const SinkMask& m, int pa, int pb, int nk) {
    hi = min(nk, pb + m.ahead + 1);
    s_end = w_lo = n_sink = n = 0;
    if (pb < pa || hi <= 0) return;
    s_end = min(m.sinks, hi);
    w_lo = max(0, pa - m.window + 1);
    if (w_lo <= s_end) {
      s_end = w_lo = 0;
    } else {
      n_sink = (s_end + 127) / 128;
    }
    n = n_sink + (hi - w_lo + 127) / 128;
  }
  __device__ int start(int j) const { return j < n_sink ? 128 * j : w_lo + 128 * (j - n_sink); }
  __device__ int valid(int j) const {
    return min(128, (j < n_sink ? s_end : hi) - start(j));
  }
};

// Does any query at [pa, pb] see any key of [ks, ke]?
__device__ __forceinline__ bool sink_touches(const SinkMask& m, int pa, int pb, int ks, int ke) {
  return pa <= pb && ks <= ke && ks <= pb + m.ahead && (ke > pa - m.window || ks < m.sinks);
}

// Does every query at [pa, pb] see every key of [ks, ke]?
__device__ __forceinline__ bool sink_sees_all(const SinkMask& m, int pa, int pb, int ks, int ke) {
  return ke <= pa + m.ahead && (ks > pb - m.window || ke < m.sinks);
}

// Visibility of 32 consecutive columns as bits: the columns [lo, hi) and those
// below `sink` (bounds relative to the first of the 32).  A tile that crosses
// the mask's edge then pays one bit test and one select an element.
__device__ __forceinline__ uint32_t bits_below(int n) {
  return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u;
}

__device__ __forceinline__ uint32_t sink_bits(int lo, int hi, int sink) {
  return bits_below(hi) & (~bits_below(lo) | bits_below(sink));
}

// Rows of no sequence: before the first boundary and from the last one on.
// Zeroed by all threads of the grid together (row r by block r mod grid).
__device__ __forceinline__ void sink_zero_rest(const int32_t* cu, int B, int L, void* base,
                                               int64_t ld, int cols) {
  const int head = sink_bound(cu, 0, L), tail = max(head, sink_bound(cu, B, L));
  const int rest = head + L - tail;
  for (int64_t i = blockIdx.x; i < rest; i += gridDim.x) {
    const int64_t r = i < head ? i : tail + (i - head);
    uint4* row = reinterpret_cast<uint4*>(static_cast<uint8_t*>(base) + r * ld * 2);
    for (int c = threadIdx.x; c < cols / 8; c += blockDim.x) row[c] = make_uint4(0, 0, 0, 0);
  }
}

// Zero rows [from, 128) of a tile of `slabs` 64-column slabs (128 rows x 128
// swizzled bytes each): the whole warp.  Zeroing whole rows needs no swizzle.
// The rows belong to another sequence or lie past the last one; as the
// right-hand operand of a product their weight is 0, but 0 x NaN is not.
__device__ __forceinline__ void sink_zero_rows(uint8_t* tile, int slabs, int from) {
  const uint4 z = make_uint4(0, 0, 0, 0);
  for (int s = 0; s < slabs; ++s)
    for (int i = from * 8 + lane_id(); i < 1024; i += 32)
      *reinterpret_cast<uint4*>(tile + s * 16384 + i * 16) = z;
  fence_proxy_async_smem();
  __syncwarp();
}

}  // namespace vdn
