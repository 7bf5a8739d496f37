// Gradients of attention with a sliding window and sinks (sink_attn.cu).
//
// With P_ij = exp(scale q_i . k_j - lse_i) over the visible keys and
// D_i = dO_i . o_i:
//   dV_j = sum_i P_ij dO_i
//   dS_ij = P_ij (dO_i . v_j - D_i)
//   dQ_i = scale sum_j dS_ij k_j,   dK_j = scale sum_i dS_ij q_i
// A query that saw nothing (lse = -inf) contributes nothing and gets dQ = 0.
//
// P is formed anew from q, k and lse.  Two passes, so that every sum has a
// fixed order (the same call gives the same bits): the key pass holds dK and
// dV of 128 keys of one key head and walks the queries of all its query heads;
// the query pass holds dQ of 128 queries.  That is seven products a pair of
// tiles where one pass with atomic adds into dQ would take five.  P and dS are
// rounded to bf16 for their products, sums stay fp32 in TMEM.
//
// Key tiles differ in work: a sink is seen by every later query, other keys by
// `window` of them, keys near a sequence's end by few.  The key pass therefore
// deals out its items (a key tile with one query tile of one head) rather
// than its tiles: every CTA takes the same number of consecutive items, and
// where a tile's items end up with several CTAs each writes its fp32 part
// and sink_join_kernel adds them in order.
#include <cuda_bf16.h>
#include <math.h>

#include "exp2_fma.cuh"
#include "sink_attn.cuh"

namespace vdn {

vdn_status sink_check(const vdn_sink_shape* shape, const void* q, int64_t ld_q, const void* k,
                      const void* v, int64_t ld_kv, const int32_t* cu_q, const int32_t* cu_k,
                      vdn_sink_shape* s);

namespace {

// Four softmax warpgroups, 32 columns of a 128 x 128 tile each: with one row a
// thread that is 32 scores and 32 products in registers, and four warps a
// scheduler to hide the tensor-memory round trips behind.  (Two warpgroups
// with 64 columns: key pass 3800 cycles an item, the tensor pipe 45 % busy.)
constexpr int kGroups = 4;
constexpr int kThreads = 128 + kGroups * 128;
constexpr int kCtas = 148;   // key pass CTAs at most: one an SM

template <int DH>
struct GradCfg {
  static constexpr int SLABS = DH / 64;
  static constexpr int TILE = SLABS * 128 * 128;  // 128 rows x DH bf16
  static constexpr int STAGES = 2;
  static constexpr int STATS = 2 * 128 * 4;       // -lse log2 e and D of 128 queries
  // two resident tiles, a ring of two-tile stages, statistics, barriers
  static constexpr int SMEM = 1024 + 2 * TILE + STAGES * (2 * TILE + STATS) + 512;
};

// Per query, in tiles of 128 (the slots of sink_attn.cuh): -lse log2 e and
// -D.  Rows past the sequence's end get -inf and 0: P = 0 there.
// D = dO . o where a query sees many keys.  o is rounded, and made from a
// rounded P, which puts D off by the same amount for all of a query's keys;
// among few keys that weighs as much as all other roundings (2 keys: dq off by
// 0.0042 of its norm in place of 0.0023; a window of 24: 0.0026, causal
// sequences of up to some 500 tokens through their first queries alone: 0.0027
// to 0.0026).  Groups of 16 queries whose first or last sees at most kFewKeys
// keys therefore get D = sum_j P_ij (dO_i . v_j) from sink_few_kernel.
// Rows of dq, dk and dv of no sequence are zeroed where asked.
// A warp takes 32 rows of a head, DH / 8 lanes a row, so that lse is read and
// both statistics are written 128 bytes at a time; the other heads' warps of
// the block read the rest of the same rows.  Reading o and dO once is the whole
// cost (a thread's rows in heads order, 4-byte accesses to [head][row] arrays:
// 19.5 us for 8097 x 16 x 128, now 14.3).
constexpr int kFewKeys = 64;
constexpr int kFewRows = 16;  // the rows of a warp's MMA
constexpr int kFewWarps = 4;  // that share a group and head's keys

struct StatsArgs {
  const __nv_bfloat16* q;
  const __nv_bfloat16* k;
  const __nv_bfloat16* v;
  const __nv_bfloat16* o;
  const __nv_bfloat16* d_o;
  int64_t ld_q, ld_kv, ld_o, ld_do;
  float scale_log2;
  int few_blocks, few_stride;  // see sink_few_kernel
  const float* lse;
  float* nlse2;
  float* ndelta;
  void* zero[3];       // dq, dk, dv or null
  int64_t ld_zero[3];
  struct SinkPlan* plan;
  struct SlotRec* rec;
  int64_t* before;
  int ctas;            // at most
  bool whole;          // a unit a CTA
};

// How the key pass's items are dealt out, written by one block of the
// statistics launch.  Slot s (a key tile of a sequence) weighs its items of a
// key head and kUnitCost more (loading the tile and storing its sums takes
// about as long as that many items: 10 units and 56 items took 198 us where 1
// and 56 took 136).  The unit (s, hk) covers [Hkv before[s] + hk weight[s], ...)
// of `total`, its cost first, then its items; CTA c of `ctas` takes
// [first[c], first[c + 1]), about total / ctas each, moved back to the unit's
// begin where it would fall inside a unit's cost or before its first item; or,
// for few and short units, one unit each (`whole`).
constexpr int kUnitCost = 3;

struct SlotRec {
  int b, tile;     // sequence and its key tile
  int t0, tiles;   // query tiles (of 128) that see it
};

struct SinkPlan {
  int64_t total;
  int ctas;
  int start[kCtas];          // slot of each CTA's first item
  int64_t first[kCtas + 1];
  SlotRec* rec;        // [slots]
  int64_t* before;     // [slots + 1]
};

__device__ __forceinline__ SlotRec key_slot(const SinkDims& s, int slot) {
  SlotRec r{0, -1, 0, 0};
  r.b = sink_slot_seq(s.cu_k, s.B, s.Lk, 128, slot);
  const int tile = slot - sink_slot_base(s.cu_k, r.b, s.Lk, 128);
  const SinkSeq seq = sink_seq(s, r.b);
  const int ks = 128 * tile, nq = seq.nq(), shift = seq.shift();
  if (tile < 0 || ks >= seq.nk()) return r;  // a slot without a tile
  const int ke = min(ks + 127, seq.nk() - 1);
  // queries [lo, hi) see a key of the tile
  const int lo = max(0, ks - shift - s.m.ahead);
  const int hi = ks < s.m.sinks ? nq : min(nq, ke - shift + s.m.window);
  r.tile = tile;
  r.t0 = lo / 128;
  r.tiles = hi > lo ? (hi + 127) / 128 - r.t0 : 0;
  return r;
}

// One block: the slots' records, their prefix sums and each CTA's first slot.
__device__ void make_plan(const SinkDims& s, const StatsArgs& a) {
  SinkPlan* p = a.plan;
  __shared__ int64_t warp_sum[8];
  __shared__ int64_t carry;
  const int slots = sink_slots(s.Lk, s.B, 128), group = s.H / s.Hkv;
  const int lane = lane_id(), warp = warp_id();
  if (threadIdx.x == 0) carry = 0;
  __syncthreads();
  for (int base = 0; base < slots; base += 256) {
    const int slot = base + threadIdx.x;
    SlotRec r{0, -1, 0, 0};
    if (slot < slots) {
      r = key_slot(s, slot);
      a.rec[slot] = r;
    }
    const int64_t w = r.tile < 0 ? 0 : r.tiles * group + kUnitCost;
    int64_t x = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) warp_sum[warp] = x;
    __syncthreads();
    int64_t off = carry;
    for (int i = 0; i < warp; ++i) off += warp_sum[i];
    if (slot < slots) a.before[slot] = off + x - w;
    __syncthreads();
    if (threadIdx.x == 255) carry = off + x;
    __syncthreads();
  }
  const int64_t total = carry * s.Hkv;
  if (threadIdx.x == 0) a.before[slots] = carry;
  // twice a unit's cost a CTA at least
  int64_t n = total / (2 * kUnitCost);
  n = n < 1 ? 1 : n > a.ctas || a.whole ? a.ctas : n;
  if (threadIdx.x == 0) {
    p->total = total;
    p->ctas = static_cast<int>(n);
    p->rec = a.rec;
    p->before = a.before;
    p->first[n] = total;
  }
  __syncthreads();
  for (int c = threadIdx.x; c < n; c += 256) {
    if (a.whole) {
      const int slot = c / s.Hkv;
      p->start[c] = slot;
      p->first[c] = a.before[slot] * s.Hkv + c % s.Hkv * (a.before[slot + 1] - a.before[slot]);
      continue;
    }
    int64_t x = total / n * c + total % n * c / n;
    // the last slot that begins at or before x: empty ones begin where the
    // next begins
    int lo = 0, hi = slots;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (a.before[mid] * s.Hkv <= x)
        lo = mid;
      else
        hi = mid;
    }
    const int64_t begin = a.before[lo] * s.Hkv, weight = a.before[lo + 1] - a.before[lo];
    const int64_t in = weight > 0 ? (x - begin) % weight : 0;
    if (in <= kUnitCost) x -= in;
    p->start[c] = lo;
    p->first[c] = x;
  }
}

// Keys that position p sees.
__device__ __forceinline__ int sink_count(const SinkMask& m, int nk, int p) {
  const int hi = min(nk, p + m.ahead + 1);
  if (hi <= 0) return 0;
  const int lo = max(0, p - m.window + 1), s = min(m.sinks, hi);
  return lo <= s ? hi : hi - lo + s;
}

// Do the queries [row, row + kFewRows) of a sequence (row < nq) see few keys?
__device__ __forceinline__ bool sink_few(const SinkMask& m, const SinkSeq& seq, int row) {
  const int p0 = row + seq.shift(), p1 = min(row + kFewRows, seq.nq()) - 1 + seq.shift();
  return min(sink_count(m, seq.nk(), p0), sink_count(m, seq.nk(), p1)) <= kFewKeys;
}

// D = sum_j P_ij (dO_i . v_j) of 16 queries and one head, over every
// kFewWarps-th eight keys from the `part`-th on: S and dP by a warp's MMAs,
// operands straight from memory (they are few).  Returns D of rows g and g + 8
// in each quad g.
template <int DH>
__device__ __forceinline__ float2 sink_few_rows(const SinkDims& s, const StatsArgs& a,
                                                const SinkSeq& seq, int row, int h, int part) {
  const int lane = lane_id(), g = lane >> 2, c2 = 2 * (lane & 3), hk = h / (s.H / s.Hkv);
  const int rows = min(kFewRows, seq.nq() - row), pa = row + seq.shift(), nk = seq.nk();
  const __nv_bfloat16* q = a.q + static_cast<int64_t>(seq.q0 + row) * a.ld_q + h * DH + c2;
  const __nv_bfloat16* w = a.d_o + static_cast<int64_t>(seq.q0 + row) * a.ld_do + h * DH + c2;
  uint32_t qf[DH / 16][4], wf[DH / 16][4];
#pragma unroll
  for (int kk = 0; kk < DH / 16; ++kk)
#pragma unroll
    for (int f = 0; f < 4; ++f) {
      const int r = g + 8 * (f & 1), col = 16 * kk + 8 * (f >> 1);
      const bool on = r < rows;
      qf[kk][f] = on ? *reinterpret_cast<const uint32_t*>(q + r * a.ld_q + col) : 0u;
      wf[kk][f] = on ? *reinterpret_cast<const uint32_t*>(w + r * a.ld_do + col) : 0u;
    }
  float nl[2], d[2] = {0.f, 0.f};  // of rows g and g + 8
#pragma unroll
  for (int i = 0; i < 2; ++i)
    nl[i] = g + 8 * i < rows ? a.lse[static_cast<int64_t>(h) * s.Lq + seq.q0 + row + g + 8 * i]
                             : -INFINITY;
#pragma unroll
  for (int i = 0; i < 2; ++i) nl[i] = nl[i] == -INFINITY ? -INFINITY : -nl[i] * 1.4426950408889634f;
  SinkKeyTiles kt;
  kt.init(s.m, pa, pa + rows - 1, nk);
  const int n_sink = (kt.s_end + 7) / 8;  // eights of the sinks, then of the window
  const int n = kt.n > 0 ? n_sink + (kt.hi - kt.w_lo + 7) / 8 : 0;
  for (int t = part; t < n; t += kFewWarps) {
    const int j0 = t < n_sink ? 8 * t : kt.w_lo + 8 * (t - n_sink);
    const int end = t < n_sink ? kt.s_end : kt.hi;
    const bool on = j0 + g < end;
    const int64_t off = static_cast<int64_t>(seq.k0 + j0 + g) * a.ld_kv + hk * DH + c2;
    uint32_t kf[DH / 16][2], vf[DH / 16][2];
#pragma unroll
    for (int kk = 0; kk < DH / 16; ++kk)
#pragma unroll
      for (int f = 0; f < 2; ++f) {
        const int64_t at = off + 16 * kk + 8 * f;
        kf[kk][f] = on ? *reinterpret_cast<const uint32_t*>(a.k + at) : 0u;
        vf[kk][f] = on ? *reinterpret_cast<const uint32_t*>(a.v + at) : 0u;
      }
    float sc[4] = {}, dp[4] = {};
#pragma unroll
    for (int kk = 0; kk < DH / 16; ++kk) {
      mma16816(sc, qf[kk], kf[kk][0], kf[kk][1]);
      mma16816(dp, wf[kk], vf[kk][0], vf[kk][1]);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int j = j0 + c2 + (e & 1), p = pa + g + 8 * (e >> 1);
      const bool see = j < end && j <= p + s.m.ahead && (p - j < s.m.window || j < s.m.sinks);
      if (see) d[e >> 1] += exp2_mufu(sc[e] * a.scale_log2 + nl[e >> 1]) * dp[e];
    }
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    d[i] += __shfl_xor_sync(0xffffffffu, d[i], 1);
    d[i] += __shfl_xor_sync(0xffffffffu, d[i], 2);
    if (nl[i] == -INFINITY) d[i] = 0.f;
  }
  return make_float2(d[0], d[1]);
}

// D of the groups with few keys, over the statistics kernel's: kFewWarps warps
// a head, a block every few_stride-th group of a sequence.  With a window of
// more than kFewKeys these are the groups that begin with a query whose look
// ahead ends among the first kFewKeys keys, and all of a sequence of so few
// keys.  Bound: the latency of a few dependent loads (8097 tokens in three
// causal sequences, 16 heads of 128: 240 groups and heads, 8.5 us more in all;
// as blocks of the statistics kernel, which then has more registers, 10 to 18).
template <int DH>
__global__ void __launch_bounds__(256, 2) sink_few_kernel(const SinkDims s, const StatsArgs a) {
  after_allow();  // sink_grad_kernel
  bool alone = false;  // the statistics kernel, whose D is overwritten, has ended
  constexpr int HEADS = 8 / kFewWarps;
  __shared__ float sums[8][kFewRows];
  const int warp = warp_id(), lane = lane_id(), blocks = (s.H + HEADS - 1) / HEADS;
  const int each = blocks * a.few_stride, slots = sink_slots(s.Lq, s.B, 128);
  for (int64_t n = blockIdx.x; n < static_cast<int64_t>(s.B) * each; n += gridDim.x) {
    const int b = static_cast<int>(n / each), i = static_cast<int>(n % each);
    const int h = i % blocks * HEADS + warp / kFewWarps;
    const SinkSeq seq = sink_seq(s, b);
    const int end = s.m.window <= kFewKeys || seq.nk() <= kFewKeys
                        ? seq.nq()
                        : min(seq.nq(), kFewKeys - s.m.ahead - seq.shift());
    for (int row = i / blocks * kFewRows; row < end; row += a.few_stride * kFewRows) {
      if (!sink_few(s.m, seq, row)) continue;  // the whole block
      if (h < s.H) {
        const float2 d = sink_few_rows<DH>(s, a, seq, row, h, warp % kFewWarps);
        if ((lane & 3) == 0) sums[warp][lane >> 2] = d.x, sums[warp][8 + (lane >> 2)] = d.y;
      }
      if (!alone) after_wait();
      alone = true;
      __syncthreads();
      if (h < s.H && warp % kFewWarps == 0 && lane < kFewRows && row + lane < seq.nq()) {
        const int64_t slot = sink_slot_base(s.cu_q, b, s.Lq, 128) + (row >> 7);
        float d = 0.f;
#pragma unroll
        for (int w = 0; w < kFewWarps; ++w) d += sums[warp + w][lane];
        a.ndelta[(h * static_cast<int64_t>(slots) + slot) * 128 + (row & 127) + lane] = -d;
      }
      __syncthreads();
    }
  }
  if (!alone) after_wait();
}

template <int DH>
__global__ void __launch_bounds__(256) sink_stats_kernel(const SinkDims dims, const StatsArgs a) {
  after_allow();  // sink_few_kernel
  constexpr int LANES = DH / 8, ROWS = 32 / LANES;  // rows a warp loads at once
  constexpr int U = 8;                              // loads in flight
  // a side without offsets has no rows outside its one sequence
  if (dims.cu_q != nullptr && a.zero[0] != nullptr)
    sink_zero_rest(dims.cu_q, dims.B, dims.Lq, a.zero[0], a.ld_zero[0], dims.H * DH);
  if (dims.cu_k != nullptr)
    for (int i = 1; i < 3; ++i)
      if (a.zero[i] != nullptr)
        sink_zero_rest(dims.cu_k, dims.B, dims.Lk, a.zero[i], a.ld_zero[i], dims.Hkv * DH);
  if (blockIdx.x == 0) {  // the other blocks have more to do
    make_plan(dims, a);
    return;
  }
  const int slots = sink_slots(dims.Lq, dims.B, 128);
  const int blk = blockIdx.x - 1;
  const int slot = blk >> 2, first = (blk & 3) * 32;
  const int b = sink_slot_seq(dims.cu_q, dims.B, dims.Lq, 128, slot);
  const SinkSeq seq = sink_seq(dims, b);
  const int tile0 = seq.q0 + 128 * (slot - sink_slot_base(dims.cu_q, b, dims.Lq, 128));
  if (tile0 < seq.q0 || tile0 >= seq.q1) return;
  const int lane = lane_id(), sub = lane / LANES, col = lane % LANES * 8;
  const int r0 = tile0 + first;
  for (int h = warp_id(); h < dims.H; h += 8) {
    const bool on = r0 + lane < seq.q1;
    const float v = on ? a.lse[static_cast<int64_t>(h) * dims.Lq + r0 + lane] : -INFINITY;
    float mine = 0.f;  // D of row `lane`
#pragma unroll
    for (int i0 = 0; i0 < 32; i0 += U * ROWS) {
      uint4 x[U], y[U];
#pragma unroll
      for (int n = 0; n < U; ++n) {
        const int64_t r = r0 + i0 + n * ROWS + sub;
        x[n] = y[n] = make_uint4(0, 0, 0, 0);
        if (r < seq.q1) {
          x[n] = *reinterpret_cast<const uint4*>(a.o + r * a.ld_o + h * DH + col);
          y[n] = *reinterpret_cast<const uint4*>(a.d_o + r * a.ld_do + h * DH + col);
        }
      }
#pragma unroll
      for (int n = 0; n < U; ++n) {
        const uint32_t xs[4] = {x[n].x, x[n].y, x[n].z, x[n].w};
        const uint32_t ys[4] = {y[n].x, y[n].y, y[n].z, y[n].w};
        float t = 0.f;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 f = unpack_bf16x2(xs[e]), g = unpack_bf16x2(ys[e]);
          t += f.x * g.x + f.y * g.y;
        }
#pragma unroll
        for (int w = LANES / 2; w > 0; w >>= 1) t += __shfl_xor_sync(0xffffffffu, t, w);
        const float got = __shfl_sync(0xffffffffu, t, lane % ROWS * LANES);
        if (lane / ROWS == i0 / ROWS + n) mine = got;
      }
    }
    const int64_t at = (static_cast<int64_t>(h) * slots + slot) * 128 + first + lane;
    const bool none = v == -INFINITY;
    a.nlse2[at] = none ? -INFINITY : -v * 1.4426950408889634f;
    a.ndelta[at] = none ? 0.f : -mine;
  }
}

// A operand (128 x 128 bf16 in TMEM; warpgroup w packed its 32 columns into
// words [32 w, 32 w + 16)) times 128 rows of `b_tile` (MN-major): the part
// that warpgroup w wrote.
template <int DH>
__device__ __forceinline__ void grad_mma_part(uint32_t d, uint32_t a, uint32_t b_tile, int w,
                                              bool accumulate) {
  constexpr uint32_t idesc = idesc_bf16(128, DH, false, true);
#pragma unroll
  for (int kk = 0; kk < 2; ++kk)
    umma_ts(d, a + 32 * w + 8 * kk, sdesc_sw128(b_tile + (2 * w + kk) * 2048, 16384, 1024), idesc,
            accumulate || w > 0 || kk > 0);
}

// 128 x 128 scores of two K-major tiles over the head dim.
template <int DH>
__device__ __forceinline__ void grad_mma_scores(uint32_t d, uint32_t a_tile, uint32_t b_tile) {
  constexpr uint32_t idesc = idesc_bf16(128, 128, false, false);
#pragma unroll
  for (int kk = 0; kk < DH / 16; ++kk) {
    const uint32_t off = (kk >> 2) * 16384 + (kk & 3) * 32;
    umma_ss(d, sdesc_sw128(a_tile + off, 16, 1024), sdesc_sw128(b_tile + off, 16, 1024), idesc,
            kk > 0);
  }
}

// ---------------------------------------------------------------- key pass

struct KeyPass {
  const SinkPlan* plan;
  float* part;        // [ctas][2][dV, dK][128][DH]: a CTA's first and last tile where shared
  const float* nlse2;
  const float* ndelta;
  __nv_bfloat16* dk;
  __nv_bfloat16* dv;
  int64_t ld;
};

// A CTA's walk over its units; every role keeps its own.
struct KeyCursor {
  int64_t x, x1;   // next item and end
  int slot, hk;
  SlotRec r;
  int weight, i0, i1;  // items [i0, i1)
  bool whole;
  __device__ void init(const SinkPlan* p, int c) {
    x = p->first[c];
    x1 = p->first[c + 1];
    slot = p->start[c] - 1;
    hk = 0;
    weight = 0;
    r.tile = -1;
  }
  // The next unit; false at the end.
  __device__ bool next(const SinkDims& s, const SinkPlan* p) {
    if (x >= x1) return false;
    if (weight == 0 || hk + 1 == s.Hkv) {
      const bool first = weight == 0;
      do {  // slots without a tile have no items
        ++slot;
        r = p->rec[slot];
      } while (r.tile < 0);
      weight = r.tiles * (s.H / s.Hkv) + kUnitCost;
      hk = first ? static_cast<int>((x - p->before[slot] * s.Hkv) / weight) : 0;
    } else {
      ++hk;
    }
    const int64_t begin = p->before[slot] * s.Hkv + static_cast<int64_t>(hk) * weight;
    const int end = static_cast<int>(min(static_cast<int64_t>(weight), x1 - begin));
    i0 = max(0, static_cast<int>(x - begin) - kUnitCost);
    i1 = end - kUnitCost;
    whole = i0 == 0 && end == weight;
    x = begin + end;
    return true;
  }
};

template <int DH>
__device__ __forceinline__ void sink_key_pass(int cta, const CUtensorMap& qmap,
                                              const CUtensorMap& domap, const CUtensorMap& kmap,
                                              const CUtensorMap& vmap, const SinkDims& dims,
                                              const KeyPass& a, float scale, uint32_t* status,
                                              uint64_t budget_ns) {
  using Cfg = GradCfg<DH>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  uint8_t* kvbuf = smem;                   // K, V
  uint8_t* ring = smem + 2 * Cfg::TILE;    // stage s: Q, dO
  uint8_t* stats = ring + Cfg::STAGES * 2 * Cfg::TILE;
  uint64_t* bars = reinterpret_cast<uint64_t*>(stats + Cfg::STAGES * Cfg::STATS);
  uint64_t* kv_full = bars;
  uint64_t* q_full = bars + 1;                  // [STAGES]
  uint64_t* do_full = q_full + Cfg::STAGES;     // [STAGES]
  uint64_t* st_full = do_full + Cfg::STAGES;    // [STAGES]
  uint64_t* q_empty = st_full + Cfg::STAGES;    // [STAGES] Q and the statistics
  uint64_t* do_empty = q_empty + Cfg::STAGES;   // [STAGES]
  uint64_t* s_full = do_empty + Cfg::STAGES;
  uint64_t* dp_full = s_full + 1;
  uint64_t* p_ready = dp_full + 1;              // [kGroups]
  uint64_t* ds_ready = p_ready + kGroups;       // [kGroups]
  uint64_t* acc_full = ds_ready + kGroups;      // a unit's sums are complete
  uint64_t* acc_free = acc_full + 1;            // and have been read
  uint64_t* kv_free = acc_free + 1;             // a unit's scores are all formed
  uint64_t* mma_done = kv_free + 1;
  uint64_t* cut = mma_done + 1;                 // tiles whose last rows are zeroed
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(cut + 1);

  if (cta >= a.plan->ctas) return;
  const int group = dims.H / dims.Hkv;
  const int q_slots = sink_slots(dims.Lq, dims.B, 128);
  const uint32_t warp = warp_id();
  KeyCursor cur;
  cur.init(a.plan, cta);

  if (threadIdx.x == 0) {
    mbar_init(kv_full, 1);
    for (int s = 0; s < Cfg::STAGES; ++s) {
      mbar_init(&q_full[s], 1);
      mbar_init(&do_full[s], 1);
      mbar_init(&st_full[s], 1);
      mbar_init(&q_empty[s], 1);
      mbar_init(&do_empty[s], 1);
    }
    mbar_init(s_full, 1);
    mbar_init(dp_full, 1);
    for (int w = 0; w < kGroups; ++w) {
      mbar_init(&p_ready[w], 128);
      mbar_init(&ds_ready[w], 128);
    }
    mbar_init(acc_full, 1);
    mbar_init(acc_free, kGroups * 128);
    mbar_init(kv_free, 1);
    mbar_init(mma_done, 1);
    mbar_init(cut, 1);
    fence_mbar_init();
    tma_prefetch_desc(&qmap);
    tma_prefetch_desc(&domap);
    tma_prefetch_desc(&kmap);
    tma_prefetch_desc(&vmap);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // columns: S^T [0, 128), dP^T [128, 256), dV, dK
  const uint32_t tmem = *tmem_slot;
  const uint32_t dv_addr = tmem + 256, dk_addr = tmem + 256 + DH;

  // Register split (launched with 96 x 640 = 61440): 128 * 64 + 512 * 104 =
  // 61440.
  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 64;\n" ::: "memory");
  }
  if (warp == 0) {
    // ================================================================ TMA
    const bool leader = lane_id() == 0;
    int n = 0, t = 0, cuts = 0;  // units with items, items and cut tiles so far
    bool ok = true;
    while (ok && cur.next(dims, a.plan)) {
      if (cur.i0 >= cur.i1) continue;
      const SinkSeq seq = sink_seq(dims, cur.r.b);
      const int q_base = sink_slot_base(dims.cu_q, cur.r.b, dims.Lq, 128);
      const int key0 = seq.k0 + 128 * cur.r.tile;
      // K and V are free once the last item's scores are formed, while its
      // sums are still to come
      if (n > 0 && !__all_sync(0xffffffffu, mbar_wait(kv_free, (n - 1) & 1, budget_ns))) {
        ok = false;
        break;
      }
      if (leader) {
        mbar_arrive_expect_tx(kv_full, 2 * Cfg::TILE);
        for (int sl = 0; sl < Cfg::SLABS; ++sl) {
          tma_load_2d(kvbuf + sl * 16384, &kmap, kv_full, cur.hk * DH + 64 * sl, key0);
          tma_load_2d(kvbuf + Cfg::TILE + sl * 16384, &vmap, kv_full, cur.hk * DH + 64 * sl,
                      key0);
        }
      }
      __syncwarp();
      ++n;
      int qi = cur.i0 % cur.r.tiles, h = cur.hk * group + cur.i0 / cur.r.tiles;
      for (int i = cur.i0; i < cur.i1; ++i, h += qi + 1 == cur.r.tiles,
               qi = qi + 1 == cur.r.tiles ? 0 : qi + 1) {
        const int s = t % Cfg::STAGES;
        const uint32_t par = ((t / Cfg::STAGES) & 1) ^ 1;
        const int qt = cur.r.t0 + qi;
        const int row = seq.q0 + 128 * qt, valid = min(128, seq.nq() - 128 * qt);
        uint8_t* qb = ring + s * 2 * Cfg::TILE;
        uint8_t* dob = qb + Cfg::TILE;
        if (t >= Cfg::STAGES &&
            !__all_sync(0xffffffffu, mbar_wait(&q_empty[s], par, budget_ns))) {
          ok = false;
          break;
        }
        uint64_t* qbar = valid < 128 ? cut : &q_full[s];
        if (leader) {
          mbar_arrive_expect_tx(&st_full[s], Cfg::STATS);
          const int64_t at = (static_cast<int64_t>(h) * q_slots + q_base + qt) * 128;
          bulk_load(stats + s * Cfg::STATS, a.nlse2 + at, 512, &st_full[s]);
          bulk_load(stats + s * Cfg::STATS + 512, a.ndelta + at, 512, &st_full[s]);
          mbar_arrive_expect_tx(qbar, (valid < 128 ? 2 : 1) * Cfg::TILE);
          for (int sl = 0; sl < Cfg::SLABS; ++sl)
            tma_load_2d(qb + sl * 16384, &qmap, qbar, h * DH + 64 * sl, row);
        }
        __syncwarp();
        ++t;
        if (t > Cfg::STAGES &&
            !__all_sync(0xffffffffu, mbar_wait(&do_empty[s], par, budget_ns))) {
          ok = false;
          break;
        }
        uint64_t* dobar = valid < 128 ? cut : &do_full[s];
        if (leader) {
          if (valid == 128) mbar_arrive_expect_tx(dobar, Cfg::TILE);
          for (int sl = 0; sl < Cfg::SLABS; ++sl)
            tma_load_2d(dob + sl * 16384, &domap, dobar, h * DH + 64 * sl, row);
        }
        __syncwarp();
        if (valid < 128) {
          // queries past the sequence's end have P = 0; their rows must not
          // be NaN
          if (!__all_sync(0xffffffffu, mbar_wait(cut, cuts & 1, budget_ns))) {
            ok = false;
            break;
          }
          ++cuts;
          sink_zero_rows(qb, Cfg::SLABS, valid);
          sink_zero_rows(dob, Cfg::SLABS, valid);
          if (leader) {
            mbar_arrive(&q_full[s]);
            mbar_arrive(&do_full[s]);
          }
        }
      }
    }
    if (!ok) record_status(status, kStatusTimeout);
    // no load may be in flight when the CTA ends
    if (n > 0) mbar_wait(kv_full, (n - 1) & 1, 200000000ull);
    for (int u = max(0, t - Cfg::STAGES); u < t; ++u) {
      const uint32_t par = (u / Cfg::STAGES) & 1;
      mbar_wait(&st_full[u % Cfg::STAGES], par, 200000000ull);
      mbar_wait(&q_full[u % Cfg::STAGES], par, 200000000ull);
      mbar_wait(&do_full[u % Cfg::STAGES], par, 200000000ull);
    }
    if (!ok) mbar_wait(cut, cuts & 1, 200000000ull);  // a cut tile's loads may be in flight
  } else if (warp == 1) {
    // ================================================================ MMA
    if (elect_one()) {
      const uint32_t kb = smem_u32(kvbuf), vb = kb + Cfg::TILE;
      auto q_tile = [&](int t) { return smem_u32(ring) + t % Cfg::STAGES * 2 * Cfg::TILE; };
      auto full = [&](uint64_t* bar, int t) {
        if (!mbar_wait(&bar[t % Cfg::STAGES], (t / Cfg::STAGES) & 1, budget_ns)) return false;
        tc_fence_after();
        return true;
      };
      auto scores = [&](int t) {  // S^T = K Q^T
        if (!full(q_full, t)) return false;
        grad_mma_scores<DH>(tmem, kb, q_tile(t));
        umma_commit(s_full);
        return true;
      };
      auto d_scores = [&](int t) {  // dP^T = V dO^T
        if (!full(do_full, t)) return false;
        grad_mma_scores<DH>(tmem + 128, vb, q_tile(t) + Cfg::TILE);
        umma_commit(dp_full);
        return true;
      };
      // dV += P^T dO or dK += dS^T Q, each part as its warpgroup is done
      auto sums = [&](uint64_t* ready, uint32_t d, uint32_t at, uint32_t tile, int t, bool more) {
        for (int w = 0; w < kGroups; ++w) {
          if (!mbar_wait(&ready[w], t & 1, budget_ns)) return false;
          tc_fence_after();
          grad_mma_part<DH>(d, at, tile, w, more);
        }
        return true;
      };
      int n = 0, loads = 0, t = 0;
      bool ok = true;
      while (ok && cur.next(dims, a.plan)) {
        const int items = cur.i1 - cur.i0;
        if (items > 0) {
          if (!(ok = mbar_wait(kv_full, loads++ & 1, budget_ns))) break;
          tc_fence_after();
          if (!(ok = scores(t) && d_scores(t))) break;
          if (items == 1) umma_commit(kv_free);
        }
        // the last unit's sums have been read
        if (n > 0 && !(ok = mbar_wait(acc_free, (n - 1) & 1, budget_ns))) break;
        tc_fence_after();
        // While the tensor core runs dV_t and S_{t+1}, the warpgroups form
        // dS_t; while it runs dK_t and dP_{t+1}, they form P_{t+1}.
        for (int i = 0; i < items; ++i, ++t) {
          const bool more = i + 1 < items;
          if (!(ok = sums(p_ready, dv_addr, tmem, q_tile(t) + Cfg::TILE, t, i > 0))) break;
          umma_commit(&do_empty[t % Cfg::STAGES]);
          if (more && !(ok = scores(t + 1))) break;
          if (!(ok = sums(ds_ready, dk_addr, tmem + 128, q_tile(t), t, i > 0))) break;
          umma_commit(&q_empty[t % Cfg::STAGES]);
          if (more && !(ok = d_scores(t + 1))) break;
          if (i + 2 == items) umma_commit(kv_free);
        }
        if (!ok) break;
        umma_commit(acc_full);
        ++n;
      }
      if (!ok) record_status(status, kStatusTimeout);
      umma_commit(mma_done);
    }
  } else if (warp >= 4) {
    // ================================================================ softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 104;\n" ::: "memory");
    // thread = key row; this warpgroup's 32 of the tile's 128 queries
    const int w = (warp - 4) >> 2;
    const uint32_t quarter = warp & 3, lane_off = (quarter * 32) << 16;
    const uint32_t s_addr = tmem + 32 * w + lane_off, dp_addr = s_addr + 128;
    const float scale_log2 = scale * 1.4426950408889634f;
    const uint64_t cc = f32x2_pack(scale_log2, scale_log2);
    const SinkMask m = dims.m;
    int n = 0, t = 0;
    bool ok = true;
    while (ok && cur.next(dims, a.plan)) {
      const SinkSeq seq = sink_seq(dims, cur.r.b);
      const int ks = 128 * cur.r.tile, kw = ks + quarter * 32, key = kw + lane_id();
      // position of this part's first query, of the unit's first query tile
      // and of the item's
      const int p_first = 128 * cur.r.t0 + seq.shift() + 32 * w;
      int qi = cur.r.tiles > 0 ? cur.i0 % cur.r.tiles : 0;
      for (int i = cur.i0; i < cur.i1; ++i, ++t) {
        const int s = t % Cfg::STAGES;
        const int p0 = p_first + 128 * qi;
        if (++qi == cur.r.tiles) qi = 0;
        const bool edge = !sink_sees_all(m, p0, p0 + 31, kw, kw + 31);
        if (!__all_sync(0xffffffffu,
                        mbar_wait(&st_full[s], (t / Cfg::STAGES) & 1, budget_ns) &&
                            mbar_wait(s_full, t & 1, budget_ns))) {
          ok = false;
          break;
        }
        tc_fence_after();
        const ulonglong2* nl = reinterpret_cast<const ulonglong2*>(stats + s * Cfg::STATS) + 8 * w;
        const ulonglong2* dl = nl + 32;
        uint32_t x[32];
        tmem_ld32(s_addr, x);
        tmem_ld_wait();
        reg_fence(x);
        // P over S: 2^(s scale log2 e - lse log2 e)
        uint32_t pk[16];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const ulonglong2 n2 = nl[e];
#pragma unroll
          for (int f = 0; f < 2; ++f) {
            const int c = 4 * e + 2 * f;
            const uint64_t y = f32x2_fma((static_cast<uint64_t>(x[c + 1]) << 32) | x[c], cc,
                                         f ? n2.y : n2.x);
            x[c] = __float_as_uint(exp2_mufu(f32x2_lo(y)));
            x[c + 1] = __float_as_uint(exp2_mufu(f32x2_hi(y)));
          }
        }
        uint32_t see = 0xffffffffu;
        if (edge) {
          see = sink_bits(key - m.ahead - p0, key < m.sinks ? 32 : key - p0 + m.window, 0);
#pragma unroll
          for (int c = 0; c < 32; ++c) x[c] = see & (1u << c) ? x[c] : 0;
        }
#pragma unroll
        for (int e = 0; e < 16; ++e)
          pk[e] = pack_bf16x2(__uint_as_float(x[2 * e]), __uint_as_float(x[2 * e + 1]));
        tmem_st16(s_addr, pk);
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(&p_ready[w]);
        // dS = P (dP - D)
        if (!__all_sync(0xffffffffu, mbar_wait(dp_full, t & 1, budget_ns))) {
          ok = false;
          break;
        }
        tc_fence_after();
        uint32_t g[32];
        tmem_ld32(dp_addr, g);
        tmem_ld_wait();
        reg_fence(g);
        if (edge) {  // dP of a hidden pair may be NaN, and 0 x NaN is not 0
#pragma unroll
          for (int c = 0; c < 32; ++c) g[c] = see & (1u << c) ? g[c] : 0;
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const ulonglong2 d2 = dl[e];
#pragma unroll
          for (int f = 0; f < 2; ++f) {
            const int c = 4 * e + 2 * f;
            const uint64_t y = f32x2_mul(
                (static_cast<uint64_t>(x[c + 1]) << 32) | x[c],
                f32x2_add((static_cast<uint64_t>(g[c + 1]) << 32) | g[c], f ? d2.y : d2.x));
            pk[2 * e + f] = pack_bf16x2(f32x2_lo(y), f32x2_hi(y));
          }
        }
        tmem_st16(dp_addr, pk);
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(&ds_ready[w]);
      }
      if (!ok) break;
      // ---- the unit's sums: warpgroups 0, 1 store dV, 2, 3 dK, half the
      // columns each
      if (!__all_sync(0xffffffffu, mbar_wait(acc_full, n & 1, budget_ns))) {
        ok = false;
        break;
      }
      tc_fence_after();
      const int which = w >> 1, c0 = (w & 1) * (DH / 2);
      const uint32_t addr = (which ? dk_addr : dv_addr) + lane_off + c0;
      const float factor = which ? scale : 1.f;
      const int row = quarter * 32 + lane_id();
      const int key0 = seq.k0 + ks;
      const bool live = ks + row < seq.nk() &&
                        in_bounds(status, key0 + row, dims.Lk, cur.hk * DH, DH,
                                  static_cast<int64_t>(dims.Hkv) * DH);
      __nv_bfloat16* dst = (which ? a.dk : a.dv) + static_cast<int64_t>(key0 + row) * a.ld +
                           cur.hk * DH + c0;
      float* part = a.part +
                    ((static_cast<int64_t>(cta) * 2 + (cur.i0 == 0)) * 2 + which) * (DH * 128) +
                    row * DH + c0;
#pragma unroll 1
      for (int c = 0; c < DH / 2; c += 32) {
        uint32_t x[32];
        if (cur.i1 > cur.i0) {
          tmem_ld32(addr + c, x);
          tmem_ld_wait();
          reg_fence(x);
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e) x[e] = 0;
        }
        if (!cur.whole) {
#pragma unroll
          for (int e = 0; e < 32; e += 4)
            *reinterpret_cast<uint4*>(part + c + e) = make_uint4(x[e], x[e + 1], x[e + 2], x[e + 3]);
        } else if (live) {
#pragma unroll
          for (int e = 0; e < 32; e += 8) {
            uint4 u;
            auto two = [&](int k) {
              return pack_bf16x2(__uint_as_float(x[e + k]) * factor,
                                 __uint_as_float(x[e + k + 1]) * factor);
            };
            u.x = two(0), u.y = two(2), u.z = two(4), u.w = two(6);
            *reinterpret_cast<uint4*>(dst + c + e) = u;
          }
        }
      }
      tc_fence_before();
      mbar_arrive(acc_free);
      ++n;
    }
    if (!ok) record_status(status, kStatusTimeout);
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    mbar_wait(mma_done, 0, 200000000ull);
    tmem_dealloc(tmem, 512);
  }
}

// dK and dV of the units that several CTAs share: the sum of their parts, the
// CTA with the unit's first items first.  blockIdx.x: the CTA whose begin is
// the first inside the unit, if there is one.
template <int DH>
__global__ void __launch_bounds__(256) sink_join_kernel(const SinkDims dims, const KeyPass a,
                                                        float scale, uint32_t* status) {
  after_wait();
  const SinkPlan* p = a.plan;
  const int c1 = blockIdx.x + 1;
  if (c1 >= p->ctas) return;
  const int slot = p->start[c1];
  const int64_t x1 = p->first[c1], x0 = p->first[c1 - 1], at = p->before[slot] * dims.Hkv;
  const SlotRec r = p->rec[slot];
  if (r.tile < 0) return;
  const int64_t weight = r.tiles * (dims.H / dims.Hkv) + kUnitCost;
  const int hk = static_cast<int>((x1 - at) / weight);
  const int64_t begin = at + hk * weight;
  if (hk >= dims.Hkv || x1 == begin || x0 > begin) return;
  const SinkSeq seq = sink_seq(dims, r.b);
  // blockIdx.y: dV or dK, and 16 of the 128 keys; a thread: 8 columns of a key
  const int which = blockIdx.y >> 3;
  const int row = (blockIdx.y & 7) * 16 + threadIdx.x / (DH / 8), c0 = threadIdx.x % (DH / 8) * 8;
  if (threadIdx.x >= 16 * (DH / 8) || 128 * r.tile + row >= seq.nk()) return;
  float x[8] = {};
  for (int c = c1 - 1; c < p->ctas && p->first[c] < begin + weight; ++c) {
    const float4* in = reinterpret_cast<const float4*>(
        a.part + ((static_cast<int64_t>(c) * 2 + (c < c1)) * 2 + which) * (DH * 128) +
        row * DH + c0);
    const float4 u = in[0], v = in[1];
    x[0] += u.x, x[1] += u.y, x[2] += u.z, x[3] += u.w;
    x[4] += v.x, x[5] += v.y, x[6] += v.z, x[7] += v.w;
  }
  const float f = which ? scale : 1.f;
  const int64_t at_row = seq.k0 + 128 * r.tile + row;
  if (!in_bounds(status, at_row, dims.Lk, hk * DH + c0, 8, static_cast<int64_t>(dims.Hkv) * DH))
    return;
  __nv_bfloat16* dst = (which ? a.dk : a.dv) + at_row * a.ld + hk * DH + c0;
  uint4 u;
  u.x = pack_bf16x2(x[0] * f, x[1] * f);
  u.y = pack_bf16x2(x[2] * f, x[3] * f);
  u.z = pack_bf16x2(x[4] * f, x[5] * f);
  u.w = pack_bf16x2(x[6] * f, x[7] * f);
  *reinterpret_cast<uint4*>(dst) = u;
}

// ---------------------------------------------------------------- query pass
//
// A CTA holds 128 queries of one head (Q and dO resident) and walks the key
// tiles they see.  TMEM columns: S [0, 128), dP twice [128, 384), dQ
// [384, 384 + DH): S_{j+1} is issued once the warpgroups have loaded S_j, dP
// alternates, so both are ready when the warpgroups come back for them.
template <int DH>
__device__ __forceinline__ void sink_query_pass(int cta, const CUtensorMap& qmap,
                                                const CUtensorMap& domap, const CUtensorMap& kmap,
                                                const CUtensorMap& vmap, const SinkDims& dims,
                                                const float* __restrict__ nlse2,
                                                const float* __restrict__ ndelta, float scale,
                                                __nv_bfloat16* __restrict__ dq, int64_t ld_dq,
                                                uint32_t* status, uint64_t budget_ns) {
  using Cfg = GradCfg<DH>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  uint8_t* qbuf = smem;                  // Q, dO
  uint8_t* ring = smem + 2 * Cfg::TILE;  // stage s: K, V
  uint64_t* bars = reinterpret_cast<uint64_t*>(ring + Cfg::STAGES * 2 * Cfg::TILE);
  uint64_t* q_full = bars;
  uint64_t* k_full = bars + 1;                // [STAGES]
  uint64_t* v_full = k_full + Cfg::STAGES;    // [STAGES]
  uint64_t* k_empty = v_full + Cfg::STAGES;   // [STAGES]
  uint64_t* v_empty = k_empty + Cfg::STAGES;  // [STAGES]
  uint64_t* s_full = v_empty + Cfg::STAGES;
  uint64_t* s_free = s_full + 1;              // S loaded by all softmax threads
  uint64_t* dp_full = s_free + 1;             // [2]
  // [2][kGroups], by the parity of the key tile: a warpgroup may be done with
  // tile j + 1 before the products of tile j have waited for the slowest one
  uint64_t* ds_ready = dp_full + 2;
  uint64_t* mma_done = ds_ready + 2 * kGroups;
  uint64_t* cut = mma_done + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(cut + 1);

  // Heaviest first: the last queries of a sequence see the most keys.
  const int slots = sink_slots(dims.Lq, dims.B, 128);
  const int slot = slots - 1 - cta / dims.H;
  const int h = cta % dims.H, hk = h / (dims.H / dims.Hkv);
  const int b = sink_slot_seq(dims.cu_q, dims.B, dims.Lq, 128, slot);
  const SinkSeq seq = sink_seq(dims, b);
  const int row0 = seq.q0 + 128 * (slot - sink_slot_base(dims.cu_q, b, dims.Lq, 128));
  if (row0 < seq.q0 || row0 >= seq.q1) return;  // the whole CTA
  const int pa = row0 - seq.q0 + seq.shift(), pb = min(pa + 127, seq.nk() - 1);
  SinkKeyTiles kt;
  kt.init(dims.m, pa, pb, seq.nk());
  const uint32_t warp = warp_id();

  if (threadIdx.x == 0) {
    mbar_init(q_full, 1);
    for (int s = 0; s < Cfg::STAGES; ++s) {
      mbar_init(&k_full[s], 1);
      mbar_init(&v_full[s], 1);
      mbar_init(&k_empty[s], 1);
      mbar_init(&v_empty[s], 1);
    }
    mbar_init(s_full, 1);
    mbar_init(s_free, kGroups * 128);
    mbar_init(&dp_full[0], 1);
    mbar_init(&dp_full[1], 1);
    for (int w = 0; w < 2 * kGroups; ++w) mbar_init(&ds_ready[w], 128);
    mbar_init(mma_done, 1);
    mbar_init(cut, 1);
    fence_mbar_init();
    tma_prefetch_desc(&qmap);
    tma_prefetch_desc(&domap);
    tma_prefetch_desc(&kmap);
    tma_prefetch_desc(&vmap);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const uint32_t dq_addr = tmem + 384;

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 64;\n" ::: "memory");
  }
  if (warp == 0) {
    // ================================================================ TMA
    const bool leader = lane_id() == 0;
    if (leader) {
      mbar_arrive_expect_tx(q_full, 2 * Cfg::TILE);
      for (int sl = 0; sl < Cfg::SLABS; ++sl) {
        tma_load_2d(qbuf + sl * 16384, &qmap, q_full, h * DH + 64 * sl, row0);
        tma_load_2d(qbuf + Cfg::TILE + sl * 16384, &domap, q_full, h * DH + 64 * sl, row0);
      }
    }
    int issued_k = 0, issued_v = 0, cuts = 0;
    bool ok = true;
    for (int j = 0; j < kt.n; ++j) {
      const int s = j % Cfg::STAGES;
      const uint32_t par = ((j / Cfg::STAGES) & 1) ^ 1;
      const int key0 = seq.k0 + kt.start(j), valid = kt.valid(j);
      uint8_t* kb = ring + s * 2 * Cfg::TILE;
      uint8_t* vb = kb + Cfg::TILE;
      if (j >= Cfg::STAGES && !__all_sync(0xffffffffu, mbar_wait(&v_empty[s], par, budget_ns))) {
        ok = false;
        break;
      }
      if (leader) {
        mbar_arrive_expect_tx(&v_full[s], Cfg::TILE);
        for (int sl = 0; sl < Cfg::SLABS; ++sl)
          tma_load_2d(vb + sl * 16384, &vmap, &v_full[s], hk * DH + 64 * sl, key0);
      }
      __syncwarp();
      ++issued_v;
      if (j >= Cfg::STAGES && !__all_sync(0xffffffffu, mbar_wait(&k_empty[s], par, budget_ns))) {
        ok = false;
        break;
      }
      uint64_t* full = valid < 128 ? cut : &k_full[s];
      if (leader) {
        mbar_arrive_expect_tx(full, Cfg::TILE);
        for (int sl = 0; sl < Cfg::SLABS; ++sl)
          tma_load_2d(kb + sl * 16384, &kmap, full, hk * DH + 64 * sl, key0);
      }
      __syncwarp();
      if (valid < 128) {
        if (!__all_sync(0xffffffffu, mbar_wait(cut, cuts & 1, budget_ns))) {
          ok = false;
          break;
        }
        ++cuts;
        sink_zero_rows(kb, Cfg::SLABS, valid);
        if (leader) mbar_arrive(&k_full[s]);
      }
      ++issued_k;
    }
    if (!ok) record_status(status, kStatusTimeout);
    mbar_wait(q_full, 0, 200000000ull);
    for (int t = max(0, issued_v - Cfg::STAGES); t < issued_v; ++t)
      mbar_wait(&v_full[t % Cfg::STAGES], (t / Cfg::STAGES) & 1, 200000000ull);
    for (int t = max(0, issued_k - Cfg::STAGES); t < issued_k; ++t)
      mbar_wait(&k_full[t % Cfg::STAGES], (t / Cfg::STAGES) & 1, 200000000ull);
    if (!ok) mbar_wait(cut, cuts & 1, 200000000ull);  // a cut tile's load may be in flight
  } else if (warp == 1) {
    // ================================================================ MMA
    if (elect_one()) {
      const uint32_t qb = smem_u32(qbuf), dob = qb + Cfg::TILE;
      auto k_tile = [&](int j) { return smem_u32(ring) + j % Cfg::STAGES * 2 * Cfg::TILE; };
      auto products = [&](int j) {  // S = Q K^T and dP = dO V^T
        const int s = j % Cfg::STAGES;
        if (!mbar_wait(&k_full[s], (j / Cfg::STAGES) & 1, budget_ns)) return false;
        tc_fence_after();
        grad_mma_scores<DH>(tmem, qb, k_tile(j));
        umma_commit(s_full);
        if (!mbar_wait(&v_full[s], (j / Cfg::STAGES) & 1, budget_ns)) return false;
        tc_fence_after();
        grad_mma_scores<DH>(tmem + 128 + 128 * (j & 1), dob, k_tile(j) + Cfg::TILE);
        umma_commit(&dp_full[j & 1]);
        umma_commit(&v_empty[s]);
        return true;
      };
      bool ok = mbar_wait(q_full, 0, budget_ns);
      if (ok && kt.n > 0) ok = products(0);
      for (int j = 0; j < kt.n && ok; ++j) {
        if (j + 1 < kt.n) {
          if (!(ok = mbar_wait(s_free, j & 1, budget_ns))) break;
          tc_fence_after();
          if (!(ok = products(j + 1))) break;
        }
        for (int w = 0; w < kGroups && ok; ++w) {
          if (!(ok = mbar_wait(&ds_ready[(j & 1) * kGroups + w], (j >> 1) & 1, budget_ns))) break;
          tc_fence_after();
          grad_mma_part<DH>(dq_addr, tmem + 128 + 128 * (j & 1), k_tile(j), w, j > 0);
        }
        if (ok) umma_commit(&k_empty[j % Cfg::STAGES]);
      }
      if (!ok) record_status(status, kStatusTimeout);
      umma_commit(mma_done);
    }
  } else if (warp >= 4) {
    // ================================================================ softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 104;\n" ::: "memory");
    const int w = (warp - 4) >> 2;           // this warpgroup's 32 keys of a tile
    const uint32_t quarter = warp & 3;
    const uint32_t lane_off = (quarter * 32) << 16;
    const int row = quarter * 32 + lane_id();
    const int p = pa + row, pw = pa + quarter * 32;
    const int64_t at = (static_cast<int64_t>(h) * slots + slot) * 128 + row;
    const float nl = nlse2[at], nd = ndelta[at];
    const float scale_log2 = scale * 1.4426950408889634f;
    const uint64_t cc = f32x2_pack(scale_log2, scale_log2), nl2 = f32x2_pack(nl, nl),
                   nd2 = f32x2_pack(nd, nd);
    const SinkMask m = dims.m;
    bool ok = true;
    for (int j = 0; j < kt.n; ++j) {
      const int ks = kt.start(j) + 32 * w, valid = kt.valid(j) - 32 * w;
      const bool edge = valid < 32 || !sink_sees_all(m, pw, pw + 31, ks, ks + 31);
      if (!__all_sync(0xffffffffu, mbar_wait(s_full, j & 1, budget_ns))) {
        ok = false;
        break;
      }
      tc_fence_after();
      uint32_t x[32];
      tmem_ld32(tmem + lane_off + 32 * w, x);
      tmem_ld_wait();
      reg_fence(x);
      tc_fence_before();
      mbar_arrive(s_free);
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const uint64_t y =
            f32x2_fma((static_cast<uint64_t>(x[2 * e + 1]) << 32) | x[2 * e], cc, nl2);
        x[2 * e] = __float_as_uint(exp2_mufu(f32x2_lo(y)));
        x[2 * e + 1] = __float_as_uint(exp2_mufu(f32x2_hi(y)));
      }
      if (!__all_sync(0xffffffffu, mbar_wait(&dp_full[j & 1], (j >> 1) & 1, budget_ns))) {
        ok = false;
        break;
      }
      tc_fence_after();
      const uint32_t g_addr = tmem + 128 + 128 * (j & 1) + 32 * w + lane_off;
      uint32_t g[32];
      tmem_ld32(g_addr, g);
      tmem_ld_wait();
      reg_fence(g);
      if (edge) {  // of a hidden pair P is not 0 here, and dP may be NaN
        const uint32_t see = sink_bits(p - m.window + 1 - ks, min(valid, p + m.ahead + 1 - ks),
                                       m.sinks - ks);
#pragma unroll
        for (int c = 0; c < 32; ++c) {
          x[c] = see & (1u << c) ? x[c] : 0;
          g[c] = see & (1u << c) ? g[c] : 0;
        }
      }
      uint32_t ds[16];
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const uint64_t y = f32x2_mul(
            (static_cast<uint64_t>(x[2 * e + 1]) << 32) | x[2 * e],
            f32x2_add((static_cast<uint64_t>(g[2 * e + 1]) << 32) | g[2 * e], nd2));
        ds[e] = pack_bf16x2(f32x2_lo(y), f32x2_hi(y));
      }
      tmem_st16(g_addr, ds);
      tmem_st_wait();
      tc_fence_before();
      mbar_arrive(&ds_ready[(j & 1) * kGroups + w]);
    }
    if (__all_sync(0xffffffffu, ok && mbar_wait(mma_done, 0, budget_ns))) {
      tc_fence_after();
      const bool live = row0 + row < seq.q1 &&
                        in_bounds(status, row0 + row, dims.Lq, h * DH, DH,
                                  static_cast<int64_t>(dims.H) * DH);
      __nv_bfloat16* dst = dq + static_cast<int64_t>(row0 + row) * ld_dq + h * DH;
      // the warpgroups take the 32-column parts in turn
#pragma unroll 1
      for (int c = 32 * w; c < DH; c += 32 * kGroups) {
        uint32_t x[32];
        if (kt.n > 0) {
          tmem_ld32(dq_addr + lane_off + c, x);
          tmem_ld_wait();
          reg_fence(x);
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e) x[e] = 0;
        }
        if (!live) continue;
#pragma unroll
        for (int e = 0; e < 32; e += 8) {
          uint4 u;
          auto two = [&](int n) {
            return pack_bf16x2(__uint_as_float(x[e + n]) * scale,
                               __uint_as_float(x[e + n + 1]) * scale);
          };
          u.x = two(0), u.y = two(2), u.z = two(4), u.w = two(6);
          *reinterpret_cast<uint4*>(dst + c + e) = u;
        }
      }
    } else {
      record_status(status, kStatusTimeout);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    mbar_wait(mma_done, 0, 200000000ull);
    tmem_dealloc(tmem, 512);
  }
}

// Both passes in one launch: they need nothing of each other, so the query
// pass's tiles fill the SMs that the key pass has left (three short sequences:
// 41 to 25 us of kernels; 8097 tokens, 16 heads over 4, window 1024: 318 to 300).
// Bound, as in the forward pass, by the chain of a tile: products, exponentials,
// TMEM stores and loads, products; the tensor pipe is 42 % busy, the
// exponentials' 25 %.  8097 tokens: 277 us, 0.70 PFLOP/s of the 14 d flop a
// visible pair that the two passes do (10 d in one pass with atomic adds), 0.43
// of the burst rate of a large product.  Measured and not kept: half the exponentials on the
// FMA pipe (148 to 152 us key pass, 135 to 147 query pass); P^T through shared
// memory in the key pass (271 to 273); query tiles dealt out like the key
// pass's items (the same).
template <int DH>
__global__ void __launch_bounds__(kThreads, 1)
    sink_grad_kernel(const __grid_constant__ CUtensorMap qmap,
                     const __grid_constant__ CUtensorMap domap,
                     const __grid_constant__ CUtensorMap kmap,
                     const __grid_constant__ CUtensorMap vmap, const SinkDims dims,
                     const KeyPass a, int key_ctas, float scale, __nv_bfloat16* __restrict__ dq,
                     int64_t ld_dq, uint32_t* status, uint64_t budget_ns) {
  const int cta = blockIdx.x;
  after_wait();
  after_allow();  // sink_join_kernel, where there is one
  if (cta < key_ctas)
    sink_key_pass<DH>(cta, qmap, domap, kmap, vmap, dims, a, scale, status, budget_ns);
  else
    sink_query_pass<DH>(cta - key_ctas, qmap, domap, kmap, vmap, dims, a.nlse2, a.ndelta, scale,
                        dq, ld_dq, status, budget_ns);
}

// ---------------------------------------------------------------- host

// Workspace: status, the two statistics, the plan with its arrays, the parts
// of shared units.
struct GradLayout {
  size_t stats;  // bytes of one statistic
  size_t plan, rec, before, part;
  int ctas;
  bool whole;  // a unit a CTA: nothing to join
  size_t total;
};

size_t align256(size_t n) { return (n + 255) / 256 * 256; }

GradLayout grad_layout(const vdn_sink_shape& s) {
  GradLayout l;
  const size_t k_slots = sink_slots(s.Lk, s.B, 128);
  // no more CTAs than the plan could give twice a unit's cost: a tile has at
  // most Lq / 128 + 2 query tiles of each of its heads
  const double items = static_cast<double>(k_slots) * s.H *
                       (s.Lq / 128 + 2 + kUnitCost) / (2 * kUnitCost);
  l.ctas = items < 1 ? 1 : items > kCtas ? kCtas : static_cast<int>(items);
  // Few and short units stay whole, which saves the join and a second load of
  // the shared units' tiles: at most one an SM, with 16 items at most
  // (a query tile more at either end of what the window or the rows allow).
  const int64_t group = s.H / s.H_kv;
  int64_t tiles = s.Lq / 128 + 2;
  if (s.sinks == 0) {
    const int64_t near = (static_cast<int64_t>(s.window) + s.ahead + 126) / 128 + 2;
    tiles = near < tiles ? near : tiles;
  }
  l.whole = static_cast<int64_t>(k_slots) * s.H_kv <= kCtas && tiles * group <= 16;
  if (l.whole) l.ctas = static_cast<int>(k_slots) * s.H_kv;
  l.stats = align256(static_cast<size_t>(s.H) * sink_slots(s.Lq, s.B, 128) * 128 * sizeof(float));
  l.plan = kStatusBytes + 2 * l.stats;
  l.rec = l.plan + align256(sizeof(SinkPlan));
  l.before = l.rec + align256(k_slots * sizeof(SlotRec));
  l.part = l.before + align256((k_slots + 1) * sizeof(int64_t));
  l.total = l.part + (l.whole ? 0 : static_cast<size_t>(l.ctas) * 4 * s.d * 128 * sizeof(float));
  return l;
}

struct GradMaps {
  CUtensorMap q, d_o, k, v;
};

template <int DH>
cudaError_t launch_sink_grad(const Launch& ctx, const SinkDims& dims, const GradMaps& t,
                             const KeyPass& a, int ctas, const StatsArgs& st, float scale,
                             __nv_bfloat16* dq, int64_t ld_dq) {
  using Cfg = GradCfg<DH>;
  static std::atomic<uint64_t> smem_set{0};
  if (cudaError_t e = set_smem_once(sink_grad_kernel<DH>, Cfg::SMEM, smem_set)) return e;
  const int q_slots = sink_slots(dims.Lq, dims.B, 128);
  sink_stats_kernel<DH><<<1 + 4 * q_slots, 256, 0, ctx.stream>>>(dims, st);
  if (cudaError_t e = cudaGetLastError()) return e;
  if (cudaError_t e = launch_after(sink_few_kernel<DH>, dim3(st.few_blocks), 256, 0, ctx.stream,
                                   dims, st))
    return e;
  const int key_ctas = dims.Lk > 0 ? ctas : 0, query_ctas = dims.Lq > 0 ? q_slots * dims.H : 0;
  if (cudaError_t e = launch_after(sink_grad_kernel<DH>, dim3(key_ctas + query_ctas), kThreads,
                                   Cfg::SMEM, ctx.stream, t.q, t.d_o, t.k, t.v, dims, a, key_ctas,
                                   scale, dq, ld_dq, ctx.status, ctx.budget_ns))
    return e;
  if (key_ctas > 1 && !st.whole)
    return launch_after(sink_join_kernel<DH>, dim3(key_ctas - 1, 16), 256, 0, ctx.stream, dims, a,
                        scale, ctx.status);
  return cudaSuccess;
}

}  // namespace

}  // namespace vdn

using namespace vdn;

extern "C" {

size_t vdn_sink_attn_backward_workspace(const vdn_sink_shape* shape) {
  vdn_sink_shape s;
  const void* p = reinterpret_cast<const void*>(256);
  if (shape == nullptr ||
      sink_check(shape, p, (int64_t)1 << 24, p, p, (int64_t)1 << 24,
                 static_cast<const int32_t*>(p), static_cast<const int32_t*>(p), &s) != VDN_OK)
    return 0;
  return grad_layout(s).total;
}

vdn_status vdn_sink_attn_backward(const vdn_sink_shape* shape, const void* q, int64_t ld_q,
                                  const void* k, const void* v, int64_t ld_kv,
                                  const int32_t* cu_q, const int32_t* cu_k, float scale,
                                  const void* o, int64_t ld_o, const float* lse, const void* d_o,
                                  int64_t ld_do, void* dq, int64_t ld_dq, void* dk, void* dv,
                                  int64_t ld_dkv, unsigned zero_rest, void* ws, size_t ws_bytes,
                                  void* stream) {
  NvtxRange nvtx("vdn_sink_attn_backward");
  vdn_sink_shape s;
  const vdn_status r = sink_check(shape, q, ld_q, k, v, ld_kv, cu_q, cu_k, &s);
  if (r != VDN_OK) return r;
  const int64_t D = static_cast<int64_t>(s.H) * s.d, Dk = static_cast<int64_t>(s.H_kv) * s.d;
  auto bad = [](const void* p, int rows, int64_t ld, int64_t cols) {
    return (p == nullptr && rows > 0) || (reinterpret_cast<uintptr_t>(p) & 15u) || ld < cols ||
           ld % 8 != 0;
  };
  if (bad(o, s.Lq, ld_o, D) || bad(d_o, s.Lq, ld_do, D) || bad(dq, s.Lq, ld_dq, D) ||
      bad(dk, s.Lk, ld_dkv, Dk) || bad(dv, s.Lk, ld_dkv, Dk) || (lse == nullptr && s.Lq > 0) ||
      (reinterpret_cast<uintptr_t>(lse) & 3u))
    return VDN_ERR_INVALID_ARG;
  const GradLayout lay = grad_layout(s);
  if (ws == nullptr || (reinterpret_cast<uintptr_t>(ws) & 255u) || ws_bytes < lay.total)
    return VDN_ERR_WORKSPACE;
  const int64_t limit = int64_t(1) << 31;
  if (static_cast<int64_t>(sink_slots(s.Lq, s.B, 128)) * s.H + kCtas >= limit ||
      static_cast<int64_t>(sink_slots(s.Lk, s.B, 128)) * s.H_kv >= limit ||
      (static_cast<int64_t>(s.Lq) + 127) / 128 * (s.H / s.H_kv) >= limit)
    return VDN_ERR_UNSUPPORTED;
  if (s.Lq == 0 && s.Lk == 0) return VDN_OK;
  const SinkDims dims{s.Lq, s.Lk, s.B, s.H, s.H_kv, cu_q, cu_k, {s.window, s.ahead, s.sinks}};
  GradMaps t;
  // without queries or keys the missing side's tiles are never loaded
  if (s.Lq > 0 && (!make_rows_map(&t.q, q, D, ld_q, s.Lq, 128) ||
                   !make_rows_map(&t.d_o, d_o, D, ld_do, s.Lq, 128)))
    return VDN_ERR_CUDA;
  if (s.Lk > 0 && (!make_rows_map(&t.k, k, Dk, ld_kv, s.Lk, 128) ||
                   !make_rows_map(&t.v, v, Dk, ld_kv, s.Lk, 128)))
    return VDN_ERR_CUDA;
  if (s.Lq == 0) t.q = t.d_o = t.k;
  if (s.Lk == 0) t.k = t.v = t.q;
  uint8_t* base = static_cast<uint8_t*>(ws);
  float* nlse2 = reinterpret_cast<float*>(base + kStatusBytes);
  float* ndelta = reinterpret_cast<float*>(base + kStatusBytes + lay.stats);
  SinkPlan* plan = reinterpret_cast<SinkPlan*>(base + lay.plan);
  const KeyPass a{plan,
                  reinterpret_cast<float*>(base + lay.part),
                  nlse2,
                  ndelta,
                  static_cast<__nv_bfloat16*>(dk),
                  static_cast<__nv_bfloat16*>(dv),
                  ld_dkv};
  const Launch ctx{static_cast<cudaStream_t>(stream), static_cast<uint32_t*>(ws),
                   current_wait_budget_ns()};
  const float sc = scale > 0.f ? scale : 1.f / sqrtf(static_cast<float>(s.d));
  StatsArgs st{};
  st.q = static_cast<const __nv_bfloat16*>(q);
  st.k = static_cast<const __nv_bfloat16*>(k);
  st.v = static_cast<const __nv_bfloat16*>(v);
  st.ld_q = ld_q, st.ld_kv = ld_kv;
  st.scale_log2 = sc * 1.4426950408889634f;
  // groups of a sequence taken side by side: those of its beginning, or, where
  // all may see few keys, as many as fill the GPU
  const int64_t each = static_cast<int64_t>(s.B) * ((s.H * kFewWarps + 7) / 8);
  int64_t side = kFewKeys / kFewRows + 1;
  if (s.window <= kFewKeys) side = 4 * kCtas / each > 1 ? 4 * kCtas / each : 1;
  st.few_stride = static_cast<int>(side);
  st.few_blocks = static_cast<int>(each * side < (1 << 16) ? each * side : 1 << 16);
  st.o = static_cast<const __nv_bfloat16*>(o);
  st.d_o = static_cast<const __nv_bfloat16*>(d_o);
  st.ld_o = ld_o, st.ld_do = ld_do;
  st.lse = lse, st.nlse2 = nlse2, st.ndelta = ndelta;
  st.plan = plan;
  st.rec = reinterpret_cast<SlotRec*>(base + lay.rec);
  st.before = reinterpret_cast<int64_t*>(base + lay.before);
  st.ctas = lay.ctas;
  st.whole = lay.whole;
  void* outs[3] = {dq, dk, dv};
  const int64_t lds[3] = {ld_dq, ld_dkv, ld_dkv};
  for (int i = 0; i < 3; ++i) {
    st.zero[i] = zero_rest >> i & 1u ? outs[i] : nullptr;
    st.ld_zero[i] = lds[i];
  }
  auto run = [&](auto dh) {
    return launch_sink_grad<decltype(dh)::value>(ctx, dims, t, a, lay.ctas, st, sc,
                                                 static_cast<__nv_bfloat16*>(dq), ld_dq);
  };
  const cudaError_t e = s.d == 128 ? run(std::integral_constant<int, 128>{})
                                   : run(std::integral_constant<int, 64>{});
  return e == cudaSuccess ? VDN_OK : VDN_ERR_CUDA;
}

}  // extern "C"
