// Query/key preparation: per-head norm of queries and keys with the rotary
// position rotation in the same pass, its gradients, and the rotation alone.
//
//   r   = (c sum_i x_i^2 + eps)^-1/2,  c = 1/d (RMS) or 1 (unit length), r = 1 without a norm
//   n_i = x_i r w_i
//   y   = R(p) n: pair (a, b) of the first rot columns turns by the angle p f_pair,
//         (a cos - b sin, b cos + a sin), cos and sin times `scale`; the rest passes through
// With g = R(p)^T dy (the same pass with -sin):
//   dw_i = sum over rows and heads of g_i x_i r
//   dx_i = r w_i g_i - x_i r^3 c sum_j g_j w_j x_j
//
// Angles.  A pair's frequency is held as a 64-bit fraction of a turn per
// position (turns x 2^64); position times it, modulo 2^64, is the phase with
// whole turns dropped exactly, whatever the position's size or sign, for one
// integer multiply.  Its top 32 bits go to sincospi.
//
// Bound: memory.  Each element is read and written once; a block computes the
// cos/sin of its few rows once into shared memory and all heads of those rows
// use them (64 sines a row against 48 x 128 elements at 24 + 24 heads).  One
// thread holds both members of its pairs (two vectors of V elements), so the
// rotation needs no exchange; the head's sum is a shuffle over its lanes.  A
// thread keeps its row and its columns and walks the heads, so the turns and
// the norm's weights stay in registers (read again for every head from shared
// memory and L1: 42336 rows of 24 + 24 heads of 128 took 234 us).  What keeps
// the memory busy is bytes in flight: loads go through a cp.async ring in
// shared memory in which every thread has its own slots (no barrier), so they
// cost no registers (prefetched into registers: 208 us, then 179 us; 175 to
// 194 us by the box, 5.4 to 5.9 TB/s).
// Blocks that walk row groups in turn instead of one group a block: 207 us.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "common.cuh"
#include "ptx.cuh"

namespace vdn {

namespace {

constexpr int kThreads = 256;
constexpr int kStages = 3;           // forward: heads in the ring (x: two vectors)
constexpr int kBwdStages = 2;        // backward (x and dy: four)
// its ring of 16-byte vectors and the turns of 16 rows of 128 pairs
constexpr int kBwdSmemMax = kBwdStages * 4 * kThreads * 16 + 16 * 128 * 8;
constexpr int kMaxBwdBlocks = 1024;  // rows of the weight-gradient partials

struct Side {            // queries or keys
  const void* x;
  const void* g;         // backward: gradient of the output
  void* y;               // forward: output; backward: dx
  const float* w;        // norm weight [d] or null
  int64_t ldx, ldg, ldy;
  int heads;
  int norm;              // VDN_NORM_*
};

struct RopeArgs {
  Side s[2];             // queries, keys
  int64_t rows;
  int64_t pos_stride;    // elements between the axes of `positions`
  const int32_t* positions;  // [axes, rows] or null: the row index on every axis
  const uint64_t* phase;
  int d, rot;
  int sec1, sec2, sec3;  // first pair of axes 1, 2, 3
  int rows_per_block;    // a power of two; in the backward pass the queries' blocks',
  int rows_per_block_k;  // and the keys'
  int lanes;             // lanes of a head (power of two)
  float scale, sin_sign, eps;
  float* partial;        // backward: [blocks, d] weight-gradient partials
  int blocks_q;          // backward: blocks that work on queries (the rest on keys)
  uint32_t* status;      // backward: device status word
};

template <int WORDS>
__device__ __forceinline__ void load_words(const void* p, uint32_t (&u)[WORDS]) {
  if constexpr (WORDS == 4) {
    const uint4 v = *static_cast<const uint4*>(p);
    u[0] = v.x, u[1] = v.y, u[2] = v.z, u[3] = v.w;
  } else {
    const uint2 v = *static_cast<const uint2*>(p);
    u[0] = v.x, u[1] = v.y;
  }
}

template <int WORDS>
__device__ __forceinline__ void store_words(void* p, const uint32_t (&u)[WORDS]) {
  if constexpr (WORDS == 4)
    *static_cast<uint4*>(p) = make_uint4(u[0], u[1], u[2], u[3]);
  else
    *static_cast<uint2*>(p) = make_uint2(u[0], u[1]);
}

// Asynchronous copy of one vector into this thread's slot of the ring.
template <int WORDS>
__device__ __forceinline__ void copy_async(uint32_t dst, const void* src) {
  if constexpr (WORDS == 4)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}

__device__ __forceinline__ void copy_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}

template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

template <typename T, int V, int WORDS>
__device__ __forceinline__ void unpack(const uint32_t (&u)[WORDS], float (&f)[V]) {
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int e = 0; e < V; ++e) f[e] = __uint_as_float(u[e]);
  } else {
#pragma unroll
    for (int e = 0; e < V; e += 2) {
      float2 v;
      if constexpr (std::is_same<T, __half>::value)
        v = __half22float2(*reinterpret_cast<const __half2*>(&u[e / 2]));
      else
        v = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&u[e / 2]));
      f[e] = v.x, f[e + 1] = v.y;
    }
  }
}

template <typename T, int V, int WORDS>
__device__ __forceinline__ void pack(const float (&f)[V], uint32_t (&u)[WORDS]) {
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int e = 0; e < V; ++e) u[e] = __float_as_uint(f[e]);
  } else {
#pragma unroll
    for (int e = 0; e < V; e += 2) {
      if constexpr (std::is_same<T, __half>::value) {
        const __half2 h = __floats2half2_rn(f[e], f[e + 1]);
        u[e / 2] = *reinterpret_cast<const uint32_t*>(&h);
      } else {
        const __nv_bfloat162 h = __floats2bfloat162_rn(f[e], f[e + 1]);
        u[e / 2] = *reinterpret_cast<const uint32_t*>(&h);
      }
    }
  }
}

// cos/sin of rows [r0, r0 + n) into shared memory, [row][pair].
__device__ __forceinline__ void fill_turns(const RopeArgs& a, float2* cs, int64_t r0, int n) {
  const int pairs = a.rot / 2;
  for (int i = threadIdx.x; i < n * pairs; i += kThreads) {
    const int row = i / pairs, pair = i - row * pairs;
    const int axis = (pair >= a.sec1) + (pair >= a.sec2) + (pair >= a.sec3);
    const int64_t pos = a.positions != nullptr ? a.positions[axis * a.pos_stride + r0 + row]
                                               : r0 + row;
    const uint64_t turn = static_cast<uint64_t>(pos) * a.phase[pair];
    float sn, cn;
    sincospif(static_cast<float>(static_cast<int32_t>(turn >> 32)) * 4.656612873077393e-10f, &sn,
              &cn);  // 2^-31: half turns
    cs[row * pairs + pair] = make_float2(cn * a.scale, sn * a.scale * a.sin_sign);
  }
}

// The turns of a unit's pairs in one row, (cos, sin, cos, sin) of two pairs a
// float4: pair e of the half layout joins element e of both vectors; in the
// interleaved layout the first V / 2 pairs lie in the vector at column ca, the
// others in that at cb.
template <int V, bool INTER>
__device__ __forceinline__ void load_turns(const float2* cs, int rot, int ca, int cb,
                                           float4 (&c)[V / 2]) {
  const float4* p = reinterpret_cast<const float4*>(cs);
#pragma unroll
  for (int j = 0; j < V / 2; ++j) {
    const int col = INTER ? (j < V / 4 ? ca + 4 * j : cb + 4 * j - V) : ca;
    if (col < (INTER ? rot : rot / 2)) c[j] = INTER ? p[col / 4] : p[ca / 2 + j];
  }
}

// `both`: the vector at cb turns too (in the half layout it always does); one
// that passes through is left alone, since x * 1 - y * 0 is not x beside an
// infinite y.
template <int V, bool INTER>
__device__ __forceinline__ void turn_unit(const float4 (&c)[V / 2], bool both, float (&fa)[V],
                                          float (&fb)[V]) {
  auto turn = [](float& x, float& y, float cn, float sn) {
    const float t = x * cn - y * sn;
    y = y * cn + x * sn;
    x = t;
  };
#pragma unroll
  for (int j = 0; j < V / 2; ++j) {
    if constexpr (INTER) {
      if (j >= V / 4 && !both) break;
      float(&f)[V] = j < V / 4 ? fa : fb;
      const int e = (4 * j) % V;
      turn(f[e], f[e + 1], c[j].x, c[j].y);
      turn(f[e + 2], f[e + 3], c[j].z, c[j].w);
    } else {
      turn(fa[2 * j], fb[2 * j], c[j].x, c[j].y);
      turn(fa[2 * j + 1], fb[2 * j + 1], c[j].z, c[j].w);
    }
  }
}

__device__ __forceinline__ float lane_sum(float v, int lanes) {
  for (int o = lanes >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

template <int V>
__device__ __forceinline__ void load_weight(const float* w, int col, float (&f)[V]) {
  if (w == nullptr) {
#pragma unroll
    for (int e = 0; e < V; ++e) f[e] = 1.f;
    return;
  }
#pragma unroll
  for (int e = 0; e < V; e += 4) {
    const float4 v = *reinterpret_cast<const float4*>(w + col + e);
    f[e] = v.x, f[e + 1] = v.y, f[e + 2] = v.z, f[e + 3] = v.w;
  }
}

// Both vectors' stores inside their tensor (debug builds; the forward calls
// have no workspace to record a miss in and only skip it)?
template <int V>
__device__ __forceinline__ bool stores_in_bounds(const RopeArgs& a, const Side& s,
                                                 uint32_t* status, int64_t r, int64_t c0,
                                                 int64_t c1) {
  const int64_t cols = static_cast<int64_t>(s.heads) * a.d;
  return in_bounds(status, r, a.rows, c0, V, cols) && in_bounds(status, r, a.rows, c1, V, cols);
}

// Columns of unit u's two vectors: side by side with the neighbouring lanes'
// in both, and in the half layout the two members of its pairs.
template <int V, bool INTER>
__device__ __forceinline__ void unit_columns(int u, int d, int rot, int& ca, int& cb) {
  ca = u * V;
  if (INTER) {
    cb = d / 2 + u * V;
  } else if (2 * ca < rot) {
    cb = rot / 2 + ca;
  } else {  // the columns that pass through, in two runs of their own
    ca += rot / 2;
    cb = ca + (d - rot) / 2;
  }
}

template <typename T, int V, bool INTER, bool NORM>
__global__ void __launch_bounds__(kThreads, NORM ? 3 : 4)
    rope_kernel(const __grid_constant__ RopeArgs a) {
  extern __shared__ float4 smem_f4[];
  constexpr int W = V * static_cast<int>(sizeof(T)) / 4;
  constexpr int SLOT = kThreads * W * 4;  // bytes of one vector of all threads
  uint8_t* ring = reinterpret_cast<uint8_t*>(smem_f4);
  float2* cs = reinterpret_cast<float2*>(ring + kStages * 2 * SLOT);
  const int64_t r0 = static_cast<int64_t>(blockIdx.x) * a.rows_per_block;
  const int n = static_cast<int>(min(static_cast<int64_t>(a.rows_per_block), a.rows - r0));
  // thread: unit u of a head; its row, and every `step`-th head from `first`
  const int u = threadIdx.x & (a.lanes - 1), slot = threadIdx.x / a.lanes;
  const int step = kThreads / a.lanes / a.rows_per_block;
  const int row = slot / step, first = slot & (step - 1);  // neighbouring heads side by side
  const bool live = row < n && u < a.d / (2 * V);
  int ca, cb;
  unit_columns<V, INTER>(u, a.d, a.rot, ca, cb);
  const bool turned = ca < (INTER ? a.rot : a.rot / 2), both = !INTER || cb < a.rot;
  // passes over the heads of the queries, then of the keys
  const int passes_q = (a.s[0].heads + step - 1) / step;
  const int passes = passes_q + (a.s[1].heads + step - 1) / step;
  const uint32_t mine = smem_u32(ring) + threadIdx.x * W * 4;
  auto fetch = [&](int k) {
    const bool key = k >= passes_q;
    const Side& s = a.s[key];
    const int h = (key ? k - passes_q : k) * step + first;
    if (k < passes && live && h < s.heads) {
      const T* src = static_cast<const T*>(s.x) + (r0 + row) * s.ldx +
                     static_cast<int64_t>(h) * a.d;
      const uint32_t dst = mine + k % kStages * 2 * SLOT;
      copy_async<W>(dst, src + ca);
      copy_async<W>(dst + SLOT, src + cb);
    }
    copy_commit();
  };
  // the first loads are in flight while the block computes its angles
#pragma unroll
  for (int k = 0; k < kStages - 1; ++k) fetch(k);
  float4 turns[V / 2];
  if (a.rot > 0) {
    fill_turns(a, cs, r0, n);
    __syncthreads();
    if (live && turned) load_turns<V, INTER>(cs + row * (a.rot / 2), a.rot, ca, cb, turns);
  }
  float wa[V], wb[V];
  // the trip count is the block's, since the sums are warp-collective
  for (int k = 0; k < passes; ++k) {
    const bool key = k >= passes_q;
    const Side& s = a.s[key];
    const int h = (key ? k - passes_q : k) * step + first;
    const bool on = live && h < s.heads;
    if (NORM && live && (k == 0 || k == passes_q)) {
      load_weight<V>(s.w, ca, wa);
      load_weight<V>(s.w, cb, wb);
    }
    fetch(k + kStages - 1);
    copy_wait<kStages - 1>();
    float fa[V], fb[V];
    if (on) {
      uint32_t xa[W], xb[W];
      const uint8_t* src = ring + k % kStages * 2 * SLOT + threadIdx.x * W * 4;
      load_words<W>(src, xa);
      load_words<W>(src + SLOT, xb);
      unpack<T, V, W>(xa, fa);
      unpack<T, V, W>(xb, fb);
    } else {
#pragma unroll
      for (int e = 0; e < V; ++e) fa[e] = fb[e] = 0.f;
    }
    if (NORM && s.norm != VDN_NORM_NONE) {
      float q = 0.f;
#pragma unroll
      for (int e = 0; e < V; ++e) q += fa[e] * fa[e] + fb[e] * fb[e];
      q = lane_sum(q, a.lanes);
      const float r =
          rsqrtf(q * (s.norm == VDN_NORM_RMS ? 1.f / static_cast<float>(a.d) : 1.f) + a.eps);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        fa[e] *= r * wa[e];
        fb[e] *= r * wb[e];
      }
    }
    if (!on) continue;
    if (turned) turn_unit<V, INTER>(turns, both, fa, fb);
    uint32_t oa[W], ob[W];
    pack<T, V, W>(fa, oa);
    pack<T, V, W>(fb, ob);
    const int64_t col = static_cast<int64_t>(h) * a.d;
    T* dst = static_cast<T*>(s.y) + (r0 + row) * s.ldy + col;
    if (!stores_in_bounds<V>(a, s, nullptr, r0 + row, col + ca, col + cb)) continue;
    store_words<W>(dst + ca, oa);
    store_words<W>(dst + cb, ob);
  }
}

// Gradients.  Each block works on queries or on keys, walks row groups with
// the grid's stride and keeps its threads' share of dw (always the same 2 V
// columns) in registers; the block's sum goes to its row of `partial`, and
// rope_dw_kernel adds the rows in a fixed order.
template <typename T, int V, bool INTER>
__global__ void __launch_bounds__(kThreads, 2) rope_backward_kernel(
    const __grid_constant__ RopeArgs a) {
  extern __shared__ float4 smem_f4[];
  constexpr int W = V * static_cast<int>(sizeof(T)) / 4;
  constexpr int SLOT = kThreads * W * 4;  // bytes of one vector of all threads
  uint8_t* ring = reinterpret_cast<uint8_t*>(smem_f4);
  float2* cs = reinterpret_cast<float2*>(ring + kBwdStages * 4 * SLOT);
  after_allow();  // rope_dw_kernel
  const bool key = static_cast<int>(blockIdx.x) >= a.blocks_q;
  const Side& s = a.s[key ? 1 : 0];
  const int blk = key ? blockIdx.x - a.blocks_q : blockIdx.x;
  const int nblk = key ? gridDim.x - a.blocks_q : a.blocks_q;
  const int u = threadIdx.x & (a.lanes - 1), slot = threadIdx.x / a.lanes;
  const int R = key ? a.rows_per_block_k : a.rows_per_block;
  const int step = kThreads / a.lanes / R;
  const int row = slot / step, first = slot & (step - 1);  // neighbouring heads side by side
  const bool unit = u < a.d / (2 * V);
  const float c = s.norm == VDN_NORM_RMS ? 1.f / static_cast<float>(a.d) : 1.f;
  int ca, cb;
  unit_columns<V, INTER>(u, a.d, a.rot, ca, cb);
  const bool turned = ca < (INTER ? a.rot : a.rot / 2), both = !INTER || cb < a.rot;
  float wa[V], wb[V], da[V], db[V];
#pragma unroll
  for (int e = 0; e < V; ++e) wa[e] = wb[e] = 1.f, da[e] = db[e] = 0.f;
  if (unit) {
    load_weight<V>(s.w, ca, wa);
    load_weight<V>(s.w, cb, wb);
  }
  // one run of passes over the heads of the block's row groups, so that the
  // ring does not drain between groups
  const int64_t groups = (a.rows + R - 1) / R;
  const int64_t my_groups = blk < groups ? (groups - blk + nblk - 1) / nblk : 0;
  const int passes = (s.heads + step - 1) / step;
  const uint32_t mine = smem_u32(ring) + threadIdx.x * W * 4;
  int64_t fg = 0;  // the next fetch: group (of this block's), pass and stage
  int fk = 0, fs = 0;
  auto fetch = [&] {
    const int64_t r = (blk + fg * nblk) * R + row;
    const int h = fk * step + first;
    if (fg < my_groups && unit && r < a.rows && h < s.heads) {
      const int64_t off = static_cast<int64_t>(h) * a.d;
      const T* x = static_cast<const T*>(s.x) + r * s.ldx + off;
      const T* g = static_cast<const T*>(s.g) + r * s.ldg + off;
      const uint32_t dst = mine + fs * 4 * SLOT;
      copy_async<W>(dst, x + ca);
      copy_async<W>(dst + SLOT, x + cb);
      copy_async<W>(dst + 2 * SLOT, g + ca);
      copy_async<W>(dst + 3 * SLOT, g + cb);
    }
    copy_commit();
    if (++fk == passes) fk = 0, ++fg;
    if (++fs == kBwdStages) fs = 0;
  };
#pragma unroll
  for (int k = 0; k < kBwdStages - 1; ++k) fetch();
  int stage = 0;
  for (int64_t group = 0; group < my_groups; ++group) {
    const int64_t r0 = (blk + group * nblk) * R;
    const int n = static_cast<int>(min(static_cast<int64_t>(R), a.rows - r0));
    const bool live = unit && row < n;
    float4 turns[V / 2];
    if (a.rot > 0) {
      __syncthreads();  // the previous group's turns have been read
      fill_turns(a, cs, r0, n);
      __syncthreads();
      if (live && turned) load_turns<V, INTER>(cs + row * (a.rot / 2), a.rot, ca, cb, turns);
    }
    for (int k = 0; k < passes; ++k) {
      const int h = k * step + first;
      const bool on = live && h < s.heads;
      fetch();
      copy_wait<kBwdStages - 1>();
      float fxa[V], fxb[V], fga[V], fgb[V];
      if (on) {
        uint32_t v[W];
        const uint8_t* src = ring + stage * 4 * SLOT + threadIdx.x * W * 4;
        load_words<W>(src, v);
        unpack<T, V, W>(v, fxa);
        load_words<W>(src + SLOT, v);
        unpack<T, V, W>(v, fxb);
        load_words<W>(src + 2 * SLOT, v);
        unpack<T, V, W>(v, fga);
        load_words<W>(src + 3 * SLOT, v);
        unpack<T, V, W>(v, fgb);
        if (turned) turn_unit<V, INTER>(turns, both, fga, fgb);
      } else {
#pragma unroll
        for (int e = 0; e < V; ++e) fxa[e] = fxb[e] = fga[e] = fgb[e] = 0.f;
      }
      if (++stage == kBwdStages) stage = 0;
      float r = 1.f, back = 0.f;
      if (s.norm != VDN_NORM_NONE) {
        float q = 0.f, t = 0.f;
#pragma unroll
        for (int e = 0; e < V; ++e) {
          q += fxa[e] * fxa[e] + fxb[e] * fxb[e];
          t += fga[e] * wa[e] * fxa[e] + fgb[e] * wb[e] * fxb[e];
        }
        q = lane_sum(q, a.lanes);
        t = lane_sum(t, a.lanes);
        r = rsqrtf(q * c + a.eps);
        back = r * r * r * c * t;
      }
      if (on) {
        float oa[V], ob[V];
#pragma unroll
        for (int e = 0; e < V; ++e) {
          const float ra = r * fga[e], rb = r * fgb[e];
          da[e] += ra * fxa[e];
          db[e] += rb * fxb[e];
          oa[e] = ra;
          ob[e] = rb;
          if (s.norm != VDN_NORM_NONE) {
            oa[e] = ra * wa[e] - fxa[e] * back;
            ob[e] = rb * wb[e] - fxb[e] * back;
          }
        }
        uint32_t pa[W], pb[W];
        pack<T, V, W>(oa, pa);
        pack<T, V, W>(ob, pb);
        const int64_t col = static_cast<int64_t>(h) * a.d;
        T* dst = static_cast<T*>(s.y) + (r0 + row) * s.ldy + col;
        if (!stores_in_bounds<V>(a, s, a.status, r0 + row, col + ca, col + cb)) continue;
        store_words<W>(dst + ca, pa);
        store_words<W>(dst + cb, pb);
      }
    }
  }
  if (a.partial == nullptr) return;
  __syncthreads();
  float* sum = reinterpret_cast<float*>(smem_f4);  // [slots][d]
  const int slots = kThreads / a.lanes;
  if (unit) {
#pragma unroll
    for (int e = 0; e < V; ++e) {
      sum[slot * a.d + ca + e] = da[e];
      sum[slot * a.d + cb + e] = db[e];
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < a.d; i += kThreads) {
    float t = 0.f;
    for (int j = 0; j < slots; ++j) t += sum[j * a.d + i];
    a.partial[static_cast<int64_t>(blockIdx.x) * a.d + i] = t;
  }
}

// dw[i] = sum of the partials' rows, in a fixed order: a block takes 32
// columns, warp w every 32nd row from row w.
__global__ void __launch_bounds__(1024) rope_dw_kernel(const float* partial, int d, int blocks_q,
                                                       int blocks, float* dwq, float* dwk) {
  after_wait();
  __shared__ float sums[32][33];
  const bool key = blockIdx.y == 1;
  float* dw = key ? dwk : dwq;
  if (dw == nullptr) return;
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31, col = blockIdx.x * 32 + lane;
  const int b1 = key ? blocks : blocks_q;
  float t = 0.f;
#pragma unroll 4
  for (int b = (key ? blocks_q : 0) + w; b < b1; b += 32)
    t += col < d ? partial[static_cast<int64_t>(b) * d + col] : 0.f;
  sums[w][lane] = t;
  __syncthreads();
  t = lane_sum(sums[lane][w], 32);  // column w of the block
  if (lane == 0 && blockIdx.x * 32 + w < d) dw[blockIdx.x * 32 + w] = t;
}

bool al(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) % n) == 0; }

int pow2_at_least(int n) {
  int p = 1;
  while (p < n) p *= 2;
  return p;
}

// V = 8 for 16-bit types where the vectors allow it (16-byte loads; gradients of
// 10080 rows of 24 + 24 heads of 128: 105 us, and 140 with V = 4), else 4.
int vector_width(int dtype, int d, int rot) {
  return dtype != VDN_DTYPE_F32 && d % 16 == 0 && rot % 16 == 0 ? 8 : 4;
}

template <class F>
cudaError_t dispatch(int dtype, int v, bool inter, F&& f) {
  auto on_layout = [&](auto t, auto w) {
    return inter ? f(t, w, std::true_type{}) : f(t, w, std::false_type{});
  };
  using V4 = std::integral_constant<int, 4>;
  using V8 = std::integral_constant<int, 8>;
  switch (dtype) {
    case VDN_DTYPE_BF16:
      return v == 8 ? on_layout(__nv_bfloat16{}, V8{}) : on_layout(__nv_bfloat16{}, V4{});
    case VDN_DTYPE_F16: return v == 8 ? on_layout(__half{}, V8{}) : on_layout(__half{}, V4{});
    default: return on_layout(float{}, V4{});
  }
}

// Host checks shared by the entry points; fills the plan's part of `a`.
vdn_status take_plan(const vdn_rope_plan* plan, int64_t rows, const int32_t* positions,
                     int64_t pos_stride, int dtype, RopeArgs* a) {
  if (plan == nullptr || rows < 0 || rows >= (int64_t(1) << 31)) return VDN_ERR_INVALID_ARG;
  if (dtype < VDN_DTYPE_BF16 || dtype > VDN_DTYPE_F32) return VDN_ERR_INVALID_ARG;
  if (plan->head_dim < 1 || plan->rot_dim < 0 || plan->rot_dim > plan->head_dim)
    return VDN_ERR_INVALID_ARG;
  if (plan->head_dim % 8 || plan->head_dim > 256 || plan->rot_dim % 8) return VDN_ERR_UNSUPPORTED;
  if (plan->layout != VDN_ROPE_HALF && plan->layout != VDN_ROPE_INTERLEAVED)
    return VDN_ERR_INVALID_ARG;
  if (plan->rot_dim > 0) {
    if (plan->n_axes < 1 || plan->n_axes > 4 || plan->phase == nullptr || !al(plan->phase, 8))
      return VDN_ERR_INVALID_ARG;
    int64_t sum = 0;
    for (int i = 0; i < plan->n_axes; ++i) {
      if (plan->section_pairs[i] < 0) return VDN_ERR_INVALID_ARG;
      sum += plan->section_pairs[i];
    }
    if (sum != plan->rot_dim / 2) return VDN_ERR_INVALID_ARG;
    if (positions != nullptr && (!al(positions, 4) ||
                                 (plan->n_axes > 1 && pos_stride != 0 && pos_stride < rows)))
      return VDN_ERR_INVALID_ARG;
  }
  const int big = 1 << 30;
  a->sec1 = plan->n_axes > 1 ? plan->section_pairs[0] : big;
  a->sec2 = plan->n_axes > 2 ? a->sec1 + plan->section_pairs[1] : big;
  a->sec3 = plan->n_axes > 3 ? a->sec2 + plan->section_pairs[2] : big;
  a->rows = rows;
  a->pos_stride = plan->n_axes > 1 ? pos_stride : 0;
  a->positions = positions;
  a->phase = plan->phase;
  a->d = plan->head_dim;
  a->rot = plan->rot_dim;
  a->scale = plan->scale;
  a->lanes = pow2_at_least(a->d / (2 * vector_width(dtype, a->d, a->rot)));
  a->partial = nullptr;
  a->blocks_q = 0;
  return VDN_OK;
}

vdn_status check_side(const Side& s, int d, int64_t rows, bool backward) {
  if (s.heads < 1 || static_cast<int64_t>(s.heads) * d >= (int64_t(1) << 24))
    return VDN_ERR_INVALID_ARG;
  if (s.norm < VDN_NORM_NONE || s.norm > VDN_NORM_L2) return VDN_ERR_INVALID_ARG;
  if ((s.norm == VDN_NORM_NONE && s.w != nullptr) || (s.w != nullptr && !al(s.w, 16)))
    return VDN_ERR_INVALID_ARG;
  const int64_t D = static_cast<int64_t>(s.heads) * d;
  auto ld_bad = [&](int64_t ld) { return ld < D || ld % 8 != 0; };
  auto ptr_bad = [&](const void* p) { return (p == nullptr && rows > 0) || !al(p, 16); };
  if (ptr_bad(s.x) || ptr_bad(s.y) || ld_bad(s.ldx) || ld_bad(s.ldy)) return VDN_ERR_INVALID_ARG;
  if (backward && (ptr_bad(s.g) || ld_bad(s.ldg))) return VDN_ERR_INVALID_ARG;
  return VDN_OK;
}

// Rows of a block (a power of two): of its slots (a head's lanes each) so many
// take different rows and the rest different heads that the fewest are left
// over in the last pass over the heads; of equal choices the one nearest 8
// from below, since a block's start-up is paid once for its rows (24 + 24 heads
// of 128, 42336 rows: 350 us with one row, 268 with 2, 209 with 4, 194 with
// 8), and fewer rows where the GPU would have less than two blocks an SM.
int rows_per_block(int64_t rows, int lanes, int heads0, int heads1, int sms) {
  const int slots = kThreads / lanes;
  int best = 1, least = 1 << 30;
  for (int n = 1; n <= slots && n <= 16; n *= 2) {
    const int step = slots / n;  // heads a pass
    const int cost = ((heads0 + step - 1) / step + (heads1 + step - 1) / step) * step;
    if (cost < least || (cost == least && n <= 8)) best = n, least = cost;
  }
  while (best > 1 && (rows + best - 1) / best < 2 * sms) best /= 2;
  return best;
}

// Rows of a group in the backward pass: the fewest passes for the block with
// the most groups, a group's turns and barriers counted as half a pass.
int backward_rows(int64_t rows, int lanes, int heads, int blocks) {
  const int slots = kThreads / lanes;
  int best = 1;
  int64_t least = int64_t(1) << 62;
  for (int n = 1; n <= slots && n <= 16; n *= 2) {
    const int step = slots / n;  // heads a pass
    const int64_t groups = ((rows + n - 1) / n + blocks - 1) / blocks;
    const int64_t cost = groups * (2 * ((heads + step - 1) / step) + 1);
    if (cost < least) best = n, least = cost;
  }
  return best;
}

vdn_status launch_forward(RopeArgs& a, int dtype, int layout, cudaStream_t stream) {
  if (a.rows == 0) return VDN_OK;
  a.rows_per_block = rows_per_block(a.rows, a.lanes, a.s[0].heads, a.s[1].heads,
                                    sm_count_of_current_device());
  const int vec = vector_width(dtype, a.d, a.rot) * (dtype == VDN_DTYPE_F32 ? 4 : 2);
  const int smem = kStages * 2 * kThreads * vec + a.rows_per_block * a.rot / 2 * 8;
  const int64_t grid = (a.rows + a.rows_per_block - 1) / a.rows_per_block;
  const cudaError_t e = dispatch(
      dtype, vector_width(dtype, a.d, a.rot), layout == VDN_ROPE_INTERLEAVED,
      [&](auto t, auto v, auto inter) {
        using T = decltype(t);
        constexpr int V = decltype(v)::value;
        constexpr bool I = decltype(inter)::value;
        if (a.s[0].norm | a.s[1].norm)
          rope_kernel<T, V, I, true><<<static_cast<unsigned>(grid), kThreads, smem, stream>>>(a);
        else
          rope_kernel<T, V, I, false><<<static_cast<unsigned>(grid), kThreads, smem, stream>>>(a);
        return cudaGetLastError();
      });
  return e == cudaSuccess ? VDN_OK : VDN_ERR_CUDA;
}

}  // namespace

}  // namespace vdn

using namespace vdn;

extern "C" {

vdn_status vdn_rope(const vdn_rope_plan* plan, int dtype, int64_t rows, int H, const void* x,
                    int64_t ld, const int32_t* positions, int64_t pos_stride, int inverse,
                    void* out, int64_t ld_out, void* stream) {
  NvtxRange nvtx("vdn_rope");
  RopeArgs a{};
  vdn_status r = take_plan(plan, rows, positions, pos_stride, dtype, &a);
  if (r != VDN_OK) return r;
  a.s[0] = Side{x, nullptr, out, nullptr, ld, 0, ld_out, H, VDN_NORM_NONE};
  a.s[1] = Side{};
  if ((r = check_side(a.s[0], a.d, rows, false)) != VDN_OK) return r;
  a.sin_sign = inverse ? -1.f : 1.f;
  return launch_forward(a, dtype, plan->layout, static_cast<cudaStream_t>(stream));
}

vdn_status vdn_qk_norm_rope(const vdn_rope_plan* plan, int dtype, int64_t rows, int H, int H_kv,
                            const void* q, int64_t ld_q, const void* k, int64_t ld_k, int q_norm,
                            int k_norm, const float* wq, const float* wk, float eps,
                            const int32_t* positions, int64_t pos_stride, void* q_out,
                            int64_t ld_qo, void* k_out, int64_t ld_ko, void* stream) {
  NvtxRange nvtx("vdn_qk_norm_rope");
  RopeArgs a{};
  vdn_status r = take_plan(plan, rows, positions, pos_stride, dtype, &a);
  if (r != VDN_OK) return r;
  a.s[0] = Side{q, nullptr, q_out, wq, ld_q, 0, ld_qo, H, q_norm};
  a.s[1] = Side{k, nullptr, k_out, wk, ld_k, 0, ld_ko, H_kv, k_norm};
  for (const Side& s : a.s)
    if ((r = check_side(s, a.d, rows, false)) != VDN_OK) return r;
  if (!(eps >= 0.f)) return VDN_ERR_INVALID_ARG;
  a.eps = eps;
  a.sin_sign = 1.f;
  return launch_forward(a, dtype, plan->layout, static_cast<cudaStream_t>(stream));
}

size_t vdn_qk_norm_rope_backward_workspace(int head_dim) {
  if (head_dim < 1 || head_dim > 256) return 0;
  return kStatusBytes + static_cast<size_t>(kMaxBwdBlocks) * head_dim * sizeof(float);
}

vdn_status vdn_qk_norm_rope_backward(const vdn_rope_plan* plan, int dtype, int64_t rows, int H,
                                     int H_kv, const void* q, int64_t ld_q, const void* k,
                                     int64_t ld_k, int q_norm, int k_norm, const float* wq,
                                     const float* wk, float eps, const int32_t* positions,
                                     int64_t pos_stride, const void* dq_out, int64_t ld_dqo,
                                     const void* dk_out, int64_t ld_dko, void* dq, int64_t ld_dq,
                                     void* dk, int64_t ld_dk, float* dwq, float* dwk, void* ws,
                                     size_t ws_bytes, void* stream) {
  NvtxRange nvtx("vdn_qk_norm_rope_backward");
  RopeArgs a{};
  vdn_status r = take_plan(plan, rows, positions, pos_stride, dtype, &a);
  if (r != VDN_OK) return r;
  a.s[0] = Side{q, dq_out, dq, wq, ld_q, ld_dqo, ld_dq, H, q_norm};
  a.s[1] = Side{k, dk_out, dk, wk, ld_k, ld_dko, ld_dk, H_kv, k_norm};
  for (const Side& s : a.s)
    if ((r = check_side(s, a.d, rows, true)) != VDN_OK) return r;
  if (!(eps >= 0.f) || (dwq && !al(dwq, 4)) || (dwk && !al(dwk, 4))) return VDN_ERR_INVALID_ARG;
  if ((dwq && q_norm == VDN_NORM_NONE) || (dwk && k_norm == VDN_NORM_NONE))
    return VDN_ERR_INVALID_ARG;
  if (ws == nullptr || !al(ws, 256) || ws_bytes < vdn_qk_norm_rope_backward_workspace(a.d))
    return VDN_ERR_WORKSPACE;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  a.eps = eps;
  a.sin_sign = -1.f;
  a.status = static_cast<uint32_t*>(ws);
  a.partial = dwq || dwk
                  ? reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + kStatusBytes)
                  : nullptr;
  const int sms = sm_count_of_current_device();
  // two blocks an SM run at a time (125 registers at most; three, with 85, spill: 97 us
  // for 10080 rows of 24 + 24 heads of 128 instead of 80; packed fp32
  // arithmetic changes nothing); shared out by heads, at most one a row
  const int most = 2 * sms < kMaxBwdBlocks ? 2 * sms : kMaxBwdBlocks - 1;  // each side has one
  auto share = [&](int heads) {
    int64_t n = static_cast<int64_t>(most) * heads / (H + H_kv);
    n = n > rows ? rows : n;
    return static_cast<int>(n < 1 ? 1 : n);
  };
  a.blocks_q = share(H);
  const int blocks = a.blocks_q + share(H_kv);
  a.rows_per_block = backward_rows(rows, a.lanes, H, a.blocks_q);
  a.rows_per_block_k = backward_rows(rows, a.lanes, H_kv, blocks - a.blocks_q);
  const int vec = vector_width(dtype, a.d, a.rot) * (dtype == VDN_DTYPE_F32 ? 4 : 2);
  const int most_rows = a.rows_per_block > a.rows_per_block_k ? a.rows_per_block : a.rows_per_block_k;
  const int ring = kBwdStages * 4 * kThreads * vec + most_rows * a.rot / 2 * 8;
  const int sums = kThreads / a.lanes * a.d * 4;
  const cudaError_t e = dispatch(
      dtype, vector_width(dtype, a.d, a.rot), plan->layout == VDN_ROPE_INTERLEAVED,
      [&](auto t, auto v, auto inter) {
        const auto kernel =
            rope_backward_kernel<decltype(t), decltype(v)::value, decltype(inter)::value>;
        const int smem = ring > sums ? ring : sums;
        static std::atomic<uint64_t> smem_set{0};  // one for each kernel
        if (cudaError_t e = set_smem_once(kernel, kBwdSmemMax, smem_set)) return e;
        kernel<<<blocks, kThreads, smem, st>>>(a);
        return cudaGetLastError();
      });
  if (e != cudaSuccess) return VDN_ERR_CUDA;
  if (a.partial != nullptr) {
    if (launch_after(rope_dw_kernel, dim3((a.d + 31) / 32, 2), 1024, 0, st,
                     static_cast<const float*>(a.partial), a.d, a.blocks_q, blocks, dwq, dwk) !=
        cudaSuccess)
      return VDN_ERR_CUDA;
  }
  return VDN_OK;
}

}  // extern "C"
