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
// rotation needs no exchange; the head's sum is a shuffle over its lanes.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "common.cuh"

namespace vdn {

namespace {

constexpr int kThreads = 256;
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
  int rows_per_block;
  int lanes;             // lanes of a head (power of two)
  float scale, sin_sign, eps;
  float* partial;        // backward: [blocks, d] weight-gradient partials
  int blocks_q;          // backward: blocks that work on queries (the rest on keys)
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

// cos/sin of rows [r0, r0 + n) into shared memory.  Unit u's V pairs lie as
// V/2 float4s (cos, sin, cos, sin) at [j][u], so that neighbouring lanes read
// neighbouring 16 bytes.
template <int V>
__device__ __forceinline__ void fill_turns(const RopeArgs& a, float2* cs, int64_t r0, int n) {
  const int pairs = a.rot / 2, units = pairs / V;
  for (int i = threadIdx.x; i < n * pairs; i += kThreads) {
    const int row = i / pairs, pair = i - row * pairs;
    const int axis = (pair >= a.sec1) + (pair >= a.sec2) + (pair >= a.sec3);
    const int64_t pos = a.positions != nullptr ? a.positions[axis * a.pos_stride + r0 + row]
                                               : r0 + row;
    const uint64_t turn = static_cast<uint64_t>(pos) * a.phase[pair];
    float sn, cn;
    sincospif(static_cast<float>(static_cast<int32_t>(turn >> 32)) * 4.656612873077393e-10f, &sn,
              &cn);  // 2^-31: half turns
    const int u = pair / V, e = pair - u * V;
    cs[row * pairs + ((e >> 1) * units + u) * 2 + (e & 1)] =
        make_float2(cn * a.scale, sn * a.scale * a.sin_sign);
  }
}

// Turn the unit's pairs by the row's cos/sin (sign: the sine's factor).
template <int V, bool INTER>
__device__ __forceinline__ void turn_unit(const float2* cs, int u, int units, float (&fa)[V],
                                          float (&fb)[V]) {
  const float4* c4 = reinterpret_cast<const float4*>(cs);
#pragma unroll
  for (int j = 0; j < V / 2; ++j) {
    const float4 c = c4[j * units + u];  // pairs 2j, 2j+1 of the unit
    auto rot2 = [](float& x, float& y, float cn, float sn) {
      const float t = x * cn - y * sn;
      y = y * cn + x * sn;
      x = t;
    };
    if constexpr (INTER) {
      float(&f)[V] = 4 * j < V ? fa : fb;
      const int e = (4 * j) % V;
      rot2(f[e], f[e + 1], c.x, c.y);
      rot2(f[e + 2], f[e + 3], c.z, c.w);
    } else {
      rot2(fa[2 * j], fb[2 * j], c.x, c.y);
      rot2(fa[2 * j + 1], fb[2 * j + 1], c.z, c.w);
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

// Columns of unit u's two vectors.
template <int V, bool INTER>
__device__ __forceinline__ void unit_columns(int u, int d, int rot, int& ca, int& cb) {
  if (!INTER && 2 * V * u < rot) {
    ca = u * V;
    cb = rot / 2 + u * V;
  } else {
    ca = 2 * V * u;
    cb = ca + V;
  }
}

template <typename T, int V, bool INTER>
__global__ void __launch_bounds__(kThreads) rope_kernel(const __grid_constant__ RopeArgs a) {
  extern __shared__ float4 smem_f4[];
  float2* cs = reinterpret_cast<float2*>(smem_f4);
  constexpr int W = V * static_cast<int>(sizeof(T)) / 4;
  const int64_t r0 = static_cast<int64_t>(blockIdx.x) * a.rows_per_block;
  const int n = static_cast<int>(min(static_cast<int64_t>(a.rows_per_block), a.rows - r0));
  const int heads = a.s[0].heads + a.s[1].heads;
  const int total = n * heads;
  const int step = kThreads / a.lanes;
  const int u = threadIdx.x & (a.lanes - 1);
  const bool live = u < a.d / (2 * V);
  const bool turned = 2 * V * u < a.rot;
  int ca, cb;
  unit_columns<V, INTER>(u, a.d, a.rot, ca, cb);

  auto address = [&](int slot, int& row, bool& key) {
    row = slot / heads;
    const int h = slot - row * heads;
    key = h >= a.s[0].heads;
    return static_cast<int64_t>(key ? h - a.s[0].heads : h) * a.d;
  };
  uint32_t na[W], nb[W];
  auto fetch = [&](int slot) {
    if (slot >= total || !live) return;
    int row;
    bool key;
    const int64_t off = address(slot, row, key);
    const Side& s = key ? a.s[1] : a.s[0];
    const T* src = static_cast<const T*>(s.x) + (r0 + row) * s.ldx + off;
    load_words<W>(src + ca, na);
    load_words<W>(src + cb, nb);
  };
  // the first loads are in flight while the block computes its angles
  const int first = threadIdx.x / a.lanes;
  fetch(first);
  if (a.rot > 0) fill_turns<V>(a, cs, r0, n);
  __syncthreads();
  // the trip count is the block's, since the sums are warp-collective
  for (int base = 0; base < total; base += step) {
    const int slot = base + first;
    const bool on = live && slot < total;
    float fa[V], fb[V];
    if (on) {
      unpack<T, V, W>(na, fa);
      unpack<T, V, W>(nb, fb);
    } else {
#pragma unroll
      for (int e = 0; e < V; ++e) fa[e] = fb[e] = 0.f;
    }
    fetch(slot + step);
    int row;
    bool key;
    const int64_t off = address(on ? slot : 0, row, key);
    const Side& s = key ? a.s[1] : a.s[0];
    if (a.s[0].norm | a.s[1].norm) {
      float q = 0.f;
#pragma unroll
      for (int e = 0; e < V; ++e) q += fa[e] * fa[e] + fb[e] * fb[e];
      q = lane_sum(q, a.lanes);
      if (s.norm != VDN_NORM_NONE && on) {
        const float r =
            rsqrtf(q * (s.norm == VDN_NORM_RMS ? 1.f / static_cast<float>(a.d) : 1.f) + a.eps);
        float wa[V], wb[V];
        load_weight<V>(s.w, ca, wa);
        load_weight<V>(s.w, cb, wb);
#pragma unroll
        for (int e = 0; e < V; ++e) {
          fa[e] *= r * wa[e];
          fb[e] *= r * wb[e];
        }
      }
    }
    if (on) {
      if (turned)
        turn_unit<V, INTER>(cs + row * (a.rot / 2), u, a.rot / (2 * V), fa, fb);
      uint32_t oa[W], ob[W];
      pack<T, V, W>(fa, oa);
      pack<T, V, W>(fb, ob);
      T* dst = static_cast<T*>(s.y) + (r0 + row) * s.ldy + off;
      store_words<W>(dst + ca, oa);
      store_words<W>(dst + cb, ob);
    }
  }
}

// Gradients.  Each block works on queries or on keys, walks row groups with
// the grid's stride and keeps its threads' share of dw (always the same 2 V
// columns) in registers; the block's sum goes to its row of `partial`, and
// rope_dw_kernel adds the rows in a fixed order.
template <typename T, int V, bool INTER>
__global__ void __launch_bounds__(kThreads) rope_backward_kernel(
    const __grid_constant__ RopeArgs a) {
  extern __shared__ float4 smem_f4[];
  float2* cs = reinterpret_cast<float2*>(smem_f4);
  constexpr int W = V * static_cast<int>(sizeof(T)) / 4;
  const bool key = static_cast<int>(blockIdx.x) >= a.blocks_q;
  const Side& s = a.s[key ? 1 : 0];
  const int blk = key ? blockIdx.x - a.blocks_q : blockIdx.x;
  const int nblk = key ? gridDim.x - a.blocks_q : a.blocks_q;
  const int step = kThreads / a.lanes;
  const int u = threadIdx.x & (a.lanes - 1);
  const bool live = u < a.d / (2 * V);
  const bool turned = 2 * V * u < a.rot;
  const float c = s.norm == VDN_NORM_RMS ? 1.f / static_cast<float>(a.d) : 1.f;
  int ca, cb;
  unit_columns<V, INTER>(u, a.d, a.rot, ca, cb);
  float wa[V], wb[V], da[V], db[V];
#pragma unroll
  for (int e = 0; e < V; ++e) wa[e] = wb[e] = 1.f, da[e] = db[e] = 0.f;
  if (live) {
    load_weight<V>(s.w, ca, wa);
    load_weight<V>(s.w, cb, wb);
  }
  const int first = threadIdx.x / a.lanes;
  for (int64_t r0 = static_cast<int64_t>(blk) * a.rows_per_block; r0 < a.rows;
       r0 += static_cast<int64_t>(nblk) * a.rows_per_block) {
    const int n = static_cast<int>(min(static_cast<int64_t>(a.rows_per_block), a.rows - r0));
    const int total = n * s.heads;
    uint32_t xa[W], xb[W], ga[W], gb[W];
    auto fetch = [&](int slot) {
      if (slot >= total || !live) return;
      const int row = slot / s.heads;
      const int64_t off = static_cast<int64_t>(slot - row * s.heads) * a.d;
      const T* x = static_cast<const T*>(s.x) + (r0 + row) * s.ldx + off;
      const T* g = static_cast<const T*>(s.g) + (r0 + row) * s.ldg + off;
      load_words<W>(x + ca, xa);
      load_words<W>(x + cb, xb);
      load_words<W>(g + ca, ga);
      load_words<W>(g + cb, gb);
    };
    fetch(first);
    __syncthreads();  // the previous group's turns have been read
    if (a.rot > 0) fill_turns<V>(a, cs, r0, n);
    __syncthreads();
    for (int base = 0; base < total; base += step) {
      const int slot = base + first;
      const bool on = live && slot < total;
      float fxa[V], fxb[V], fga[V], fgb[V];
      if (on) {
        unpack<T, V, W>(xa, fxa);
        unpack<T, V, W>(xb, fxb);
        unpack<T, V, W>(ga, fga);
        unpack<T, V, W>(gb, fgb);
      } else {
#pragma unroll
        for (int e = 0; e < V; ++e) fxa[e] = fxb[e] = fga[e] = fgb[e] = 0.f;
      }
      fetch(slot + step);
      const int row = on ? slot / s.heads : 0;
      const int64_t off = static_cast<int64_t>(slot - row * s.heads) * a.d;
      if (on && turned)
        turn_unit<V, INTER>(cs + row * (a.rot / 2), u, a.rot / (2 * V), fga, fgb);
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
          oa[e] = ra * wa[e] - fxa[e] * back;
          ob[e] = rb * wb[e] - fxb[e] * back;
        }
        uint32_t pa[W], pb[W];
        pack<T, V, W>(oa, pa);
        pack<T, V, W>(ob, pb);
        T* dst = static_cast<T*>(s.y) + (r0 + row) * s.ldy + off;
        store_words<W>(dst + ca, pa);
        store_words<W>(dst + cb, pb);
      }
    }
  }
  if (a.partial == nullptr) return;
  __syncthreads();
  float* sum = reinterpret_cast<float*>(smem_f4);  // [step][d]
  if (live) {
#pragma unroll
    for (int e = 0; e < V; ++e) {
      sum[first * a.d + ca + e] = da[e];
      sum[first * a.d + cb + e] = db[e];
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < a.d; i += kThreads) {
    float t = 0.f;
    for (int j = 0; j < step; ++j) t += sum[j * a.d + i];
    a.partial[static_cast<int64_t>(blockIdx.x) * a.d + i] = t;
  }
}

// dw[i] = sum of the partials' rows, in a fixed order: 8 columns a block (one
// per warp), a lane takes every 32nd row.
__global__ void __launch_bounds__(kThreads) rope_dw_kernel(const float* partial, int d,
                                                           int blocks_q, int blocks, float* dwq,
                                                           float* dwk) {
  const bool key = blockIdx.y == 1;
  float* dw = key ? dwk : dwq;
  const int col = blockIdx.x * 8 + (threadIdx.x >> 5);
  if (dw == nullptr || col >= d) return;
  const int lane = threadIdx.x & 31;
  const int b1 = key ? blocks : blocks_q;
  float t = 0.f;
  for (int b = (key ? blocks_q : 0) + lane; b < b1; b += 32)
    t += partial[static_cast<int64_t>(b) * d + col];
  t = lane_sum(t, 32);
  if (lane == 0) dw[col] = t;
}

bool al(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) % n) == 0; }

int pow2_at_least(int n) {
  int p = 1;
  while (p < n) p *= 2;
  return p;
}

// V = 8 for 16-bit types where the vectors allow it (16-byte loads), else 4.
// At least half as many bytes a load cost little: 96-wide heads with a
// 24-column rotation are the common reason for 4.
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
    if (positions != nullptr && (!al(positions, 4) || (plan->n_axes > 1 && pos_stride < rows)))
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

// Rows of a block: enough that every thread computes about one sine and
// cosine, but no more than leaves four blocks an SM.
int rows_per_block(int64_t rows, int rot, int sms) {
  int n = rot > 0 ? 2 * kThreads / rot : 4;
  n = n < 1 ? 1 : n > 8 ? 8 : n;
  while (n > 1 && (rows + n - 1) / n < 4 * sms) n /= 2;
  return n;
}

vdn_status launch_forward(RopeArgs& a, int dtype, int layout, cudaStream_t stream) {
  if (a.rows == 0) return VDN_OK;
  a.rows_per_block = rows_per_block(a.rows, a.rot, sm_count_of_current_device());
  const int smem = a.rows_per_block * a.rot / 2 * 8;
  const int64_t grid = (a.rows + a.rows_per_block - 1) / a.rows_per_block;
  const cudaError_t e = dispatch(
      dtype, vector_width(dtype, a.d, a.rot), layout == VDN_ROPE_INTERLEAVED,
      [&](auto t, auto v, auto inter) {
        rope_kernel<decltype(t), decltype(v)::value, decltype(inter)::value>
            <<<static_cast<unsigned>(grid), kThreads, smem, stream>>>(a);
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
  a.partial = dwq || dwk
                  ? reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + kStatusBytes)
                  : nullptr;
  const int sms = sm_count_of_current_device();
  a.rows_per_block = rows_per_block(rows, a.rot, sms);
  // blocks shared out by heads; at most four an SM, at most one a row group
  const int64_t groups = (rows + a.rows_per_block - 1) / a.rows_per_block;
  const int most = 4 * sms < kMaxBwdBlocks ? 4 * sms : kMaxBwdBlocks - 1;  // each side has one
  auto share = [&](int heads) {
    int64_t n = static_cast<int64_t>(most) * heads / (H + H_kv);
    n = n > groups ? groups : n;
    return static_cast<int>(n < 1 ? 1 : n);
  };
  a.blocks_q = share(H);
  const int blocks = a.blocks_q + share(H_kv);
  const int turns = a.rows_per_block * a.rot / 2 * 8;
  const int sums = kThreads / a.lanes * a.d * 4;
  const cudaError_t e = dispatch(
      dtype, vector_width(dtype, a.d, a.rot), plan->layout == VDN_ROPE_INTERLEAVED,
      [&](auto t, auto v, auto inter) {
        rope_backward_kernel<decltype(t), decltype(v)::value, decltype(inter)::value>
            <<<blocks, kThreads, turns > sums ? turns : sums, st>>>(a);
        return cudaGetLastError();
      });
  if (e != cudaSuccess) return VDN_ERR_CUDA;
  if (a.partial != nullptr) {
    rope_dw_kernel<<<dim3((a.d + 7) / 8, 2), kThreads, 0, st>>>(a.partial, a.d, a.blocks_q,
                                                                blocks, dwq, dwk);
    if (cudaGetLastError() != cudaSuccess) return VDN_ERR_CUDA;
  }
  return VDN_OK;
}

}  // extern "C"
