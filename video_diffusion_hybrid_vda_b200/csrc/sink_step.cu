// One new token per sequence of a sink-window attention stream, over a rolling
// cache of `sinks` + `window` slots, the new key and value written into their
// slot by the same launch.
//
// Position p lives in slot p while p < sinks + window, and in slot
// sinks + (p - sinks) mod window after that, so the slots hold exactly the
// keys that position p sees (j < sinks or p - j < window), in an order the
// softmax does not care about:
//   o = sum_j softmax(scale q . k_j) v_j over the min(p + 1, slots) live slots
//
// Bound: reading the live keys and values once.  The heads that share a key
// head (up to 16, the rows of one MMA) are taken together, so no key is read
// twice.  A cluster of CTAs splits the live slots; each warp streams tiles of
// 16 slots through its own cp.async ring (no block barrier in the loop) and
// keeps its own running maximum, sum and output; warps join in shared memory,
// then every CTA writes each other CTA of the cluster its share of the columns
// into distributed shared memory, and all add their columns' parts in rank
// order: one launch, no workspace, the same bits every time.  mma.sync suffices: at 8 query heads a
// key head the products are 8 flop a byte, a hundredth of the tensor rate.
#include <cuda_bf16.h>
#include <math.h>

#include "common.cuh"
#include "exp2_fma.cuh"
#include "ptx.cuh"

namespace vdn {

namespace {

constexpr int kWarps = 4;
constexpr int kStages = 3;
constexpr int kTile = 16;   // slots a tile
constexpr int kRows = 16;   // query heads a CTA

struct StepArgs {
  int H, Hkv, window, sinks;
  int blocks;               // CTAs' worth of query heads a key head
  const __nv_bfloat16* q;
  const __nv_bfloat16* k_new;
  const __nv_bfloat16* v_new;
  __nv_bfloat16* k_cache;
  __nv_bfloat16* v_cache;
  __nv_bfloat16* o;
  int64_t ld_q, ld_new, ld_cache, batch_stride, ld_o;
  const int32_t* positions;
  float scale_log2;
};

template <int DH>
struct StepCfg {
  static constexpr int ROW = DH * 2;               // bytes of a slot's key
  static constexpr int STAGE = 2 * kTile * ROW;    // K tile, V tile
  static constexpr int RING = kWarps * kStages * STAGE;
  // after the loop the ring holds each warp's output [16][DH] fp32
  static constexpr int SMEM = RING + kWarps * 2 * kRows * 4 + kRows * DH * 4 + 16 * 2 * kRows * 4;
};

__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool on) {
  // 16 bytes, or 16 zero bytes where the slot holds nothing
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(on ? 16 : 0)
               : "memory");
}

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

__device__ __forceinline__ void st_cluster(uint32_t saddr, uint32_t rank, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(mapa_shared(saddr, rank)), "f"(v)
               : "memory");
}

template <int DH>
__global__ void __launch_bounds__(kWarps * 32) sink_step_kernel(const StepArgs a) {
  using Cfg = StepCfg<DH>;
  constexpr int CH = DH / 8;  // 16-byte chunks of a row
  extern __shared__ uint4 smem_u4[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(smem_u4);
  float* red = reinterpret_cast<float*>(smem + Cfg::RING);  // [warp][m 16, l 16]
  // from every CTA of the cluster: its part of this CTA's columns
  // [rank][16][DH / splits], and its [m 16, l 16]
  float* part = red + kWarps * 2 * kRows;
  float* part_ml = part + kRows * DH;
  const uint32_t splits = gridDim.x, split = blockIdx.x;    // the cluster is one row of the grid
  const int hk = blockIdx.y / a.blocks, block = blockIdx.y % a.blocks, b = blockIdx.z;
  const int group = a.H / a.Hkv;
  const int heads = min(kRows, group - block * kRows);
  const int h0 = hk * group + block * kRows;
  const int pos = a.positions[b];
  if (pos < 0) return;  // the whole cluster: an inactive sequence
  // "this CTA runs", waited for before anything is written to it
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  const int slots = a.sinks + a.window;
  const int slot = pos < slots ? pos : a.sinks + (pos - a.sinks) % a.window;
  const int live = min(pos, slots - 1) + 1;
  const int tiles = (live + kTile - 1) / kTile;
  const int t0 = static_cast<int>(static_cast<int64_t>(tiles) * split / splits);
  const int t1 = static_cast<int>(static_cast<int64_t>(tiles) * (split + 1) / splits);
  const int warp = warp_id(), lane = lane_id();

  const __nv_bfloat16* kc = a.k_cache + b * a.batch_stride + hk * DH;
  const __nv_bfloat16* vc = a.v_cache + b * a.batch_stride + hk * DH;
  const __nv_bfloat16* kn = a.k_new + b * a.ld_new + hk * DH;
  const __nv_bfloat16* vn = a.v_new + b * a.ld_new + hk * DH;
  const uint32_t ring = smem_u32(smem) + warp * kStages * Cfg::STAGE;

  // tile t of this warp's ring into stage s: 16-byte chunks, swizzled by row
  auto fetch = [&](int t, int s) {
    if (t < t1) {
      const uint32_t base = ring + s * Cfg::STAGE;
#pragma unroll
      for (int i = 0; i < kTile * CH / 32; ++i) {
        const int c = i * 32 + lane, row = c / CH, ch = c % CH;
        const int at = t * kTile + row;
        // the new token comes from its own tensors: its slot may be being
        // written by another CTA
        const int64_t off = static_cast<int64_t>(at) * a.ld_cache + ch * 8;
        const __nv_bfloat16* ks = at == slot ? kn + ch * 8 : kc + off;
        const __nv_bfloat16* vs = at == slot ? vn + ch * 8 : vc + off;
        const uint32_t dst = base + row * Cfg::ROW + ((ch ^ (row & 7)) << 4);
        cp16(dst, at < live ? ks : kn, at < live);
        cp16(dst + kTile * Cfg::ROW, at < live ? vs : vn, at < live);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int s = 0; s < kStages - 1; ++s) fetch(t0 + warp + s * kWarps, s);

  // the new key and value into the cache (by the first CTA of the first block)
  if (split == 0 && block == 0 && threadIdx.x < 2 * CH) {
    const bool v = threadIdx.x >= CH;
    const int ch = threadIdx.x % CH;
    __nv_bfloat16* dst = (v ? a.v_cache : a.k_cache) + b * a.batch_stride +
                         static_cast<int64_t>(slot) * a.ld_cache + hk * DH;
    // (no workspace: a debug build skips a miss without recording it)
    if (in_bounds(nullptr, slot, slots, hk * DH + 8 * ch, 8, static_cast<int64_t>(a.Hkv) * DH))
      reinterpret_cast<uint4*>(dst)[ch] = reinterpret_cast<const uint4*>(v ? vn : kn)[ch];
  }

  // Q as MMA rows (query heads g and g + 8 of this lane's quad)
  const int g = lane >> 2, c2 = 2 * (lane & 3);
  uint32_t qf[DH / 16][4];
  {
    const __nv_bfloat16* q = a.q + b * a.ld_q + static_cast<int64_t>(h0) * DH;
#pragma unroll
    for (int kk = 0; kk < DH / 16; ++kk)
#pragma unroll
      for (int f = 0; f < 4; ++f) {
        const int row = g + 8 * (f & 1), col = 16 * kk + c2 + 8 * (f >> 1);
        qf[kk][f] = row < heads ? *reinterpret_cast<const uint32_t*>(q + row * DH + col) : 0u;
      }
  }
  float o[DH / 8][4] = {};
  float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;  // rows g and g + 8, log2 domain
  int s = 0;
  for (int t = t0 + warp; t < t1; t += kWarps) {
    fetch(t + (kStages - 1) * kWarps, (s + kStages - 1) % kStages);
    asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
    __syncwarp();
    const uint32_t kb = ring + s * Cfg::STAGE, vb = kb + kTile * Cfg::ROW;
    // S [16 heads, 16 slots]: two 8-slot halves
    float sc[2][4] = {};
#pragma unroll
    for (int kk = 0; kk < DH / 16; ++kk) {
      // matrices: slots 0-7 columns 16 kk.., +8; slots 8-15 the same
      const int row = (lane & 7) + ((lane >> 4) << 3), ch = 2 * kk + ((lane >> 3) & 1);
      uint32_t f[4];
      ldsm4(kb + row * Cfg::ROW + ((ch ^ (row & 7)) << 4), f);
      mma16816(sc[0], qf[kk], f[0], f[1]);
      mma16816(sc[1], qf[kk], f[2], f[3]);
    }
    const int left = live - t * kTile;  // slots of this tile that hold something
    float n0 = m0, n1 = m1;
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        sc[n][e] = 8 * n + c2 + (e & 1) < left ? sc[n][e] * a.scale_log2 : -INFINITY;
        float& top = e < 2 ? n0 : n1;
        top = fmaxf(top, sc[n][e]);
      }
    n0 = fmaxf(n0, __shfl_xor_sync(0xffffffffu, n0, 1));
    n1 = fmaxf(n1, __shfl_xor_sync(0xffffffffu, n1, 1));
    n0 = fmaxf(n0, __shfl_xor_sync(0xffffffffu, n0, 2));
    n1 = fmaxf(n1, __shfl_xor_sync(0xffffffffu, n1, 2));
    // a tile has a live slot, so n0 and n1 are above -inf unless every score
    // is -inf itself
    const float b0 = n0 == -INFINITY ? 0.f : n0, b1 = n1 == -INFINITY ? 0.f : n1;
    const float f0 = exp2_mufu(m0 - b0), f1 = exp2_mufu(m1 - b1);
    m0 = n0;
    m1 = n1;
    float p[2][4];
    float s0 = 0.f, s1 = 0.f;
#pragma unroll
    for (int n = 0; n < 2; ++n) {
#pragma unroll
      for (int e = 0; e < 4; ++e) p[n][e] = exp2_mufu(sc[n][e] - (e < 2 ? b0 : b1));
      s0 += p[n][0] + p[n][1];
      s1 += p[n][2] + p[n][3];
    }
    l0 = l0 * f0 + s0;
    l1 = l1 * f1 + s1;
    // P rounded to bf16 for the product (the sum adds it unrounded)
    const uint32_t pf[4] = {pack_bf16x2(p[0][0], p[0][1]), pack_bf16x2(p[0][2], p[0][3]),
                            pack_bf16x2(p[1][0], p[1][1]), pack_bf16x2(p[1][2], p[1][3])};
#pragma unroll
    for (int n = 0; n < DH / 16; ++n) {
      // matrices: slots 0-7, 8-15 of columns 16 n.., then of columns 16 n + 8..
      const int row = lane & 15, ch = 2 * n + (lane >> 4);
      uint32_t f[4];
      ldsm4_t(vb + row * Cfg::ROW + ((ch ^ (row & 7)) << 4), f);
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        float(&c)[4] = o[2 * n + half];
        c[0] *= f0, c[1] *= f0, c[2] *= f1, c[3] *= f1;
        mma16816(c, pf, f[2 * half], f[2 * half + 1]);
      }
    }
    __syncwarp();  // the stage is read before it is filled again
    s = (s + 1) % kStages;
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  l0 += __shfl_xor_sync(0xffffffffu, l0, 1);
  l1 += __shfl_xor_sync(0xffffffffu, l1, 1);
  l0 += __shfl_xor_sync(0xffffffffu, l0, 2);
  l1 += __shfl_xor_sync(0xffffffffu, l1, 2);
  __syncthreads();  // every ring is done with
  // ---- join the warps
  float* out = reinterpret_cast<float*>(smem) + warp * kRows * DH;
#pragma unroll
  for (int n = 0; n < DH / 8; ++n) {
    *reinterpret_cast<float2*>(out + g * DH + 8 * n + c2) = make_float2(o[n][0], o[n][1]);
    *reinterpret_cast<float2*>(out + (g + 8) * DH + 8 * n + c2) = make_float2(o[n][2], o[n][3]);
  }
  if ((lane & 3) == 0) {
    red[warp * 2 * kRows + g] = m0;
    red[warp * 2 * kRows + g + 8] = m1;
    red[warp * 2 * kRows + kRows + g] = l0;
    red[warp * 2 * kRows + kRows + g + 8] = l1;
  }
  __syncthreads();
  asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
  const int cols = DH / splits;  // of each CTA; DH >= 4 splits
  for (int i = threadIdx.x; i < heads * DH; i += kWarps * 32) {
    const int r = i / DH, c = i % DH;
    float top = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) top = fmaxf(top, red[w * 2 * kRows + r]);
    const float base = top == -INFINITY ? 0.f : top;
    float acc = 0.f, sum = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float f = exp2_mufu(red[w * 2 * kRows + r] - base);  // 0 for a warp without tiles
      acc += f * reinterpret_cast<const float*>(smem)[w * kRows * DH + i];
      sum += f * red[w * 2 * kRows + kRows + r];
    }
    const uint32_t to = c / cols;
    st_cluster(smem_u32(part + (split * kRows + r) * cols + c % cols), to, acc);
    if (c % cols == 0) {
      st_cluster(smem_u32(part_ml + split * 2 * kRows + r), to, top);
      st_cluster(smem_u32(part_ml + split * 2 * kRows + kRows + r), to, sum);
    }
  }
  cluster_sync();  // every part has arrived; nothing remote follows
  // ---- join the cluster: this CTA's columns
  for (int i = 2 * threadIdx.x; i < heads * cols; i += 2 * kWarps * 32) {
    const int r = i / cols, c = i % cols;
    float top = -INFINITY;
    for (uint32_t k = 0; k < splits; ++k) top = fmaxf(top, part_ml[k * 2 * kRows + r]);
    const float base = top == -INFINITY ? 0.f : top;
    float x = 0.f, y = 0.f, sum = 0.f;
    for (uint32_t k = 0; k < splits; ++k) {
      const float f = exp2_mufu(part_ml[k * 2 * kRows + r] - base);
      const float2 v = *reinterpret_cast<const float2*>(part + (k * kRows + r) * cols + c);
      x += f * v.x;
      y += f * v.y;
      sum += f * part_ml[k * 2 * kRows + kRows + r];
    }
    const float inv = 1.f / sum;
    const int col = (h0 + r) * DH + split * cols + c;
    if (in_bounds(nullptr, b, gridDim.z, col, 2, static_cast<int64_t>(a.H) * DH))
      *reinterpret_cast<uint32_t*>(a.o + b * a.ld_o + col) = pack_bf16x2(x * inv, y * inv);
  }
}

// CTAs a cluster: enough in all to give each SM four (two run at a time), while
// a CTA has at least two tiles for each of its warps.  32 sequences of 100 to
// 12000 tokens, 8 key heads, 4096 slots: 81.4 us at two CTAs an SM, 80.2 at
// four, 98 at eight.
int step_splits(int64_t rows, int slots) {
  int n = 1;
  while (n < 16 && rows * n < 4 * 148 && slots / (kTile * kWarps * 2) >= 2 * n) n *= 2;
  return n;
}

template <int DH>
cudaError_t launch_step(const StepArgs& a, int B, cudaStream_t stream) {
  using Cfg = StepCfg<DH>;
  static std::atomic<uint64_t> smem_set{0}, cluster_set{0};
  if (cudaError_t e = set_smem_once(sink_step_kernel<DH>, Cfg::SMEM, smem_set)) return e;
  int dev = 0;
  if (cudaError_t e = cudaGetDevice(&dev)) return e;
  const uint64_t bit = uint64_t(1) << (dev & 63);
  if (!(cluster_set.load(std::memory_order_acquire) & bit)) {
    if (cudaError_t e = cudaFuncSetAttribute(sink_step_kernel<DH>,
                                             cudaFuncAttributeNonPortableClusterSizeAllowed, 1))
      return e;
    cluster_set.fetch_or(bit, std::memory_order_release);
  }
  const int y = a.Hkv * a.blocks;
  const int splits = step_splits(static_cast<int64_t>(B) * y, a.sinks + a.window);
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = splits;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(splits, y, B);
  cfg.blockDim = dim3(kWarps * 32);
  cfg.dynamicSmemBytes = Cfg::SMEM;
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, sink_step_kernel<DH>, a);
}

}  // namespace

}  // namespace vdn

using namespace vdn;

extern "C" {

vdn_status vdn_sink_attn_step(int B, int H, int H_kv, int d, int window, int sinks, const void* q,
                              int64_t ld_q, const void* k_new, const void* v_new, int64_t ld_new,
                              void* k_cache, void* v_cache, int64_t ld_cache,
                              int64_t batch_stride, const int32_t* positions, float scale, void* o,
                              int64_t ld_o, void* stream) {
  NvtxRange nvtx("vdn_sink_attn_step");
  if (B < 0 || H < 1 || H_kv < 1 || H % H_kv || d < 1 || window < 1 || sinks < 0)
    return VDN_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return VDN_ERR_UNSUPPORTED;
  const int64_t slots = static_cast<int64_t>(window) + sinks;
  const int64_t D = static_cast<int64_t>(H) * d, Dk = static_cast<int64_t>(H_kv) * d;
  if (D >= (int64_t(1) << 24) || slots >= (int64_t(1) << 30)) return VDN_ERR_INVALID_ARG;
  const int blocks = (H / H_kv + kRows - 1) / kRows;
  if (B > 65535 || static_cast<int64_t>(H_kv) * blocks > 65535) return VDN_ERR_UNSUPPORTED;
  if (B == 0) return VDN_OK;
  for (const void* p : {q, k_new, v_new, static_cast<const void*>(k_cache),
                        static_cast<const void*>(v_cache), static_cast<const void*>(o)})
    if (p == nullptr || (reinterpret_cast<uintptr_t>(p) & 15u)) return VDN_ERR_INVALID_ARG;
  if (positions == nullptr || (reinterpret_cast<uintptr_t>(positions) & 3u))
    return VDN_ERR_INVALID_ARG;
  if (ld_q < D || ld_q % 8 || ld_o < D || ld_o % 8 || ld_new < Dk || ld_new % 8 ||
      ld_cache < Dk || ld_cache % 8 || batch_stride % 8 ||
      (B > 1 && batch_stride < (slots - 1) * ld_cache + Dk))
    return VDN_ERR_INVALID_ARG;
  StepArgs a{};
  a.H = H, a.Hkv = H_kv, a.window = window, a.sinks = sinks;
  a.blocks = blocks;
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.k_new = static_cast<const __nv_bfloat16*>(k_new);
  a.v_new = static_cast<const __nv_bfloat16*>(v_new);
  a.k_cache = static_cast<__nv_bfloat16*>(k_cache);
  a.v_cache = static_cast<__nv_bfloat16*>(v_cache);
  a.o = static_cast<__nv_bfloat16*>(o);
  a.ld_q = ld_q, a.ld_new = ld_new, a.ld_cache = ld_cache, a.ld_o = ld_o;
  a.batch_stride = batch_stride;
  a.positions = positions;
  a.scale_log2 =
      (scale > 0.f ? scale : 1.f / sqrtf(static_cast<float>(d))) * 1.4426950408889634f;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = d == 128 ? launch_step<128>(a, B, st) : launch_step<64>(a, B, st);
  return e == cudaSuccess ? VDN_OK : VDN_ERR_CUDA;
}

}  // extern "C"
