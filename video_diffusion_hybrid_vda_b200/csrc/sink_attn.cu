// Attention with a sliding window and a few first tokens that stay visible
// (sinks), over packed sequences with shared key heads: the forward pass.
//
//   s_ij = scale q_i . k_j over the visible keys (mask: sink_attn.cuh)
//   o_i  = sum_j exp(s_ij - lse_i) v_j,   lse_i = log sum_j exp(s_ij)
// A query that sees nothing gives o = 0 and lse = -inf.
//
// One pass over the keys with a running maximum and sum.  The unit of work is
// 256 rows (two 128-row tiles) of one sequence and key head: 256 queries of a
// head, or, where sequences are short and heads share a key head, fewer
// queries of several heads, so that a key tile is loaded and multiplied once
// for all of them.  A CTA takes a unit, heaviest first, and walks the keys its
// queries see between them in tiles of 128; a row tile leaves out the key
// tiles it does not touch (the window's two ends), and only key tiles that
// cross the mask's edge pay for comparisons.  (Persistent CTAs that begin the
// next unit's loads and scores while the last output is stored were not
// faster: 8097 tokens, 16 heads, window 1024 took 122 us with units dealt out
// in turn against 104 us with one CTA a unit, 16384 tokens the same.)
//   warp 0      TMA: Q, then K and V tiles through a ring; rows of a V tile
//               past its interval are zeroed before the tile is handed on
//   warp 1      tcgen05.mma: S_i = Q_i K^T, O_i += P_i V (P_i from TMEM)
//   warps 4-7   softmax of row tile 0, warps 8-11 of tile 1, one row a thread
// TMEM columns: S0 S1 O0 O1, 128 each; P_i overwrites S_i as bf16 (its
// rounding averages out over the keys; the row sum adds the unrounded P).
//
// Few queries leave most SMs without a unit: then the key tiles of each unit
// are split over several, each writes its normalised part in fp32 with its
// lse, and sink_combine_kernel joins them, o = sum_s e^(lse_s - lse) o_s.
//
// Bound: the chain score product -> softmax -> product with V of a row tile,
// which the other row tile half hides (two S and two O accumulators fill TMEM
// at d = 128).  16384 tokens, 16 heads over 4, window 4096: 432 to 514 us by the
// box and its clocks under the power cap (eager and in a graph alike: 488 to 502
// and 498 us on one box), 0.94 to 1.11 PFLOP/s of visible pairs (0.57 to 0.68 of
// the burst rate of a large product, 0.68 to 0.81 of its sustained one); tensor
// and exponential pipes each 40 % busy.  Also measured, on a box where it took
// 450 us: a quarter of the exponentials on the FMA pipe 500, two warpgroups a row
// tile 513, key tiles of up to 64 valid keys taken by halves 456 (and 15.4 in
// place of 16.2 us for three short sequences).
#include <cuda_bf16.h>
#include <math.h>

#include <type_traits>

#include "exp2_fma.cuh"
#include "sink_attn.cuh"

namespace vdn {

namespace {

template <int DH>
struct SinkCfg {
  static constexpr int SLABS = DH / 64;
  static constexpr int TILE_BYTES = SLABS * 128 * 128;  // 128 rows x DH bf16
  static constexpr int STAGES = DH == 64 ? 4 : 2;
  static constexpr int THREADS = 384;
  static constexpr int SMEM = 1024 + 2 * TILE_BYTES + STAGES * 2 * TILE_BYTES + 512;
};

struct SinkOut {
  __nv_bfloat16* o;  // [Lq, ld_o], or null where parts are written
  int64_t ld_o;
  float* lse;        // [H, Lq] or null
  float* part_o;     // [splits, Lq, H, DH]
  float* part_lse;   // [splits, H, Lq]
  bool zero_rest;    // zero the rows of o of no sequence
};

// How rows are made into units: `rows` queries (a power of two, 8 to 256) of
// 256 / rows heads that share a key head; each unit's keys in `splits` parts.
struct SinkCut {
  int rows, splits;
};

struct SinkUnit {
  int row0, row1;     // query rows of the unit and the end of its sequence
  int h0, hk, split;  // first head, key head
  int pa, pb;         // positions of its first and last query
  int k0, j0, j1;     // first key row of the sequence; key tiles [j0, j1)
  SinkKeyTiles kt;
  // The CTA's unit; false if it has no queries.
  __device__ bool init(const SinkDims& s, const SinkCut& c) {
    const int per_slot = s.H * c.rows / 256 * c.splits;
    // heaviest first: the last queries of a sequence see the most keys
    const int slot = sink_slots(s.Lq, s.B, c.rows) - 1 - static_cast<int>(blockIdx.x) / per_slot;
    const int in = static_cast<int>(blockIdx.x) % per_slot;
    const int b = sink_slot_seq(s.cu_q, s.B, s.Lq, c.rows, slot);
    const SinkSeq seq = sink_seq(s, b);
    const int at = c.rows * (slot - sink_slot_base(s.cu_q, b, s.Lq, c.rows));
    if (at < 0 || at >= seq.nq()) return false;
    row0 = seq.q0 + at;
    row1 = seq.q1;
    h0 = in / c.splits * (256 / c.rows);
    split = in % c.splits;
    hk = h0 / (s.H / s.Hkv);
    pa = at + seq.shift();
    pb = min(pa + c.rows - 1, seq.nk() - 1);
    k0 = seq.k0;
    kt.init(s.m, pa, pb, seq.nk());
    j0 = static_cast<int>(static_cast<int64_t>(kt.n) * split / c.splits);
    j1 = static_cast<int>(static_cast<int64_t>(kt.n) * (split + 1) / c.splits);
    return true;
  }
  // Positions of row tile i (none: last < first).
  __device__ int first(const SinkCut& c, int i) const { return c.rows == 256 ? pa + 128 * i : pa; }
  __device__ int last(const SinkCut& c, int i) const {
    return c.rows == 256 && i == 0 ? min(pa + 127, pb) : pb;
  }
  // Does row tile i take key tile j?
  __device__ bool takes(const SinkDims& s, const SinkCut& c, int i, int j) const {
    const int ks = kt.start(j);
    return sink_touches(s.m, first(c, i), last(c, i), ks, ks + kt.valid(j) - 1);
  }
};

// Softmax of one 128-row tile of the unit: one thread per row.
template <int DH>
__device__ __forceinline__ bool sink_softmax(int i, uint32_t tmem, const SinkUnit& cur,
                                             const SinkDims& dims, const SinkCut& cut,
                                             uint64_t* s_full, uint64_t* o_done, uint64_t* p_half,
                                             uint64_t* p_ready, float scale_log2,
                                             const SinkOut& out, uint32_t* status,
                                             uint64_t budget_ns) {
  const uint32_t quarter = warp_id() & 3;
  const int row = quarter * 32 + lane_id();
  const uint32_t lane_off = (quarter * 32) << 16;
  const uint32_t s_addr = tmem + 128 * i + lane_off;
  const uint32_t o_addr = tmem + 256 + 128 * i + lane_off;
  const SinkMask m = dims.m;
  // this row's query and head within the unit, and its warp's first query
  const int query = (128 * i + row) & (cut.rows - 1), head = (128 * i + row) / cut.rows;
  const int r = cur.row0 + query, h = cur.h0 + head;
  // A maximum that has grown by less than this is kept: P stays below 2^8 and
  // O is not rescaled for nothing.  Rows past the sequence never ask for it,
  // so what they hold does not reach the other rows' roundings.
  const float slack = r < cur.row1 ? 8.f : INFINITY;
  const int wq = (128 * i + quarter * 32) & (cut.rows - 1);
  const int warp_queries = min(32, cut.rows);
  const int p = cur.pa + query, pw = cur.pa + wq;
  float m_used = -INFINITY;  // running maximum, log2 domain (scaled)
  float l = 0.f;
  int n = 0;                 // key tiles taken so far
  for (int j = cur.j0; j < cur.j1; ++j) {
    if (!cur.takes(dims, cut, i, j)) continue;
    const int ks = cur.kt.start(j);
    const int valid = cur.kt.valid(j);
    const bool edge = valid < 128 || !sink_sees_all(m, pw, pw + warp_queries - 1, ks, ks + 127);
    // warp-uniform decision: tcgen05.ld/st below are warp-collective
    if (!__all_sync(0xffffffffu, mbar_wait(&s_full[i], n & 1, budget_ns))) return false;
    tc_fence_after();
    uint32_t sr[128];
    uint32_t (&s0)[32] = *reinterpret_cast<uint32_t(*)[32]>(&sr[0]);
    uint32_t (&s1)[32] = *reinterpret_cast<uint32_t(*)[32]>(&sr[32]);
    uint32_t (&s2)[32] = *reinterpret_cast<uint32_t(*)[32]>(&sr[64]);
    uint32_t (&s3)[32] = *reinterpret_cast<uint32_t(*)[32]>(&sr[96]);
    auto hide = [&](int c0) {  // of columns [c0, c0 + 64), those that are not visible
#pragma unroll
      for (int w = c0; w < c0 + 64; w += 32) {
        const uint32_t see = sink_bits(p - m.window + 1 - ks - w,
                                       min(valid, p + m.ahead + 1 - ks) - w, m.sinks - ks - w);
#pragma unroll
        for (int c = 0; c < 32; ++c)
          sr[w + c] = see & (1u << c) ? sr[w + c] : __float_as_uint(-INFINITY);
      }
    };
    tmem_ld32(s_addr, s0);
    tmem_ld32(s_addr + 32, s1);
    tmem_ld_wait();
    reg_fence(s0);
    reg_fence(s1);
    tmem_ld32(s_addr + 64, s2);
    tmem_ld32(s_addr + 96, s3);
    if (edge) hide(0);
    auto sv = [&](int c) { return __uint_as_float(sr[c]); };
    float mx8[8];
#pragma unroll
    for (int a = 0; a < 8; ++a) mx8[a] = fmax3(sv(a), sv(a + 8), sv(a + 16));
#pragma unroll
    for (int c = 24; c < 56; c += 16)
#pragma unroll
      for (int a = 0; a < 8; ++a) mx8[a] = fmax3(mx8[a], sv(c + a), sv(c + 8 + a));
#pragma unroll
    for (int a = 0; a < 8; ++a) mx8[a] = fmaxf(mx8[a], sv(56 + a));
    tmem_ld_wait();
    reg_fence(s2);
    reg_fence(s3);
    if (edge) hide(64);
#pragma unroll
    for (int c = 64; c < 128; c += 16)
#pragma unroll
      for (int a = 0; a < 8; ++a) mx8[a] = fmax3(mx8[a], sv(c + a), sv(c + 8 + a));
    const float mt = fmax3(fmax3(mx8[0], mx8[1], mx8[2]), fmax3(mx8[3], mx8[4], mx8[5]),
                           fmaxf(mx8[6], mx8[7])) *
                     scale_log2;
    // The maxima in use move when some row's has grown enough.  A row that
    // has seen no key keeps -inf: its factor is 0 and its P below takes 0.
    if (__any_sync(0xffffffffu, mt > m_used + slack)) {
      const float m_new = fmaxf(m_used, mt);
      const float factor = m_used == -INFINITY ? 0.f : exp2_mufu(m_used - m_new);
      l *= factor;
      if (n > 0) {
        if (!__all_sync(0xffffffffu, mbar_wait(&o_done[i], (n - 1) & 1, budget_ns)))
          return false;
        tc_fence_after();
#pragma unroll 1
        for (int c = 0; c < DH; c += 32) {
          uint32_t o[32];
          tmem_ld32(o_addr + c, o);
          tmem_ld_wait();
          reg_fence(o);
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * factor);
          tmem_st32(o_addr + c, o);
        }
      }
      m_used = m_new;
    }
    const float m_sub = m_used == -INFINITY ? 0.f : m_used;
    const uint64_t cc = f32x2_pack(scale_log2, scale_log2);
    const uint64_t nm = f32x2_pack(-m_sub, -m_sub);
    uint64_t acc2[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      uint32_t pk[16];
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const uint64_t xs = f32x2_fma(
            (static_cast<uint64_t>(sr[32 * q + 2 * e + 1]) << 32) | sr[32 * q + 2 * e], cc, nm);
        const uint64_t pp = f32x2_pack(exp2_mufu(f32x2_lo(xs)), exp2_mufu(f32x2_hi(xs)));
        acc2[e & 3] = f32x2_add(acc2[e & 3], pp);
        pk[e] = pack_bf16x2(f32x2_lo(pp), f32x2_hi(pp));
      }
      tmem_st16(s_addr + 16 * q, pk);
      if (q == 1) {  // the product over the first 64 keys starts now
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(&p_half[i]);
      }
    }
    acc2[0] = f32x2_add(f32x2_add(acc2[0], acc2[1]), f32x2_add(acc2[2], acc2[3]));
    l += f32x2_lo(acc2[0]) + f32x2_hi(acc2[0]);
    tmem_st_wait();
    tc_fence_before();
    mbar_arrive(&p_ready[i]);
    ++n;
  }
  // ------------------------------------------------------------ output
  const bool any = n > 0;
  if (any && !__all_sync(0xffffffffu, mbar_wait(&o_done[i], (n - 1) & 1, budget_ns)))
    return false;
  tc_fence_after();
  const bool live = r < cur.row1 && in_bounds(status, r, dims.Lq, static_cast<int64_t>(h) * DH,
                                              DH, static_cast<int64_t>(dims.H) * DH);
  const float inv = l == 0.f ? 0.f : 1.f / l;  // nothing seen: o = 0 (O holds no value if n == 0)
  __nv_bfloat16* dst = out.o + static_cast<int64_t>(r) * out.ld_o + h * DH;
  float* part = out.part_o + ((static_cast<int64_t>(cur.split) * dims.Lq + r) * dims.H + h) * DH;
#pragma unroll 1
  for (int c = 0; c < DH; c += 32) {
    uint32_t o[32];
    if (any) {
      tmem_ld32(o_addr + c, o);
      tmem_ld_wait();
      reg_fence(o);
    } else {
#pragma unroll
      for (int e = 0; e < 32; ++e) o[e] = 0;
    }
    if (!live) continue;
    if (out.o != nullptr) {
#pragma unroll
      for (int e = 0; e < 32; e += 8) {
        uint4 u;
        auto two = [&](int k) {
          return pack_bf16x2(__uint_as_float(o[e + k]) * inv, __uint_as_float(o[e + k + 1]) * inv);
        };
        u.x = two(0), u.y = two(2), u.z = two(4), u.w = two(6);
        *reinterpret_cast<uint4*>(dst + c + e) = u;
      }
    } else {
#pragma unroll
      for (int e = 0; e < 32; e += 4)
        *reinterpret_cast<float4*>(part + c + e) =
            make_float4(__uint_as_float(o[e]) * inv, __uint_as_float(o[e + 1]) * inv,
                        __uint_as_float(o[e + 2]) * inv, __uint_as_float(o[e + 3]) * inv);
    }
  }
  if (!live) return true;
  const float lse = l == 0.f ? -INFINITY : (m_used + log2f(l)) * 0.69314718055994531f;
  const int64_t at = static_cast<int64_t>(h) * dims.Lq + r;
  if (out.o == nullptr)
    out.part_lse[static_cast<int64_t>(cur.split) * dims.H * dims.Lq + at] = lse;
  else if (out.lse != nullptr)
    out.lse[at] = lse;
  return true;
}

template <int DH>
__global__ void __launch_bounds__(SinkCfg<DH>::THREADS, 1)
    sink_attn_kernel(const __grid_constant__ CUtensorMap qmap,
                     const __grid_constant__ CUtensorMap kmap,
                     const __grid_constant__ CUtensorMap vmap, const SinkDims dims,
                     const SinkCut cut, float scale_log2, const SinkOut out, uint32_t* status,
                     uint64_t budget_ns) {
  using Cfg = SinkCfg<DH>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  uint8_t* qbuf = smem;                         // Q0, Q1
  uint8_t* kvbuf = smem + 2 * Cfg::TILE_BYTES;  // stage s: K then V
  uint64_t* bars = reinterpret_cast<uint64_t*>(kvbuf + Cfg::STAGES * 2 * Cfg::TILE_BYTES);
  uint64_t* q_full = bars;
  uint64_t* k_full = bars + 1;              // [STAGES]
  uint64_t* v_full = k_full + Cfg::STAGES;  // [STAGES]
  uint64_t* k_empty = v_full + Cfg::STAGES;
  uint64_t* v_empty = k_empty + Cfg::STAGES;
  uint64_t* s_full = v_empty + Cfg::STAGES;  // [2]
  uint64_t* p_half = s_full + 2;             // [2] P of keys 0..63 stored
  uint64_t* p_ready = p_half + 2;            // [2] all of P stored
  uint64_t* o_done = p_ready + 2;            // [2]
  uint64_t* mma_done = o_done + 2;
  uint64_t* v_cut = mma_done + 1;            // V tiles whose last rows are zeroed
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(v_cut + 1);

  if (out.zero_rest && out.o != nullptr)
    sink_zero_rest(dims.cu_q, dims.B, dims.Lq, out.o, out.ld_o, dims.H * DH);
  after_allow();  // sink_combine_kernel, where there is one
  SinkUnit cur;
  if (!cur.init(dims, cut)) return;  // the whole CTA
  const uint32_t warp = warp_id();

  if (threadIdx.x == 0) {
    mbar_init(q_full, 1);
    for (int s = 0; s < Cfg::STAGES; ++s) {
      mbar_init(&k_full[s], 1);
      mbar_init(&v_full[s], 1);
      mbar_init(&k_empty[s], 1);
      mbar_init(&v_empty[s], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&p_half[i], 128);
      mbar_init(&p_ready[i], 128);
      mbar_init(&o_done[i], 1);
    }
    mbar_init(mma_done, 1);
    mbar_init(v_cut, 1);
    fence_mbar_init();
    tma_prefetch_desc(&qmap);
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

  // Register split (launched with 168 x 384 = 64512): 128 * 96 + 256 * 200 =
  // 63488.
  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 96;\n" ::: "memory");
  }
  if (warp == 0) {
    // ================================================================ TMA
    // the whole warp walks the loop (it zeroes rows together); lane 0 issues
    const bool leader = lane_id() == 0;
    const int box = min(cut.rows, 128);
    if (leader) {
      mbar_arrive_expect_tx(q_full, 2 * Cfg::TILE_BYTES);
      for (int r = 0; r < 256; r += box)  // `box` rows of one head at a time
        for (int sl = 0; sl < Cfg::SLABS; ++sl)
          tma_load_2d(qbuf + (r >> 7) * Cfg::TILE_BYTES + sl * 16384 + (r & 127) * 128, &qmap,
                      q_full, (cur.h0 + r / cut.rows) * DH + 64 * sl,
                      cur.row0 + (r & (cut.rows - 1)));
    }
    int issued_k = 0, issued_v = 0, cuts = 0;
    bool ok = true;
    for (int j = cur.j0; j < cur.j1; ++j) {
      const int t = j - cur.j0, s = t % Cfg::STAGES;
      const uint32_t par = ((t / Cfg::STAGES) & 1) ^ 1;
      uint8_t* kb = kvbuf + s * 2 * Cfg::TILE_BYTES;
      uint8_t* vb = kb + Cfg::TILE_BYTES;
      const int key0 = cur.k0 + cur.kt.start(j);
      const int valid = cur.kt.valid(j);
      if (t >= Cfg::STAGES)
        ok = __all_sync(0xffffffffu, mbar_wait(&k_empty[s], par, budget_ns));
      if (!ok) break;
      if (leader) {
        mbar_arrive_expect_tx(&k_full[s], Cfg::TILE_BYTES);
        for (int sl = 0; sl < Cfg::SLABS; ++sl)
          tma_load_2d(kb + sl * 16384, &kmap, &k_full[s], cur.hk * DH + 64 * sl, key0);
      }
      ++issued_k;
      if (t >= Cfg::STAGES)
        ok = __all_sync(0xffffffffu, mbar_wait(&v_empty[s], par, budget_ns));
      if (!ok) break;
      uint64_t* full = valid < 128 ? v_cut : &v_full[s];
      if (leader) {
        mbar_arrive_expect_tx(full, Cfg::TILE_BYTES);
        for (int sl = 0; sl < Cfg::SLABS; ++sl)
          tma_load_2d(vb + sl * 16384, &vmap, full, cur.hk * DH + 64 * sl, key0);
      }
      __syncwarp();
      if (valid < 128) {
        // the tile lands on a barrier of its own, loses its last rows, and
        // is then handed on
        ok = __all_sync(0xffffffffu, mbar_wait(v_cut, cuts & 1, budget_ns));
        if (!ok) break;
        ++cuts;
        sink_zero_rows(vb, Cfg::SLABS, valid);
        if (leader) mbar_arrive(&v_full[s]);
      }
      ++issued_v;
    }
    if (!ok) record_status(status, kStatusTimeout);
    // no load may be in flight when the CTA ends
    mbar_wait(q_full, 0, 200000000ull);
    for (int t = max(0, issued_k - Cfg::STAGES); t < issued_k; ++t)
      mbar_wait(&k_full[t % Cfg::STAGES], (t / Cfg::STAGES) & 1, 200000000ull);
    for (int t = max(0, issued_v - Cfg::STAGES); t < issued_v; ++t)
      mbar_wait(&v_full[t % Cfg::STAGES], (t / Cfg::STAGES) & 1, 200000000ull);
    if (!ok) mbar_wait(v_cut, cuts & 1, 200000000ull);  // a cut tile's load may be in flight
  } else if (warp == 1) {
    // ================================================================ MMA
    if (elect_one()) {
      constexpr uint32_t idesc_s = idesc_bf16(128, 128, false, false);
      constexpr uint32_t idesc_o = idesc_bf16(128, DH, false, true);
      const uint32_t qb = smem_u32(qbuf);
      bool ok = mbar_wait(q_full, 0, budget_ns);
      int done[2] = {0, 0};  // key tiles each row tile has taken
      auto stage = [&](int j) { return (j - cur.j0) % Cfg::STAGES; };
      auto phase = [&](int j) { return ((j - cur.j0) / Cfg::STAGES) & 1; };
      auto issue_s = [&](int i, int j) {
        if (!cur.takes(dims, cut, i, j)) return;
        const uint32_t kb = smem_u32(kvbuf + stage(j) * 2 * Cfg::TILE_BYTES);
#pragma unroll
        for (int kk = 0; kk < DH / 16; ++kk) {
          const uint32_t off = (kk >> 2) * 16384 + (kk & 3) * 32;
          umma_ss(tmem + 128 * i, sdesc_sw128(qb + i * Cfg::TILE_BYTES + off, 16, 1024),
                  sdesc_sw128(kb + off, 16, 1024), idesc_s, kk > 0);
        }
        umma_commit(&s_full[i]);
      };
      // O_i += P_i V of tile j, the first 64 keys as soon as their P is there
      auto issue_o = [&](int i, int j) {
        if (!cur.takes(dims, cut, i, j)) return true;
        const uint32_t vb = smem_u32(kvbuf + stage(j) * 2 * Cfg::TILE_BYTES + Cfg::TILE_BYTES);
        for (int half = 0; half < 2; ++half) {
          if (!mbar_wait(half ? &p_ready[i] : &p_half[i], done[i] & 1, budget_ns)) return false;
          tc_fence_after();
#pragma unroll
          for (int kk = 4 * half; kk < 4 * half + 4; ++kk)
            umma_ts(tmem + 256 + 128 * i, tmem + 128 * i + kk * 8,
                    sdesc_sw128(vb + kk * 2048, 16384, 1024), idesc_o, done[i] > 0 || kk > 0);
        }
        umma_commit(&o_done[i]);
        ++done[i];
        return true;
      };
      if (ok && cur.j0 < cur.j1 && (ok = mbar_wait(&k_full[0], 0, budget_ns))) {
        tc_fence_after();
        issue_s(0, cur.j0);
        issue_s(1, cur.j0);
        umma_commit(&k_empty[0]);
      }
      for (int j = cur.j0; j < cur.j1 && ok; ++j) {
        const bool more = j + 1 < cur.j1;
        if (!(ok = mbar_wait(&v_full[stage(j)], phase(j), budget_ns))) break;
        tc_fence_after();
        if (!(ok = issue_o(0, j))) break;
        if (more) {
          if (!(ok = mbar_wait(&k_full[stage(j + 1)], phase(j + 1), budget_ns))) break;
          tc_fence_after();
          issue_s(0, j + 1);
        }
        if (!(ok = issue_o(1, j))) break;
        umma_commit(&v_empty[stage(j)]);
        if (more) {
          issue_s(1, j + 1);
          umma_commit(&k_empty[stage(j + 1)]);
        }
      }
      if (!ok) record_status(status, kStatusTimeout);
      umma_commit(mma_done);
    }
  } else if (warp >= 4) {
    // ================================================================ softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 200;\n" ::: "memory");
    if (!sink_softmax<DH>((warp - 4) >> 2, tmem, cur, dims, cut, s_full, o_done, p_half, p_ready,
                          scale_log2, out, status, budget_ns))
      record_status(status, kStatusTimeout);
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    mbar_wait(mma_done, 0, 200000000ull);
    tmem_dealloc(tmem, 512);
  }
}

// o and lse of (row, head) from its parts: a warp each, DH / 32 columns a
// lane; lane s holds part s's lse (at most 32 parts).
template <int DH>
__global__ void __launch_bounds__(256) sink_combine_kernel(const SinkDims dims, int splits,
                                                           const SinkOut parts,
                                                           __nv_bfloat16* __restrict__ o,
                                                           int64_t ld_o,
                                                           float* __restrict__ lse,
                                                           uint32_t* status) {
  constexpr int W = DH / 32;
  constexpr int U = 16;  // parts whose loads are in flight before the first weight is known
  after_wait();
  if (parts.zero_rest) sink_zero_rest(dims.cu_q, dims.B, dims.Lq, o, ld_o, dims.H * DH);
  const int64_t w = static_cast<int64_t>(blockIdx.x) * 8 + warp_id();
  const int r = static_cast<int>(w / dims.H), h = static_cast<int>(w % dims.H);
  if (r >= dims.Lq) return;
  if (dims.cu_q != nullptr &&  // rows of no sequence have no parts
      (r < sink_bound(dims.cu_q, 0, dims.Lq) || r >= sink_bound(dims.cu_q, dims.B, dims.Lq)))
    return;
  const int lane = lane_id();
  const int64_t at = static_cast<int64_t>(h) * dims.Lq + r;
  const int64_t step = static_cast<int64_t>(dims.H) * dims.Lq;
  using Vec = std::conditional_t<W == 4, float4, float2>;
  const Vec* src = reinterpret_cast<const Vec*>(
                       parts.part_o + (static_cast<int64_t>(r) * dims.H + h) * DH) + lane;
  const float part = lane < splits ? parts.part_lse[lane * step + at] : -INFINITY;
  Vec v[U];
#pragma unroll
  for (int s = 0; s < U; ++s)
    if (s < splits) v[s] = src[s * step * 32];
  float top = part;
#pragma unroll
  for (int x = 16; x > 0; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
  // a part that saw nothing weighs 0 (its fp32 rows are zeros); a NaN goes through
  const float f = part == -INFINITY ? 0.f : __expf(part - top);
  float sum = f;
#pragma unroll
  for (int x = 16; x > 0; x >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
  float acc[W] = {};
  auto add = [&](int s, const Vec& u) {
    const float fs = __shfl_sync(0xffffffffu, f, s);
    const float* x = reinterpret_cast<const float*>(&u);
#pragma unroll
    for (int c = 0; c < W; ++c) acc[c] += fs * x[c];
  };
#pragma unroll
  for (int s = 0; s < U; ++s)
    if (s < splits) add(s, v[s]);
#pragma unroll 8
  for (int s = U; s < splits; ++s) add(s, src[s * step * 32]);
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  if (!in_bounds(status, r, dims.Lq, static_cast<int64_t>(h) * DH, DH,
                 static_cast<int64_t>(dims.H) * DH))
    return;
  uint32_t* dst = reinterpret_cast<uint32_t*>(o + static_cast<int64_t>(r) * ld_o + h * DH) +
                  W / 2 * lane;
#pragma unroll
  for (int c = 0; c < W; c += 2) dst[c / 2] = pack_bf16x2(acc[c] * inv, acc[c + 1] * inv);
  if (lse != nullptr && lane == 0) lse[at] = sum == 0.f ? -INFINITY : top + logf(sum);
}

// Rows and splits of a unit, from the shape alone (the workspace depends on
// them).  Heads share a unit where their queries fill it together: while a
// sequence has on average no more queries than half the unit's (64 queries, 16
// heads over 4, 24000 keys: 44 us with a unit a head, 27 with one for four).
// Key tiles are split where units would leave half of 148 SMs idle, over as many
// CTAs as make the longest walk and the join together shortest.  Measured: a
// key tile takes 1.7 us (d 128) or 1.3 (64), a join 2.3 us and 0.45 for each MB
// of parts.  Queries of 16 heads over 4: 32 over 1000 keys 11.9 us and 17.0
// without a split, 64 over 6000 keys 19.6 and 22.3 with four tiles a split, 64
// over 24000 keys 30 with 32 splits and 35.7 with 18; 1500 tokens of 6 heads over
// 2 18.7 and 23.2 without; but 600 tokens of 8 heads 17.7 in five splits and 14.4
// in one.  The walk is bounded by the window and by the keys of all sequences
// together: many short sequences under a window that forgets nothing are split
// although each has a tile or two (16 of 100 tokens, 2 heads: five splits).
SinkCut sink_cut(const vdn_sink_shape& s) {
  SinkCut c{256, 1};
  const int group = s.H / s.H_kv, mean = (s.Lq + s.B - 1) / s.B;
  while (c.rows > 8 && mean <= c.rows / 2 && group % (512 / c.rows) == 0) c.rows /= 2;
  // the most that B sequences can have of Lq rows
  const int64_t slots = (s.Lq + static_cast<int64_t>(s.B) * (c.rows - 1)) / c.rows;
  const int64_t units = slots * (s.H * c.rows / 256 < 1 ? 1 : s.H * c.rows / 256);
  if (units < 1 || units > 74) return c;
  int64_t keys = static_cast<int64_t>(s.window) + s.ahead + c.rows + s.sinks;
  if (keys > s.Lk) keys = s.Lk;
  const int tiles = static_cast<int>((keys + 127) / 128);
  const float tile = s.d == 128 ? 1.7f : 1.3f;
  const float part = 0.45e-6f * 4.f * static_cast<float>(s.Lq) * s.H * s.d;
  float best = tiles * tile;
  for (int n = 2; n <= 32 && n * units <= 148 && n <= tiles; ++n) {
    const float t = (tiles + n - 1) / n * tile + 2.3f + n * part;
    if (t < best) best = t, c.splits = n;
  }
  return c;
}

size_t align256(size_t n) { return (n + 255) / 256 * 256; }

template <int DH>
cudaError_t launch_sink(const Launch& ctx, const SinkDims& dims, const SinkCut& cut,
                        const CUtensorMap& qmap, const CUtensorMap& kmap, const CUtensorMap& vmap,
                        float scale, __nv_bfloat16* o, int64_t ld_o, float* lse, bool zero_rest,
                        uint8_t* ws) {
  using Cfg = SinkCfg<DH>;
  static std::atomic<uint64_t> smem_set{0};
  if (cudaError_t e = set_smem_once(sink_attn_kernel<DH>, Cfg::SMEM, smem_set)) return e;
  SinkOut out{};
  const int splits = cut.splits;
  out.o = splits == 1 ? o : nullptr;
  out.ld_o = ld_o;
  out.lse = lse;
  out.zero_rest = zero_rest && dims.cu_q != nullptr;
  out.part_o = reinterpret_cast<float*>(ws + kStatusBytes);
  out.part_lse = reinterpret_cast<float*>(
      ws + kStatusBytes +
      align256(static_cast<size_t>(splits) * dims.Lq * dims.H * DH * sizeof(float)));
  const int grid = sink_slots(dims.Lq, dims.B, cut.rows) * (dims.H * cut.rows / 256) * splits;
  sink_attn_kernel<DH><<<grid, Cfg::THREADS, Cfg::SMEM, ctx.stream>>>(
      qmap, kmap, vmap, dims, cut, scale * 1.4426950408889634f, out, ctx.status, ctx.budget_ns);
  if (cudaError_t e = cudaGetLastError()) return e;
  if (splits > 1) {
    const int64_t warps = static_cast<int64_t>(dims.Lq) * dims.H;
    if (cudaError_t e = launch_after(sink_combine_kernel<DH>,
                                     dim3(static_cast<unsigned>((warps + 7) / 8)), 256, 0,
                                     ctx.stream, dims, splits, out, o, ld_o, lse, ctx.status))
      return e;
  }
  return cudaGetLastError();
}

}  // namespace

// Checks shared by the forward and the gradient call; `s` gets the clamped
// mask.
vdn_status sink_check(const vdn_sink_shape* shape, const void* q, int64_t ld_q, const void* k,
                      const void* v, int64_t ld_kv, const int32_t* cu_q, const int32_t* cu_k,
                      vdn_sink_shape* s) {
  if (shape == nullptr) return VDN_ERR_INVALID_ARG;
  *s = *shape;
  if (s->Lq < 0 || s->Lk < 0 || s->Lq > kSinkMax - 1024 || s->Lk > kSinkMax - 1024 || s->B < 1 ||
      s->B > (1 << 20) || s->H < 1 || s->H_kv < 1 || s->H % s->H_kv || s->d < 1)
    return VDN_ERR_INVALID_ARG;
  if (s->d != 64 && s->d != 128) return VDN_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(s->H) * s->d >= (int64_t(1) << 24)) return VDN_ERR_INVALID_ARG;
  if (s->window < 1 || s->ahead < 0 || s->sinks < 0) return VDN_ERR_INVALID_ARG;
  if (s->window > kSinkMax) s->window = kSinkMax;
  if (s->ahead > kSinkMax) s->ahead = kSinkMax;
  if (s->sinks > kSinkMax) s->sinks = kSinkMax;
  auto bad = [](const void* p, int rows) {
    return (p == nullptr && rows > 0) || (reinterpret_cast<uintptr_t>(p) & 15u);
  };
  if (bad(q, s->Lq) || bad(k, s->Lk) || bad(v, s->Lk)) return VDN_ERR_INVALID_ARG;
  if (ld_q < static_cast<int64_t>(s->H) * s->d || ld_q % 8 ||
      ld_kv < static_cast<int64_t>(s->H_kv) * s->d || ld_kv % 8)
    return VDN_ERR_INVALID_ARG;
  if (s->B > 1 && (cu_q == nullptr || cu_k == nullptr)) return VDN_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(cu_q) & 3u) || (reinterpret_cast<uintptr_t>(cu_k) & 3u))
    return VDN_ERR_INVALID_ARG;
  return VDN_OK;
}

}  // namespace vdn

using namespace vdn;

extern "C" {

size_t vdn_sink_attn_workspace(const vdn_sink_shape* shape) {
  vdn_sink_shape s;
  const void* p = reinterpret_cast<const void*>(256);
  if (shape == nullptr ||
      sink_check(shape, p, (int64_t)1 << 24, p, p, (int64_t)1 << 24,
                 static_cast<const int32_t*>(p), static_cast<const int32_t*>(p), &s) != VDN_OK)
    return 0;
  const int n = sink_cut(s).splits;
  if (n == 1) return kStatusBytes;
  const size_t rows = static_cast<size_t>(n) * s.Lq * s.H;
  return kStatusBytes + align256(rows * s.d * sizeof(float)) + align256(rows * sizeof(float));
}

vdn_status vdn_sink_attn(const vdn_sink_shape* shape, const void* q, int64_t ld_q, const void* k,
                         const void* v, int64_t ld_kv, const int32_t* cu_q, const int32_t* cu_k,
                         float scale, void* o, int64_t ld_o, int zero_rest, float* lse_opt,
                         void* ws, size_t ws_bytes, void* stream) {
  NvtxRange nvtx("vdn_sink_attn");
  vdn_sink_shape s;
  const vdn_status r = sink_check(shape, q, ld_q, k, v, ld_kv, cu_q, cu_k, &s);
  if (r != VDN_OK) return r;
  const int64_t D = static_cast<int64_t>(s.H) * s.d, Dk = static_cast<int64_t>(s.H_kv) * s.d;
  if ((o == nullptr && s.Lq > 0) || (reinterpret_cast<uintptr_t>(o) & 15u) || ld_o < D ||
      ld_o % 8 || (reinterpret_cast<uintptr_t>(lse_opt) & 3u))
    return VDN_ERR_INVALID_ARG;
  if (ws == nullptr || (reinterpret_cast<uintptr_t>(ws) & 255u) ||
      ws_bytes < vdn_sink_attn_workspace(shape))
    return VDN_ERR_WORKSPACE;
  if (s.Lq == 0) return VDN_OK;
  const SinkCut cut = sink_cut(s);
  if (static_cast<int64_t>(sink_slots(s.Lq, s.B, cut.rows)) * s.H * cut.splits >=
          (int64_t(1) << 31) ||
      static_cast<int64_t>(s.Lq) * s.H >= (int64_t(1) << 33))
    return VDN_ERR_UNSUPPORTED;
  const SinkDims dims{s.Lq, s.Lk, s.B, s.H, s.H_kv, cu_q, cu_k, {s.window, s.ahead, s.sinks}};
  CUtensorMap qmap, kmap, vmap;
  if (!make_rows_map(&qmap, q, D, ld_q, s.Lq, cut.rows < 128 ? cut.rows : 128)) return VDN_ERR_CUDA;
  kmap = vmap = qmap;  // no keys: never loaded
  if (s.Lk > 0 && (!make_rows_map(&kmap, k, Dk, ld_kv, s.Lk, 128) ||
                   !make_rows_map(&vmap, v, Dk, ld_kv, s.Lk, 128)))
    return VDN_ERR_CUDA;
  const Launch ctx{static_cast<cudaStream_t>(stream), static_cast<uint32_t*>(ws),
                   current_wait_budget_ns()};
  const float sc = scale > 0.f ? scale : 1.f / sqrtf(static_cast<float>(s.d));
  auto* ob = static_cast<__nv_bfloat16*>(o);
  auto* wb = static_cast<uint8_t*>(ws);
  const bool z = zero_rest != 0;
  const cudaError_t e =
      s.d == 128
          ? launch_sink<128>(ctx, dims, cut, qmap, kmap, vmap, sc, ob, ld_o, lse_opt, z, wb)
          : launch_sink<64>(ctx, dims, cut, qmap, kmap, vmap, sc, ob, ld_o, lse_opt, z, wb);
  return e == cudaSuccess ? VDN_OK : VDN_ERR_CUDA;
}

}  // extern "C"
