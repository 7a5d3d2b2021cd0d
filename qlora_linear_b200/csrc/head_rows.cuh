// head_rows.cuh — the head's forward (head.cuh) for a few rows: single tokens and decoding
// batches of up to 128.
//
// Bound by HBM: the head W [V, D] is read once, 2·V·D bytes, against 2·M·V·D flops.  One CTA
// per SM owns a contiguous range of vocabulary entries (multiples of 16, so the ranges differ
// by at most 16) and walks it in tiles of up to 128 entries; X stays in L2.  Per tile the
// tensor core computes the 128 × 128 accumulator of all rows (unused rows hold whatever shared
// memory held; nobody reads them): half of what a CTA pair's 256 rows would cost for the same
// bytes of W.  The statistics and the alternatives' bound stay with the CTA over its whole range,
// so a row leaves one partial a CTA.
//
// W goes through a ring of stages of 128 entries × 128 of the D columns, which HBM serves in
// 256-byte pieces (V = 128256, D = 4096, 1 row: 182 us with them, 186 us with 256 entries × 64,
// 196 us with 64 × 256; V = 32000, D = 8192: 121, 140 and 122 us).  A range's last tile takes boxes
// of 64, 32 and 16 entries.  The stages' number follows from what X leaves of shared memory (6 up
// to 8 rows, 3 at 128).
// Roles: warp 0 TMA producer, warp 1 MMA issuer and TMEM owner, warps 2-5 epilogue (thread =
// row).  Every wait is bounded.
#pragma once

#include "head.cuh"

namespace lora {

constexpr int HR_ROWS = 128;        // rows at most
constexpr int HR_BN = 128;          // vocabulary entries a tile
constexpr int HR_BK = 128;          // of D per stage: two 64-wide swizzle atoms
constexpr int HR_ATOMS = HR_BK / 64;
constexpr int HR_UNIT = 16;         // granularity of the CTAs' ranges
constexpr int HR_MAX_STAGES = 6;
constexpr int HR_THREADS = 192;
constexpr int HR_W_BYTES = HR_BN * HR_BK * 2;  // 32 KB
constexpr int HR_SMEM_MAX = 232448 - 2048;  // dynamic; the barriers are static

// CTAs: one per SM, at least 32 entries each.
__host__ __device__ constexpr int hr_ctas(long long V) {
  return static_cast<int>((V + 31) / 32 < 148 ? (V + 31) / 32 : 148);
}
// Bytes of X in a stage: the rows rounded up to the 8-row swizzle atom.
__host__ __device__ constexpr int hr_x_bytes(int M) { return (M + 7) / 8 * 8 * HR_BK * 2; }
// Stages that fit; the MMA reads 128 rows of X from any stage, so as many must fit behind the
// last stage's W.
__host__ __device__ constexpr int hr_stages(int M) {
  const int behind = (128 - (M + 7) / 8 * 8) * 128;
  const int n = (HR_SMEM_MAX - 1024 - behind) / (HR_W_BYTES + hr_x_bytes(M));
  return n < HR_MAX_STAGES ? n : HR_MAX_STAGES;
}
// Chunks of 32 entries of the longest range.
__host__ __device__ constexpr int hr_chunks(long long V) {
  return static_cast<int>((((V + 15) / 16 + hr_ctas(V) - 1) / hr_ctas(V) + 1) / 2);
}

struct HeadRowsParams {
  HeadArgs h;              // sorted and bound are not used; part is [M][CTAs]
  int cpp;                 // chunks a CTA (cmax is [M][CTAs · cpp])
  const int32_t* ids;      // [M][n]
  int M, V, D;
  int stages;
  uint32_t* status;
  uint64_t wait_ns;
};

// The head in boxes of 64 columns × 128, 64, 32 and 16 entries.
struct HeadRowsMaps {
  CUtensorMap box[4];
};

// A third look at the tile, for the alternatives: the column groups' maxima over the CTA's range
// so far, and the least of the kp groups that they fold into.
__device__ __forceinline__ float head_rows_bound(const HeadArgs& h, uint32_t tbase, int nv, float (&groups)[32]) {
#pragma unroll 1
  for (int c = 0; c * 32 < nv; ++c) {
    uint32_t v[32];
    tmem_ld_32x32b_x32(tbase + c * 32, v);
    tmem_ld_wait();
    const int n = nv - c * 32;
#pragma unroll
    for (int j = 0; j < 32; ++j)
      if (j < n) groups[j] = fmaxf(groups[j], __uint_as_float(v[j]));
  }
  float g[32];
#pragma unroll
  for (int j = 0; j < 32; ++j) g[j] = groups[j];
#pragma unroll
  for (int s = 16; s > 0; s >>= 1)
    if (h.kp <= s) {
#pragma unroll
      for (int j = 0; j < s; ++j) g[j] = fmaxf(g[j], g[j + s]);
    }
  float low = g[0];
#pragma unroll
  for (int j = 1; j < 32; ++j)
    if (j < h.kp) low = fminf(low, g[j]);
  return low;
}

__global__ void __launch_bounds__(HR_THREADS, 1)
    head_rows_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ HeadRowsMaps tmW,
                     const HeadRowsParams p) {
  griddep_enter();  // the previous kernel in the stream completed (see ptx.cuh)
  extern __shared__ __align__(1024) uint8_t hr_raw[];
  __shared__ __align__(8) uint64_t full[HR_MAX_STAGES], empty[HR_MAX_STAGES], tfull[2], tempty[2], drain;
  __shared__ uint32_t tmem_slot, abort_s, never_s;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(hr_raw) + 1023) & ~uintptr_t(1023));

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int S = p.stages;
  const int xbytes = hr_x_bytes(p.M);
  const int stage_bytes = HR_W_BYTES + xbytes;
  const int r0 = hr_first(p.V, blockIdx.x, gridDim.x);
  const int r1 = hr_first(p.V, blockIdx.x + 1, gridDim.x);
  const int ntiles = (r1 - r0 + HR_BN - 1) / HR_BN;
  const int nkb = (p.D + HR_BK - 1) / HR_BK;
  const WaitCtl wc{&abort_s, p.status, p.wait_ns};

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(smem_u32(&full[s]), 1);
      mbar_init(smem_u32(&empty[s]), 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(smem_u32(&tfull[a]), 1);
      mbar_init(smem_u32(&tempty[a]), 4);
    }
    mbar_init(smem_u32(&drain), 1);
    abort_s = 0;
    never_s = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tmX);
    tma_prefetch_desc(&tmW.box[0]);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(&tmem_slot), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = tmem_slot;

  if (warp == 0) {
    // ------------------------------------------------------------ TMA producer
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      long long fills = 0;
      bool ok = true;
      for (int t = 0; ok && t < ntiles; ++t) {
        const int v0 = r0 + t * HR_BN;
        const int rows = min(HR_BN, r1 - v0);  // a multiple of 16
        // checked build: the tile starts inside the head and its boxes inside the stage
        if (!lora_check(v0 < p.V && rows > 0 && rows % HR_UNIT == 0 && p.M <= HR_ROWS && S <= HR_MAX_STAGES, wc)) {
          ok = false;
          break;
        }
        for (int kb = 0; kb < nkb; ++kb) {
          if (!mbar_wait(smem_u32(&empty[stage]), phase ^ 1u, wc)) { ok = false; break; }
          const uint32_t sW = smem_u32(smem + stage * stage_bytes);
          const uint32_t bar = smem_u32(&full[stage]);
          mbar_arrive_expect_tx(bar, rows * HR_BK * 2 + xbytes);
#pragma unroll
          for (int a = 0; a < HR_ATOMS; ++a) {
            const int x = kb * HR_BK + a * 64;
            int u = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (rows & (HR_BN >> i)) {
                tma_load_2d(sW + a * (HR_W_BYTES / HR_ATOMS) + u * 128, &tmW.box[i], bar, x, v0 + u);
                u += HR_BN >> i;
              }
            tma_load_2d(sW + HR_W_BYTES + a * (xbytes / HR_ATOMS), &tmX, bar, x, 0);
          }
          ++fills;
          if (++stage == S) { stage = 0; phase ^= 1u; }
        }
      }
      // after an abort, loads still in flight land before shared memory goes away
      if (!ok) {
        const WaitCtl drain_wc{&never_s, nullptr, p.wait_ns};
        for (long long f = fills > S ? fills - S : 0; f < fills; ++f)
          mbar_wait(smem_u32(&full[f % S]), static_cast<uint32_t>((f / S) & 1), drain_wc);
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0, acc_phase = 0;
      int acc = 0;
      bool ok = true;
      for (int t = 0; ok && t < ntiles; ++t) {
        const uint32_t idesc = idesc_bf16_f32(HR_ROWS, min(HR_BN, r1 - r0 - t * HR_BN), false, false);
        if (!mbar_wait(smem_u32(&tempty[acc]), acc_phase ^ 1u, wc)) break;
        tc_fence_after();
        for (int kb = 0; kb < nkb; ++kb) {
          if (!mbar_wait(smem_u32(&full[stage]), phase, wc)) { ok = false; break; }
          tc_fence_after();
          const uint32_t sW = smem_u32(smem + stage * stage_bytes);
#pragma unroll
          for (int k = 0; k < HR_BK / 16; ++k)
            tc_mma_bf16(tmem_base + acc * HR_BN,
                        sdesc_sw128(sW + HR_W_BYTES + (k >> 2) * (xbytes / HR_ATOMS) + (k & 3) * 32, 16, 1024),
                        sdesc_sw128(sW + (k >> 2) * (HR_W_BYTES / HR_ATOMS) + (k & 3) * 32, 16, 1024), idesc,
                        (kb > 0 || k > 0) ? 1u : 0u);
          tc_commit(smem_u32(&empty[stage]));
          if (++stage == S) { stage = 0; phase ^= 1u; }
        }
        if (!ok) break;
        tc_commit(smem_u32(&tfull[acc]));
        if (++acc == 2) { acc = 0; acc_phase ^= 1u; }
      }
      // every MMA issued so far must finish before TMEM is released
      tc_commit(smem_u32(&drain));
      const WaitCtl drain_wc{&never_s, nullptr, p.wait_ns};
      mbar_wait(smem_u32(&drain), 0, drain_wc);
    }
  } else {
    // ------------------------------------------------------------ epilogue (thread = row)
    const int quarter = warp & 3;
    const int row = quarter * 32 + lane;
    const bool in = row < p.M;
    const HeadArgs& h = p.h;
    RowStats st{-INFINITY, 0.0f, 0.0f};
    float raw = -INFINITY;  // the largest accumulator (st.m in units of log 2)
    float groups[32];  // maxima of the CTA's logits by tile column mod kp: their least is a bound
#pragma unroll
    for (int j = 0; j < 32; ++j) groups[j] = -INFINITY;
    float low = -INFINITY;
    const size_t at = static_cast<size_t>(row) * gridDim.x + blockIdx.x;
    int acc = 0;
    uint32_t acc_phase = 0;
    bool ok = true;
    for (int t = 0; t < ntiles; ++t) {
      if (!mbar_wait_warp(smem_u32(&tfull[acc]), acc_phase, wc)) { ok = false; break; }
      tc_fence_after();
      if (quarter * 32 < p.M) {  // a warp without rows has nothing to read
        const int v0 = r0 + t * HR_BN;
        const int nv = min(HR_BN, min(r1, p.V) - v0);
        const uint32_t tbase = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) + acc * HR_BN;
        for (int i = 0; i < h.n; ++i) {
          int col = -1;
          if (in) {
            const uint32_t off = static_cast<uint32_t>(p.ids[static_cast<size_t>(row) * h.n + i]) - static_cast<uint32_t>(v0);
            if (off < static_cast<uint32_t>(nv)) col = static_cast<int>(off);
          }
          uint32_t want = __ballot_sync(0xffffffffu, col >= 0);
          while (want) {
            const int at = __shfl_sync(0xffffffffu, col, __ffs(want) - 1);
            const float z = __uint_as_float(tmem_ld_32x32b_x1(tbase + at));
            if (col == at) h.id_logit[static_cast<size_t>(row) * h.n + i] = z;
            want &= ~__ballot_sync(0xffffffffu, col == at);
          }
        }
        float cm[HR_BN / 32];
        const float tile_max = head_tile_max<HR_BN / 32>(tbase, nv, cm), m = tile_max * h.c2;
        raw = fmaxf(raw, tile_max);
        uint32_t hits = 0;
        if (h.k > 0) {
          low = head_rows_bound(h, tbase, nv, groups);
          if (in) {
#pragma unroll
            for (int c = 0; c < HR_BN / 32; ++c)
              if (t * (HR_BN / 32) + c < p.cpp) {
                h.cmax[at * p.cpp + t * (HR_BN / 32) + c] = cm[c];
                if (c * 32 < nv && cm[c] >= low) hits |= 1u << c;
              }
          }
          __syncwarp();
        }
        st = join_stats(st, head_tile_sums(tbase, nv, h.c2, m, hits,
                                           h.zlog + static_cast<size_t>(row) * p.V + v0));
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&tempty[acc]));
      if (++acc == 2) { acc = 0; acc_phase ^= 1u; }
    }
    if (ok && in) {
      h.part[at] = make_float4(raw, st.s, st.t, low);
      if (h.k > 0)  // a range may be a chunk shorter than the longest
        for (int c = ntiles * (HR_BN / 32); c < p.cpp; ++c) h.cmax[at * p.cpp + c] = -INFINITY;
    }
  }

  // ------------------------------------------------------------ teardown
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, 512);
  }
}

}  // namespace lora
