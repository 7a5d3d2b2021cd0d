// head_rows.cuh — the head's forward (head.cuh) for a few rows: single tokens and decoding
// batches of up to 128.
//
// Bound by HBM: the head W [V, D] is read once, 2·V·D bytes, against 2·M·V·D flops.  One CTA
// per SM owns a contiguous range of vocabulary entries (multiples of 16, so the ranges differ
// by at most 16) and walks it in tiles of up to 128; X stays in L2.  The vocabulary is the
// MMA's M dimension (128) and the rows its N (16 to 128): the tensor core works for the rows
// there are.  (With the roles the other way round, 128 rows of which few are real, the GPU's power
// limit lowered the clock and one row took 194 us instead of 171.)
//
// W goes through a ring of stages of 128 entries × 128 of the D columns, which HBM serves in
// 256-byte pieces, each CTA starting at another column (V = 128256, D = 4096, 1 row, with an earlier
// issue loop: 182 us; 186 us with 256 entries × 64, 196 us with 64 × 256).  A range's last tile takes boxes of 64, 32
// and 16 entries.  The producer and the MMA issuer run as whole warps that issue under elect_one():
// under `lane == 0` a TMA load cost its thread 230 cycles and an MMA 78, 1200 and 900 a fill, which
// bounded short ranges (16 rows, V = 280, D = 8192: 48 us, now 29) and left HBM little slack.
//
// Epilogue: a lane holds one entry's logits of 32 rows.  Sums over the 32 entries of a warp go
// by transposing reductions (31 shuffles for 32 rows, lane i ending with row i), so a warp keeps the
// running statistics of row i in lane i, and leaves one partial a CTA, warp and row.
//
// Alternatives: a warp's 32 entries are a chunk.  Its maxima are written, and its logits of the rows
// whose maximum reaches a bound of their k-th largest logit (as the pair kernel's: the least of kp
// groups' maxima over the chunks seen; a chunk below it has k better ones, so none of its entries is
// wanted).  The bounds' first values have to come before their first use without a grid barrier or
// another launch: one warp clears them and sets `live`, a warp that does not see it yet keeps
// everything and raises nothing, and the row kernel behind clears `live`.  How much is written varies,
// the results do not.  Once a tile and row a CTA reads the bounds, through shared memory: read by every
// warp, the 128 bytes a row for k > 16 cost more than the stores saved (48 rows, k = 20: 195 us).  All
// logits written: 189 us, and 182 so; k = 1: 182 and 172.
//
// Given tokens: a warp looks at its 32 rows' ids one position after the other, 4·n loads and votes a
// tile for 128 rows.  Long lists on many rows take longer than the products (128 rows, V = 128256,
// D = 4096: 187 us at n = 1, 194 at 16, 680 at 128; D = 256: 58, 112 and 620).
//
// W's lines leave L2 first (evict_first), so the logits stay for the row kernel: 1 row, k = 8 163 -> 159 us,
// 8 rows 171 -> 165; with all logits written 48 rows lost 1.5% to it.
//
// Roles: warp 0 TMA producer, warp 1 MMA issuer and TMEM owner, warps 2-5 epilogue.  Every wait
// is bounded.
#pragma once

#include "head.cuh"

namespace lora {

constexpr int HR_ROWS = 128;        // rows at most
constexpr int HR_BN = 128;          // vocabulary entries a tile
constexpr int HR_BK = 128;          // of D per stage: two 64-wide swizzle atoms
constexpr int HR_ATOMS = HR_BK / 64;
constexpr int HR_UNIT = 16;         // granularity of the CTAs' ranges
// 128 KB of W in flight a SM; with more HBM gets slower (V = 128256, D = 4096, 5 rows: 165, 160, 163
// and 167 us with 3, 4, 5 and 6 stages).
constexpr int HR_MAX_STAGES = 4;
constexpr int HR_THREADS = 192;
constexpr int HR_WARPS = 4;         // epilogue warps: partials a CTA
constexpr int HR_W_BYTES = HR_BN * HR_BK * 2;  // 32 KB
constexpr int HR_SMEM_MAX = 232448 - 2048;  // dynamic; the barriers are static

// CTAs: one per SM, at least 32 entries each.
__host__ __device__ constexpr int hr_ctas(long long V) {
  return static_cast<int>((V + 31) / 32 < 148 ? (V + 31) / 32 : 148);
}
// Rows of the MMA's N dimension, and X's bytes in a stage.
__host__ __device__ constexpr int hr_n(int M) { return (M + 15) / 16 * 16; }
__host__ __device__ constexpr int hr_x_bytes(int M) { return hr_n(M) * HR_BK * 2; }
__host__ __device__ constexpr int hr_stages(int M) {
  const int n = (HR_SMEM_MAX - 1024) / (HR_W_BYTES + hr_x_bytes(M));
  return n < HR_MAX_STAGES ? n : HR_MAX_STAGES;
}
// Chunks of 32 entries of the longest range.
__host__ __device__ constexpr int hr_chunks(long long V) {
  return static_cast<int>((((V + 15) / 16 + hr_ctas(V) - 1) / hr_ctas(V) + 1) / 2);
}

struct HeadRowsParams {
  HeadArgs h;              // sorted is not used; part is [M][4·CTAs]
  int cpp;                 // chunks a CTA (cmax is [M][CTAs · cpp])
  const int32_t* ids;      // [M][n]
  int M, V, D;
  int stages;
  uint32_t* live;          // not 0 once the bounds are cleared
  uint32_t* status;
  uint64_t wait_ns;
};

// The head in boxes of 64 columns × 128, 64, 32 and 16 entries.
struct HeadRowsMaps {
  CUtensorMap box[4];
};

// x[i] of every lane reduced over the lanes, into lane i.
template <typename Op>
__device__ __forceinline__ float transpose_reduce(float (&x)[32], int lane, Op op) {
#pragma unroll
  for (int s = 16; s > 0; s >>= 1) {
    const bool hi = lane & s;
#pragma unroll
    for (int j = 0; j < s; ++j) {
      const float give = hi ? x[j] : x[j + s], keep = hi ? x[j + s] : x[j];
      x[j] = op(keep, __shfl_xor_sync(0xffffffffu, give, s));
    }
  }
  return x[0];
}

__global__ void __launch_bounds__(HR_THREADS, 1)
    head_rows_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ HeadRowsMaps tmW,
                     const HeadRowsParams p) {
  griddep_enter();  // the previous kernel in the stream completed (see ptx.cuh)
  extern __shared__ __align__(1024) uint8_t hr_raw[];
  __shared__ __align__(8) uint64_t full[HR_MAX_STAGES], empty[HR_MAX_STAGES], tfull[2], tempty[2], drain;
  __shared__ uint32_t tmem_slot, abort_s, never_s;
  // bounds of the rows' k-th largest logits (ord_f32); a warp refreshes 32 rows' and reads the others'
  // as they are: they only rise, an older one keeps more
  __shared__ uint32_t lows[HR_ROWS];
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

  if (threadIdx.x < HR_ROWS) lows[threadIdx.x] = 0;
  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(smem_u32(&full[s]), 1);
      mbar_init(smem_u32(&empty[s]), 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(smem_u32(&tfull[a]), 1);
      mbar_init(smem_u32(&tempty[a]), HR_WARPS);
    }
    mbar_init(smem_u32(&drain), 1);
    abort_s = 0;
    never_s = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tmX);
    tma_prefetch_desc(&tmW.box[0]);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(&tmem_slot), 2 * HR_ROWS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = tmem_slot;

  if (warp == 0) {
    // ------------------------------------------------------------ TMA producer
    {
      int stage = 0;
      uint32_t phase = 0;
      long long fills = 0;
      bool ok = true;
      const uint64_t once = l2_evict_first();
      const int shift = static_cast<int>(static_cast<long long>(blockIdx.x) * nkb / gridDim.x);
      for (int t = 0; ok && t < ntiles; ++t) {
        const int v0 = r0 + t * HR_BN;
        const int rows = min(HR_BN, r1 - v0);  // a multiple of 16
        // checked build: the tile starts inside the head and its boxes inside the stage
        if (!lora_check(v0 < p.V && rows > 0 && rows % HR_UNIT == 0 && p.M <= HR_ROWS && S <= HR_MAX_STAGES, wc)) {
          ok = false;
          break;
        }
        for (int kb = 0; kb < nkb; ++kb) {
          if (!mbar_wait_warp(smem_u32(&empty[stage]), phase ^ 1u, wc)) { ok = false; break; }
          const int kx = kb + shift < nkb ? kb + shift : kb + shift - nkb;
          const uint32_t sW = smem_u32(smem + stage * stage_bytes);
          const uint32_t bar = smem_u32(&full[stage]);
          if (elect_one()) {
            mbar_arrive_expect_tx(bar, rows * HR_BK * 2 + xbytes);
#pragma unroll
            for (int a = 0; a < HR_ATOMS; ++a) {
              const int x = kx * HR_BK + a * 64;
              int u = 0;
#pragma unroll
              for (int i = 0; i < 4; ++i)
                if (rows & (HR_BN >> i)) {
                  tma_load_2d_hint(sW + a * (HR_W_BYTES / HR_ATOMS) + u * 128, &tmW.box[i], bar, x, v0 + u, once);
                  u += HR_BN >> i;
                }
              tma_load_2d(sW + HR_W_BYTES + a * (xbytes / HR_ATOMS), &tmX, bar, x, 0);
            }
          }
          __syncwarp();
          ++fills;
          if (++stage == S) { stage = 0; phase ^= 1u; }
        }
      }
      // after an abort, loads still in flight land before shared memory goes away
      if (!ok) {
        const WaitCtl drain_wc{&never_s, nullptr, p.wait_ns};
        for (long long f = fills > S ? fills - S : 0; f < fills; ++f)
          mbar_wait_warp(smem_u32(&full[f % S]), static_cast<uint32_t>((f / S) & 1), drain_wc);
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    {
      // entries a last tile did not load hold what shared memory held: their lanes are not used
      const uint32_t idesc = idesc_bf16_f32(HR_BN, hr_n(p.M), false, false);
      const uint64_t w_desc = sdesc_sw128(smem_u32(smem), 16, 1024);
      const uint64_t x_desc = sdesc_sw128(smem_u32(smem) + HR_W_BYTES, 16, 1024);
      int stage = 0;
      uint32_t phase = 0, acc_phase = 0;
      int acc = 0;
      bool ok = true;
      for (int t = 0; ok && t < ntiles; ++t) {
        if (!mbar_wait_warp(smem_u32(&tempty[acc]), acc_phase ^ 1u, wc)) break;
        tc_fence_after();
        const uint64_t w_atom = (HR_W_BYTES / HR_ATOMS) >> 4, x_atom = (xbytes / HR_ATOMS) >> 4;
        for (int kb = 0; kb < nkb; ++kb) {
          if (!mbar_wait_warp(smem_u32(&full[stage]), phase, wc)) { ok = false; break; }
          tc_fence_after();
          // the descriptors' address field counts 16 bytes: a step of 16 columns is 2
          const uint64_t wd = w_desc + ((stage * stage_bytes) >> 4), xd = x_desc + ((stage * stage_bytes) >> 4);
          const uint32_t d = tmem_base + acc * HR_ROWS;
          if (elect_one()) {
#pragma unroll
            for (int k = 0; k < HR_BK / 16; ++k)
              tc_mma_bf16(d, wd + (k >> 2) * w_atom + (k & 3) * 2, xd + (k >> 2) * x_atom + (k & 3) * 2, idesc,
                          (kb > 0 || k > 0) ? 1u : 0u);
            tc_commit(smem_u32(&empty[stage]));
          }
          __syncwarp();
          if (++stage == S) { stage = 0; phase ^= 1u; }
        }
        if (!ok) break;
        if (elect_one()) tc_commit(smem_u32(&tfull[acc]));
        __syncwarp();
        if (++acc == 2) { acc = 0; acc_phase ^= 1u; }
      }
      // every MMA issued so far must finish before TMEM is released
      if (elect_one()) tc_commit(smem_u32(&drain));
      __syncwarp();
      const WaitCtl drain_wc{&never_s, nullptr, p.wait_ns};
      mbar_wait_warp(smem_u32(&drain), 0, drain_wc);
    }
  } else {
    // ------------------------------------------------------------ epilogue
    const int quarter = warp & 3;
    const HeadArgs& h = p.h;
    // one warp of the grid clears the bounds
    if (h.k > 0 && blockIdx.x == 0 && warp == 2) {
      for (int i = lane; i < p.M * h.kp; i += 32) h.bound[i] = 0u;
      __threadfence();
      __syncwarp();
      if (lane == 0) atomicExch(p.live, 1u);
    }
    const int np = static_cast<int>(gridDim.x) * HR_WARPS, pi = static_cast<int>(blockIdx.x) * HR_WARPS + quarter;
    constexpr int GROUPS = HR_ROWS / 32;
    RowStats st[GROUPS];  // of row 32·g + lane
    float raw[GROUPS];    // their largest accumulators (st.m in units of log 2)
#pragma unroll
    for (int g = 0; g < GROUPS; ++g) {
      st[g] = RowStats{-INFINITY, 0.0f, 0.0f};
      raw[g] = -INFINITY;
    }
    int acc = 0;
    uint32_t acc_phase = 0;
    bool ok = true;
    volatile uint32_t* vlow = lows;
    bool live = false;
    for (int t = 0; t < ntiles; ++t) {
      const int mine = quarter * 32 + lane;
      if (live && mine < p.M) vlow[mine] = head_bound(h.bound + static_cast<size_t>(mine) * h.kp, h.kp);
      if (!mbar_wait_warp(smem_u32(&tfull[acc]), acc_phase, wc)) { ok = false; break; }
      if (h.k > 0 && !live) {
        live = __shfl_sync(0xffffffffu, lane == 0 ? ld_acquire_gpu(p.live) : 0u, 0) != 0u;
        __syncwarp();
      }
      tc_fence_after();
      const int c0 = r0 + t * HR_BN + quarter * 32;  // the warp's chunk of entries
      const int nc = min(32, min(r1, p.V) - c0);     // <= 0: past the range
      const bool valid = lane < nc;
      const uint32_t tbase = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) + acc * HR_ROWS;
#pragma unroll
      for (int g = 0; g < GROUPS; ++g) {
        if (g * 32 >= p.M || nc <= 0) break;  // warp-uniform
        const int row = g * 32 + lane;
        uint32_t v[32];
        tmem_ld_32x32b_x32(tbase + g * 32, v);  // columns past the MMA's N are not used
        tmem_ld_wait();
        // given tokens: row i's ids are looked at by lane i, their logits stored by the lanes that
        // hold their entries
        for (int i = 0; i < h.n; ++i) {
          uint32_t off = 0xffffffffu;
          if (row < p.M)
            off = static_cast<uint32_t>(p.ids[static_cast<size_t>(row) * h.n + i]) - static_cast<uint32_t>(c0);
          uint32_t want = __ballot_sync(0xffffffffu, off < static_cast<uint32_t>(nc));
          while (want) {
            const int r = __ffs(want) - 1;
            want &= want - 1;
            const uint32_t at = __shfl_sync(0xffffffffu, off, r);
            const uint32_t z = tmem_ld_32x32b_x1(tbase + g * 32 + r);
            if (lane == at) h.id_logit[static_cast<size_t>(g * 32 + r) * h.n + i] = __uint_as_float(z);
            __syncwarp();
          }
        }
        const uint32_t low = vlow[row];
        float x[32];
#pragma unroll
        for (int j = 0; j < 32; ++j) x[j] = valid ? __uint_as_float(v[j]) : -INFINITY;
        const float top = transpose_reduce(x, lane, [](float a, float b) { return fmaxf(a, b); });
        if (h.k > 0) {
          const uint32_t o = ord_f32(fmaxf(top, -INFINITY));
          const bool keep = row < p.M && o >= low;
          const uint32_t kept = __ballot_sync(0xffffffffu, keep);
          if (row < p.M)
            h.cmax[(static_cast<size_t>(row) * gridDim.x + blockIdx.x) * p.cpp + t * (HR_BN / 32) + quarter] =
                fmaxf(top, -INFINITY);
          if (live && keep)
            atomicMax(h.bound + static_cast<size_t>(row) * h.kp + ((blockIdx.x * HR_WARPS + quarter + t) & (h.kp - 1)), o);
          if (valid) {
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (kept >> j & 1u)
                h.zlog[static_cast<size_t>(g * 32 + j) * p.V + c0 + lane] = __uint_as_float(v[j]);
          }
        }
        const float m = head_max_y(top, h.c2);
        float y[32];
#pragma unroll
        for (int j = 0; j < 32; ++j) {
          const float d = fmaf(__uint_as_float(v[j]), h.c2, -__shfl_sync(0xffffffffu, m, j));
          const float e = ex2_approx(d);
          x[j] = valid ? e : 0.0f;
          y[j] = valid ? d * e : 0.0f;
        }
        const float s = transpose_reduce(x, lane, [](float a, float b) { return a + b; });
        const float dt = transpose_reduce(y, lane, [](float a, float b) { return a + b; });
        st[g] = join_stats(st[g], RowStats{m, s, dt});
        raw[g] = fmaxf(raw[g], top);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&tempty[acc]));
      if (++acc == 2) { acc = 0; acc_phase ^= 1u; }
    }
    if (ok) {
#pragma unroll
      for (int g = 0; g < GROUPS; ++g) {
        const int row = g * 32 + lane;
        if (row >= p.M) continue;
        h.part[static_cast<size_t>(row) * np + pi] = make_float4(raw[g], st[g].s, st[g].t, 0.0f);
        // chunks that a shorter range does not have
        for (int c = (r1 - r0 + 31) / 32 + quarter; h.k > 0 && c < p.cpp; c += HR_WARPS)
          h.cmax[(static_cast<size_t>(row) * gridDim.x + blockIdx.x) * p.cpp + c] = -INFINITY;
      }
    }
  }

  // ------------------------------------------------------------ teardown
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, 2 * HR_ROWS);
  }
}

}  // namespace lora
