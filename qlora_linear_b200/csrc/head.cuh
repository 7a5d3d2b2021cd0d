// head.cuh — per-row work over a frozen LM head, never writing the logits: what the GEMMs'
// head epilogues compute from an accumulator tile, and the row kernels around them.
//
// With hidden states X [M, D], head W [V, D] and z = scale·X·Wᵀ:
//
//   forward    lse = log Σ_v e^{z_v},   H = lse - Σ_v p_v z_v  (p = e^{z-lse}),
//              lp_i = z_{id_i} - lse of the given tokens, the k largest z with their ids
//   backward   dz_v = Σ_{i: id_i = v} c_i - p_v·(Σ_i c_i + g_H·(log p_v + H)),  dX = scale·dz·W
//
// for upstream gradients c_i of lp_i and g_H of H.  Distillation over a teacher's list is the
// case c_i = -g·q_i, g_H = 0 (q the softmax of the listed teacher logits).
//
// Everything between the accumulator and the row kernels is in units of log 2: with
// y = c·acc, c = scale/ln 2 (rounded once), e^z = 2^y costs one fma, one ex2 and the sums.  A tile
// (128 vocabulary entries of one row, in one thread) leaves (m, Σe, Σd·e) with m = max y,
// d = y - m, e = 2^d; d comes from one fma, so m's own rounding cancels.  Both sums stay well
// conditioned: the entropy of the tile is log Σe - ln 2·Σd·e/Σe, a sum of non-negative terms, and
// tiles are joined by Σe ← 2^{m-M}·Σe, Σd·e ← 2^{m-M}·(Σd·e + (m - M)·Σe).  Given tokens and
// alternatives are kept as accumulators.
//
// The alternatives.  Every 32 columns (a chunk) leave their maximum, and (pair kernel) their 32
// logits only if that reaches a lower bound of the row's k-th largest logit;
// head_finalize_top_kernel then looks at the k best chunks.  The bound: cut what was seen so far
// into kp >= k disjoint groups; the least of the groups' maxima is at most the k-th largest.  It
// never falls, so a chunk that reaches a later bound has been written.  In random order about
// k·log k chunks of the whole vocabulary reach it.
#pragma once

#include "gemm_common.cuh"

namespace lora {

constexpr int kHeadMaxIds = 128;   // given tokens (or teacher entries) a row
constexpr int kHeadMaxTop = 32;    // alternatives a row
constexpr int kHeadTile = 128;     // columns of a partial of the pair kernel
constexpr float kLog2e = 1.44269504f, kLn2 = 0.69314718f;

// ---------------------------------------------------------------- keys of the alternatives
// Larger key = larger logit, and among equal logits the smaller id.  -0 counts as +0; the
// key 0 stands for "no entry" (the smallest key of a number, that of -inf, is above it).
__device__ __forceinline__ uint32_t ord_f32(float f) {
  const uint32_t b = __float_as_uint(f + 0.0f);
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float unord_f32(uint32_t o) {
  return __uint_as_float((o & 0x80000000u) ? (o & 0x7fffffffu) : ~o);
}
__device__ __forceinline__ unsigned long long top_key(float z, int id) {
  return (static_cast<unsigned long long>(ord_f32(z)) << 32) | (0xffffffffu - static_cast<uint32_t>(id));
}

// A maximum of accumulators in units of log 2, rounded.  The sums beside it are relative to this
// value, so a join has to take it too: an fma of the product with the difference that follows (the
// compiler's choice for a plain `*`) shifts a tile by the rounding, half an ulp of m (logits around 100:
// 5e-6 in the log-probability of a certain token).
__device__ __forceinline__ float head_max_y(float raw, float c2) { return __fmul_rn(raw, c2); }

struct RowStats {
  float m, s, t;  // max y, Σ 2^{y-m}, Σ (y-m)·2^{y-m}
};
// a and b joined (either may be the empty {-inf, 0, 0}).
__device__ __forceinline__ RowStats join_stats(const RowStats& a, const RowStats& b) {
  RowStats o;
  o.m = fmaxf(a.m, b.m);
  const float da = a.m == -INFINITY ? 0.0f : a.m - o.m, db = b.m == -INFINITY ? 0.0f : b.m - o.m;
  const float ea = ex2_approx(da), eb = ex2_approx(db);
  o.s = a.s * ea + b.s * eb;
  o.t = (a.t + da * a.s) * ea + (b.t + db * b.s) * eb;
  return o;
}

// ---------------------------------------------------------------- one accumulator tile
// The least of a row's kp group maxima (ord_f32; 0: a group without any yet).
__device__ __forceinline__ uint32_t head_bound(const unsigned* bound, int kp) {
  uint32_t low = 0xffffffffu;
  if (kp >= 4) {
    for (int j = 0; j < kp; j += 4) {
      const uint4 b = __ldcg(reinterpret_cast<const uint4*>(bound + j));
      low = min(min(low, min(b.x, b.y)), min(b.z, b.w));
    }
  } else {
    for (int j = 0; j < kp; ++j) low = min(low, __ldcg(bound + j));
  }
  return low;
}
// The first n <= 32 accumulators of a chunk (n a multiple of 8) to z.
__device__ __forceinline__ void head_store_chunk(const uint32_t (&v)[32], int n, float* z) {
#pragma unroll
  for (int q = 0; q < 8; ++q)
    if (q * 4 < n)
      *reinterpret_cast<uint4*>(z + q * 4) = make_uint4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
}

// First pass over a row's nv <= 32·NC accumulator columns at tbase: the chunks' maxima
// (-inf past nv).  Returns the tile's.
template <int NC>
__device__ __forceinline__ float head_tile_max(uint32_t tbase, int nv, float (&cm)[NC]) {
  float m = -INFINITY;
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    cm[c] = -INFINITY;
    if (c * 32 < nv) {  // warp-uniform
      uint32_t v[32];
      tmem_ld_32x32b_x32(tbase + c * 32, v);
      tmem_ld_wait();
      const int n = nv - c * 32;
      if (n < 32) {  // the vocabulary's last chunk
#pragma unroll
        for (int j = 0; j < 32; ++j)
          if (j >= n) v[j] = 0xff800000u;
      }
      float a = __uint_as_float(v[0]), b = __uint_as_float(v[1]);
#pragma unroll
      for (int j = 2; j < 32; j += 2) {
        a = fmaxf(a, __uint_as_float(v[j]));
        b = fmaxf(b, __uint_as_float(v[j + 1]));
      }
      cm[c] = fmaxf(fmaxf(a, b), -INFINITY);  // a chunk of NaNs counts as empty
      m = fmaxf(m, cm[c]);
    }
  }
  return m;
}

// A row's first given token at or above a tile: its index among the sorted ones, its entry
// (0x7fffffff where there is none) and the next one's, so that the load behind a token found is
// not waited for.
struct HeadFirst {
  int pos;
  int2 e, next;
};
__device__ __forceinline__ int2 head_entry(const int2* sorted, int n, int pos) {
  return pos < n ? sorted[pos] : make_int2(0x7fffffff, 0);
}
__device__ __forceinline__ HeadFirst head_load_first(const HeadArgs& h, int row, int pos) {
  HeadFirst f{pos, make_int2(0x7fffffff, 0), make_int2(0x7fffffff, 0)};
  if (row >= 0) {
    const int2* sorted = h.sorted + static_cast<size_t>(row) * h.n;
    f.e = head_entry(sorted, h.n, pos);
    f.next = head_entry(sorted, h.n, pos + 1);
  }
  return f;
}
__device__ __forceinline__ void head_advance(const int2* sorted, int n, HeadFirst& f) {
  f.e = f.next;
  f.next = head_entry(sorted, n, ++f.pos + 1);
}

// The logits of the row's given tokens that fall into columns [v0, v0 + nv).  A register cannot be
// indexed, so the warp reads each wanted column again from TMEM.
__device__ __forceinline__ void head_tile_ids(const HeadArgs& h, uint32_t tbase, int nv, int v0, int row, HeadFirst f) {
  const int2* sorted = h.sorted + static_cast<size_t>(row) * h.n;
  while (true) {
    const uint32_t want = __ballot_sync(0xffffffffu, f.e.x < v0 + nv);
    if (!want) return;
    const int col = __shfl_sync(0xffffffffu, f.e.x, __ffs(want) - 1) - v0;
    const float z = __uint_as_float(tmem_ld_32x32b_x1(tbase + col));
    while (f.e.x - v0 == col) {
      h.id_logit[static_cast<size_t>(row) * h.n + f.e.y] = z;
      head_advance(sorted, h.n, f);
    }
    __syncwarp();
  }
}

// Calls f(registers, c) for the chunks of nv <= 128 columns at tbase, the next chunk's load in
// flight meanwhile, and release() once the last one has landed.
template <typename F, typename Release>
__device__ __forceinline__ void head_tile_chunks(uint32_t tbase, int nv, uint32_t (&va)[32], uint32_t (&vb)[32], F f,
                                                 Release release) {
  tmem_ld_32x32b_x32(tbase, va);
  tmem_ld_wait();
#pragma unroll
  for (int c = 0; c < kHeadTile / 32; ++c) {
    const bool more = c + 1 < kHeadTile / 32 && (c + 1) * 32 < nv;  // warp-uniform
    if (more) {
      if (c & 1) tmem_ld_32x32b_x32(tbase + (c + 1) * 32, va);
      else tmem_ld_32x32b_x32(tbase + (c + 1) * 32, vb);
    } else {
      release();
    }
    if (c & 1) f(vb, c);
    else f(va, c);
    if (!more) return;
    tmem_ld_wait();
  }
}

// Output of the pair kernel's head epilogues.  A warp's 32 rows × 32 columns (lane: row) go through
// one of its two staging buffers and a TMA store, in the 64-byte swizzle of the output's map: rows
// and columns outside are not written, and L2 sees whole sectors.  (16-byte stores, a row a lane,
// write every 32-byte sector twice: 52 us more on 1500 rows x 65536 x 1024.)  c: the chunk of the
// tile; a tile starts on the first buffer.
constexpr int kHeadStageBytes = 2048;
__device__ __forceinline__ void head_store_bf16(const CUtensorMap& tm, uint32_t stage, int lane, int c,
                                                const uint32_t (&o)[16], int x, int y) {
  const uint32_t buf = stage + (c & 1) * kHeadStageBytes;
  if (lane == 0) {  // the stores that last read this buffer
    if (c == 0) bulk_wait_read<0>();
    else bulk_wait_read<1>();
  }
  __syncwarp();
#pragma unroll
  for (int q = 0; q < 4; ++q)
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(buf + lane * 64 + ((q ^ ((lane >> 1) & 3)) << 4)),
                 "r"(o[4 * q]), "r"(o[4 * q + 1]), "r"(o[4 * q + 2]), "r"(o[4 * q + 3])
                 : "memory");
  fence_proxy_async_smem();  // the generic writes before the TMA store reads them
  __syncwarp();
  if (lane == 0) {
    tma_store_2d(&tm, buf, x, y);
    bulk_commit();
  }
}

// The pair kernel's forward epilogue of one row's columns [nt·128, +128) (all lanes of the warp
// take part), in two passes over TMEM.  32 columns' exponentials are independent instructions
// without a branch, and the next 32 columns load meanwhile: with two warps a scheduler nothing else
// hides their latency.  (All 128 columns in registers saved the second read and cost more in
// spills; a test per pair of columns took three times as long.)  The accumulator is released
// with the last load.
//
// The bound's groups are the chunks modulo kp, over every tile of the row so far, in h.bound:
// which tiles got there first changes how many chunks are written, never the k best of them.
//
// expz != null keeps p's numerator for the backward in bf16: e^z itself, so that one factor
// per row turns the row into probabilities and the dX GEMM can take it as it is.  A tile whose
// maximum is below 2^-43 or above 2^86 keeps 2^{y - tau} with tau its maximum instead (tau 0
// elsewhere).
template <typename Release>
__device__ __forceinline__ void head_fwd_tile(const HeadArgs& h, uint32_t tbase, int nv, int nt, int np, bool in,
                                              int M, int row, const HeadFirst& first, int V, const CUtensorMap& tm,
                                              uint32_t stage, Release release) {
  constexpr int NC = kHeadTile / 32;
  const size_t at = static_cast<size_t>(row) * np + nt;
  const size_t col0 = static_cast<size_t>(row) * V + nt * kHeadTile;
  uint32_t low = 0xffffffffu;
  if (h.k > 0 && in) low = head_bound(h.bound + static_cast<size_t>(row) * h.kp, h.kp);
  float cm[NC];
  float m = head_tile_max<NC>(tbase, nv, cm);
  uint32_t hits = 0;
  if (h.k > 0 && in) {
    unsigned* bound = h.bound + static_cast<size_t>(row) * h.kp;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const uint32_t o = ord_f32(cm[c]);
      if (o >= low) {  // cannot raise the least group otherwise
        atomicMax(bound + ((nt * NC + c) & (h.kp - 1)), o);
        if (c * 32 < nv) hits |= 1u << c;
      }
    }
    *reinterpret_cast<float4*>(h.cmax + at * NC) = make_float4(cm[0], cm[1], cm[2], cm[3]);
  }
  if (h.n > 0) head_tile_ids(h, tbase, nv, nt * kHeadTile, row, first);
  __syncwarp();
  const float raw = m;
  m = head_max_y(m, h.c2);
  const bool keep = h.expz != nullptr;
  const float tau = m < -43.0f || m > 86.0f ? m : 0.0f;
  const float f = ex2_approx(m - tau);
  const uint64_t c2 = pack_f32x2(h.c2, h.c2), mm = pack_f32x2(-m, -m), ff = pack_f32x2(f, f);
  uint64_t s[4] = {0, 0, 0, 0}, t[4] = {0, 0, 0, 0};
  const int lane = threadIdx.x & 31;
  const bool some = row - lane < M;  // warp-uniform: the warp has rows
  uint32_t va[32], vb[32];
  auto chunk = [&](const uint32_t (&v)[32], int c) {
    if ((hits >> c) & 1u) head_store_chunk(v, nv - c * 32, h.zlog + col0 + c * 32);
    uint32_t o[16];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      if (c * 32 + q * 8 < nv) {  // warp-uniform: nv is a multiple of 8
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint64_t d = fma_f32x2(pack_f32x2(__uint_as_float(v[8 * q + 2 * j]), __uint_as_float(v[8 * q + 2 * j + 1])),
                                       c2, mm);
          float d0, d1;
          unpack_f32x2(d, d0, d1);
          uint64_t e = pack_f32x2(ex2_approx(d0), ex2_approx(d1));
          s[j] = add_f32x2(s[j], e);
          t[j] = fma_f32x2(d, e, t[j]);
          e = mul_f32x2(e, ff);
          unpack_f32x2(e, d0, d1);
          o[4 * q + j] = pack_bf16x2(d0, d1);
        }
      }
    }
    __syncwarp();
    if (keep && some) head_store_bf16(tm, stage, lane, c, o, nt * kHeadTile + c * 32, row - lane);
  };
  head_tile_chunks(tbase, nv, va, vb, chunk, release);
  if (!in) return;
  float a0, a1, b0, b1;
  unpack_f32x2(add_f32x2(add_f32x2(s[0], s[1]), add_f32x2(s[2], s[3])), a0, a1);
  unpack_f32x2(add_f32x2(add_f32x2(t[0], t[1]), add_f32x2(t[2], t[3])), b0, b1);
  h.part[at] = make_float4(raw, a0 + a1, b0 + b1, 0.0f);
  if (keep) h.tau[at] = tau;
}

// dz of one accumulator tile of nv <= 128 columns in bf16 (recomputed logits).  rowp: (lse / ln 2,
// Σc + g_H·H, g_H·ln 2, 0 for a row without a gradient); x0: the tile's first column of the output.
template <typename Release>
__device__ __forceinline__ void head_dlogits_tile(const HeadArgs& h, uint32_t tbase, int nv, int v0, int x0, bool in,
                                                  int M, int row, HeadFirst f, const CUtensorMap& tm, uint32_t stage,
                                                  Release release) {
  const int lane = threadIdx.x & 31;
  const bool some = row - lane < M;  // warp-uniform: the warp has rows
  const int2* sorted = h.sorted + static_cast<size_t>(row) * h.n;
  const float4 rp = in ? h.rowp[row] : make_float4(0.f, 0.f, 0.f, 0.f);
  uint32_t va[32], vb[32];
  auto chunk = [&](const uint32_t (&v)[32], int c) {
    float d[32];
    if (rp.w == 0.0f) {
#pragma unroll
      for (int j = 0; j < 32; ++j) d[j] = 0.0f;
    } else if (rp.z == 0.0f) {
      const float w = -h.scale * rp.y;
#pragma unroll
      for (int j = 0; j < 32; ++j) d[j] = w * ex2_approx(fmaf(__uint_as_float(v[j]), h.c2, -rp.x));
    } else {
#pragma unroll
      for (int j = 0; j < 32; ++j) {
        const float lp = fmaf(__uint_as_float(v[j]), h.c2, -rp.x);
        d[j] = -h.scale * ex2_approx(lp) * fmaf(rp.z, lp, rp.y);
      }
    }
    while (f.e.x < v0 + min(nv, c * 32 + 32)) {
      const int at = f.e.x - v0 - c * 32;
#pragma unroll
      for (int j = 0; j < 32; ++j)
        if (j == at) d[j] = fmaf(h.scale, __int_as_float(f.e.y), d[j]);
      head_advance(sorted, h.n, f);
    }
    uint32_t o[16];
#pragma unroll
    for (int j = 0; j < 16; ++j) o[j] = pack_bf16x2(d[2 * j], d[2 * j + 1]);
    __syncwarp();
    if (some) head_store_bf16(tm, stage, lane, c, o, x0 + c * 32, row - lane);
  };
  head_tile_chunks(tbase, nv, va, vb, chunk, release);
}

// ---------------------------------------------------------------- row kernels
__device__ __forceinline__ float warp_max(float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
  return x;
}
__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// The softmax of one row's listed teacher logits, over its entries that are not ignored:
// lane i holds entries i, i + 32, ...; t[] becomes log q, and q = e^{t}.  Returns false for a
// row without any mass (no entry, or only -inf): it has no loss and no gradient.  A NaN among
// the entries makes every log q NaN.
constexpr int kHeadPerLane = kHeadMaxIds / 32;
__device__ __forceinline__ bool teacher_log_softmax(const int32_t* ids, const float* teacher, int n, int ignore,
                                                    float scale, int lane, float (&t)[kHeadPerLane]) {
  float tm = -INFINITY;
  bool nan = false;
#pragma unroll
  for (int u = 0; u < kHeadPerLane; ++u) {
    const int i = lane + 32 * u;
    t[u] = i < n && ids[i] != ignore ? teacher[i] * scale : -INFINITY;
    tm = fmaxf(tm, t[u]);
    nan |= t[u] != t[u];
  }
  tm = warp_max(tm);
  nan = __any_sync(0xffffffffu, nan);
  if (tm == -INFINITY && !nan) return false;
  float sum = 0.0f;
#pragma unroll
  for (int u = 0; u < kHeadPerLane; ++u)
    if (t[u] != -INFINITY) sum += expf(t[u] - tm);
  const float ls = nan ? NAN : logf(warp_sum(sum));
#pragma unroll
  for (int u = 0; u < kHeadPerLane; ++u) t[u] = (t[u] - tm) - ls;
  return true;
}

struct HeadRowArgs {
  int M, V, n, ignore;
  float scale, c2;         // scale, scale / ln 2
  const int32_t* ids;      // [M][n]
  const float* teacher;    // distillation: [M][n]
  // forward
  const float4* part;      // [M][np]
  int np;
  const float* id_logit;   // [M][n]
  int k, kp;
  int cpp;                 // chunks a partial
  int ctas;                // chunks are head_rows_kernel's, cpp a CTA; 0: cpp a partial of 128 columns
  const float* cmax;       // [M][chunks] maxima (-inf past a CTA's or the vocabulary's last)
  const float* zlog;       // [M][V] logits of the chunks that were kept
  float* logprob;          // [M][n] or null
  float* entropy;          // [M] or null
  float* lse_out;          // [M]
  float* loss;             // distillation: [M]
  int32_t* top_ids;        // [M][k]
  float* top_logprob;      // [M][k]
  // rows compacted by head_compact_kernel; else null.  The caller's arrays go by its rows, the
  // scratch by compacted ones.
  int* m_dev;              // their number
  int32_t* rowmap;         // [M] the caller's row of each
  int32_t* slot_of;        // [M] of the caller's rows, -1: left out
  const __nv_bfloat16* X;  // [M][D]
  __nv_bfloat16* Xc;       // [M][D] compacted
  __nv_bfloat16* dX;       // backward: [M][D]
  int D;
  // preparation
  int2* sorted;            // [M][n]
  uint8_t* first;          // [M][tiles]: tokens before each 128-column tile
  float* rowf;             // backward from a saved forward: [M] see head_saved_rows_kernel
  unsigned* bound;         // [M][kp] or null
  unsigned* live;          // head_rows_kernel's, or null: cleared for the next call
  float4* rowp;            // backward: [M]
  const float* lse;        // [M]
  const float* ent;        // [M] or null
  const float* dlogprob;   // [M][n] or null
  const float* dentropy;   // [M] or null
  const float* dloss;      // distillation: [M]
};

constexpr int kHeadRowWarps = 4;

// Distillation skips rows without an entry (prompts, padding): the others' hidden states are moved
// together, their number counted on the device, and the GEMMs stop there.  A row's results do not
// depend on its place, so the order in which blocks get theirs does not show.  Rows left out have
// loss 0 (and lse 0).  One warp a row.
constexpr int kCompactWarps = 8;
__global__ void __launch_bounds__(32 * kCompactWarps) head_compact_kernel(const HeadRowArgs a) {
  griddep_enter();  // the previous kernel in the stream completed (see ptx.cuh)
  __shared__ int base;
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row = blockIdx.x * kCompactWarps + w;
  bool any = false;
  if (row < a.M)
    for (int i = lane; i < a.n; i += 32) any |= a.ids[static_cast<size_t>(row) * a.n + i] != a.ignore;
  any = __any_sync(0xffffffffu, any);
  __shared__ int taken[kCompactWarps];
  if (lane == 0) taken[w] = any;
  __syncthreads();
  int before = 0, all = 0;
  for (int i = 0; i < kCompactWarps; ++i) {
    before += i < w ? taken[i] : 0;
    all += taken[i];
  }
  if (threadIdx.x == 0) base = all > 0 ? atomicAdd(a.m_dev, all) : 0;
  __syncthreads();
  if (row >= a.M) return;
  const int slot = any ? base + before : -1;
  if (lane == 0) {
    a.slot_of[row] = slot;
    if (any) a.rowmap[slot] = row;
    else a.loss[row] = a.lse_out[row] = 0.0f;
  }
  if (!any) return;
  const uint4* src = reinterpret_cast<const uint4*>(a.X + static_cast<size_t>(row) * a.D);
  uint4* dst = reinterpret_cast<uint4*>(a.Xc + static_cast<size_t>(slot) * a.D);
#pragma unroll 4
  for (int i = lane; i < a.D / 8; i += 32) dst[i] = src[i];
}

// What the backward needs of a row besides its tokens.
struct HeadRowGrad {
  float4 rp;  // (lse / ln 2, Σc + g_H·H, g_H·ln 2, 0 for a row without a gradient)
  float f;    // factor of a row from a saved forward, see head_saved_rows_kernel
};

// One warp sorts a row's tokens by id, by counting the entries before each (n <= 128 values in
// shared memory): at(sorted index, id, position, coefficient) for every one; ignored and
// out-of-range entries go last as 0x7fffffff and match no column.  The coefficients (backward) are
// the upstream gradients c_i: dlogprob, or -dloss·q_i.
//
// The factor f: with g_H = 0 the row's dz is -scale·C·e^{-lse} (C = Σc) times the saved e^z, but for
// its given tokens: that factor, if lse is within what e^z can hold in bf16 ([-20, 60]: the maximum
// is at most log V below it, and tiles beyond have their tau), C is not small against Σ|c| and the
// factor does not underflow; 1 for rows whose dz has to be written out; 0 for rows without a
// gradient.
template <bool BWD, typename At>
__device__ __forceinline__ HeadRowGrad head_row_tokens(const HeadRowArgs& a, int row, int lane, int* sid, At at) {
  const int32_t* ids = a.ids + static_cast<size_t>(row) * a.n;
  HeadRowGrad g{make_float4(0.f, 0.f, 0.f, 0.f), 0.0f};
  float coef[kHeadPerLane];
  if (BWD) {
    if (a.teacher != nullptr) {
      const bool any = teacher_log_softmax(ids, a.teacher + static_cast<size_t>(row) * a.n, a.n, a.ignore, a.scale,
                                           lane, coef);
      const float dl = any ? -a.dloss[row] : 0.0f;
#pragma unroll
      for (int u = 0; u < kHeadPerLane; ++u) coef[u] = any ? dl * expf(coef[u]) : 0.0f;
    } else {
#pragma unroll
      for (int u = 0; u < kHeadPerLane; ++u) {
        const int i = lane + 32 * u;
        coef[u] = a.dlogprob != nullptr && i < a.n && ids[i] != a.ignore ? a.dlogprob[static_cast<size_t>(row) * a.n + i]
                                                                       : 0.0f;
      }
    }
    float csum = 0.0f, cabs = 0.0f;
#pragma unroll
    for (int u = 0; u < kHeadPerLane; ++u) {
      csum += coef[u];
      cabs += fabsf(coef[u]);
    }
    csum = warp_sum(csum);
    cabs = warp_sum(cabs);
    const float gh = a.dentropy != nullptr ? a.dentropy[row] : 0.0f;
    const bool none = gh == 0.0f && cabs == 0.0f;  // no gradient, whatever the logits
    const float lse = none ? 0.0f : a.lse[row];
    g.rp = make_float4(lse * kLog2e, gh != 0.0f ? fmaf(gh, a.ent[row], csum) : csum, gh * kLn2, none ? 0.0f : 1.0f);
    g.f = -a.scale * csum * expf(-lse);
    if (!(gh == 0.0f && lse >= -20.0f && lse <= 60.0f && fabsf(csum) >= cabs * 0x1p-6f && fabsf(g.f) > 1e-30f)) g.f = 1.0f;
    if (none) g.f = 0.0f;
  }
  for (int i = lane; i < a.n; i += 32) {
    const int id = ids[i];
    sid[i] = id == a.ignore || id < 0 || id >= a.V ? 0x7fffffff : id;
  }
  __syncwarp();
#pragma unroll
  for (int u = 0; u < kHeadPerLane; ++u) {
    const int i = lane + 32 * u;
    if (i < a.n) {
      const int id = sid[i];
      int before = 0;
      for (int j = 0; j < a.n; ++j) before += sid[j] < id || (sid[j] == id && j < i);
      at(before, id, i, BWD ? coef[u] : 0.0f);
    }
  }
  __syncwarp();
  return g;
}

// One warp a row: the row's tokens in order, with their position (forward) or coefficient
// (backward), and how many precede each tile, for the GEMM epilogues; the forward's bounds
// cleared, the backward's row coefficients.
template <bool BWD>
__global__ void __launch_bounds__(32 * kHeadRowWarps) head_prep_kernel(const HeadRowArgs a) {
  griddep_enter();  // the previous kernel in the stream completed (see ptx.cuh)
  __shared__ int sid[kHeadRowWarps][kHeadMaxIds], ordered[kHeadRowWarps][kHeadMaxIds];
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int slot = blockIdx.x * kHeadRowWarps + w;
  if (slot >= (a.m_dev != nullptr ? *a.m_dev : a.M)) return;  // whole warps
  const int row = a.m_dev != nullptr ? a.rowmap[slot] : slot;
  int2* sorted = a.sorted + static_cast<size_t>(slot) * a.n;
  const HeadRowGrad g = head_row_tokens<BWD>(a, row, lane, sid[w], [&](int k, int id, int i, float c) {
    ordered[w][k] = id;
    sorted[k] = make_int2(id, BWD ? __float_as_int(c) : i);
  });
  if (BWD && lane == 0) a.rowp[slot] = g.rp;
  if (a.first != nullptr) {
    const int tiles = (a.V + kHeadTile - 1) / kHeadTile;
    uint8_t* first = a.first + static_cast<size_t>(slot) * tiles;
    for (int t = lane; t < tiles; t += 32) {
      int lo = 0, hi = a.n;
      while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (ordered[w][mid] < t * kHeadTile) lo = mid + 1;
        else hi = mid;
      }
      first[t] = static_cast<uint8_t>(lo);
    }
  }
  if (!BWD && a.bound != nullptr && lane < a.kp) a.bound[static_cast<size_t>(slot) * a.kp + lane] = 0u;
}

// First vocabulary entry of CTA i of head_rows_kernel: ranges of multiples of 16.
__host__ __device__ __forceinline__ int hr_first(int V, int i, int ctas) {
  return static_cast<int>(static_cast<long long>((V + 15) / 16) * i / ctas) * 16;
}

// One warp a row: joins the row's partials (in a fixed order), and from them the
// log-probabilities, the entropy and the distillation loss.
__global__ void __launch_bounds__(32 * kHeadRowWarps) head_finalize_kernel(const HeadRowArgs a) {
  griddep_enter();  // the previous kernel in the stream completed (see ptx.cuh)
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int slot = blockIdx.x * kHeadRowWarps + w;
  if (slot >= (a.m_dev != nullptr ? *a.m_dev : a.M)) return;  // whole warps
  const int row = a.m_dev != nullptr ? a.rowmap[slot] : slot;
  const float4* part = a.part + static_cast<size_t>(slot) * a.np;
  float m = -INFINITY;
  for (int i = lane; i < a.np; i += 32) m = fmaxf(m, part[i].x);
  m = head_max_y(warp_max(m), a.c2);
  float s = 0.0f, t = 0.0f;
  for (int i = lane; i < a.np; i += 32) {
    const float4 q = part[i];
    if (q.y == 0.0f) continue;  // no entries
    const float d = head_max_y(q.x, a.c2) - m, e = exp2f(d);
    s = fmaf(q.y, e, s);
    t = fmaf(fmaf(d, q.y, q.z), e, t);
  }
  s = warp_sum(s);
  t = warp_sum(t);
  const float ls = logf(s);
  if (lane == 0) {
    a.lse_out[row] = fmaf(m, kLn2, ls);
    if (a.entropy != nullptr) a.entropy[row] = ls - kLn2 * (t / s);
  }
  // the given tokens: z - lse as (z - max) - log Σe, which keeps the small ones' digits
  const int32_t* ids = a.ids + static_cast<size_t>(row) * a.n;
  float lp[kHeadPerLane];
#pragma unroll
  for (int u = 0; u < kHeadPerLane; ++u) {
    const int i = lane + 32 * u;
    lp[u] = 0.0f;
    if (i < a.n) {
      const int id = ids[i];
      if (id != a.ignore)
        lp[u] = id >= 0 && id < a.V ? fmaf(a.id_logit[static_cast<size_t>(slot) * a.n + i], a.c2, -m) * kLn2 - ls : NAN;
      if (a.logprob != nullptr) a.logprob[static_cast<size_t>(row) * a.n + i] = lp[u];
    }
  }
  if (a.loss != nullptr) {
    float t2[kHeadPerLane];
    const bool any =
        teacher_log_softmax(ids, a.teacher + static_cast<size_t>(row) * a.n, a.n, a.ignore, a.scale, lane, t2);
    float l = 0.0f;
    if (any) {
#pragma unroll
      for (int u = 0; u < kHeadPerLane; ++u) {
        const float q = expf(t2[u]);
        if (q != 0.0f) l = fmaf(q, t2[u] - lp[u], l);  // also where q is NaN
      }
    }
    l = warp_sum(l);
    if (lane == 0) a.loss[row] = l;
  }
}

// One block a row, with alternatives: as head_finalize_kernel (no loss), then the k best.  First the
// k best chunks by their maxima (an element of another chunk has k better ones), from those that
// reach the row's bound; then the k best elements of these.  Bound by latency: 4600 maxima are in
// flight at once, about k·log k of them reach the bound, at most 1024 elements are looked at.
constexpr int kTopThreads = 512, kTopWarps = kTopThreads / 32, kTopBuf = 1024, kTopPer = 9;
__global__ void __launch_bounds__(kTopThreads) head_finalize_top_kernel(const HeadRowArgs a) {
  griddep_enter();  // the previous kernel in the stream completed (see ptx.cuh)
  __shared__ unsigned long long buf[kTopBuf], top[kHeadMaxTop];
  __shared__ float red[kTopWarps][2], groups[kTopWarps][32];
  __shared__ int buf_n, above;
  const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31;
  const int row = blockIdx.x;
  const float4* part = a.part + static_cast<size_t>(row) * a.np;
  const int chunks = (a.ctas > 0 ? a.ctas : a.np) * a.cpp;
  const float* cmax = a.cmax + static_cast<size_t>(row) * chunks;
  constexpr int HELD = 2;  // partials a thread keeps in registers
  float4 held[HELD];
#pragma unroll
  for (int u = 0; u < HELD; ++u) {
    const int i = tid + u * kTopThreads;
    held[u] = i < a.np ? part[i] : make_float4(-INFINITY, 0.f, 0.f, 0.f);
  }
  float cm[kTopPer];
  auto load_maxima = [&](int q0) {
#pragma unroll
    for (int u = 0; u < kTopPer; ++u) {
      const int q = q0 + u * kTopThreads + tid;
      cm[u] = q < chunks ? cmax[q] : -INFINITY;
    }
  };
  load_maxima(0);
  float m = -INFINITY;
#pragma unroll
  for (int u = 0; u < HELD; ++u) m = fmaxf(m, held[u].x);
  for (int i = tid + HELD * kTopThreads; i < a.np; i += kTopThreads) m = fmaxf(m, part[i].x);
  // few rows: the partials' maxima in groups (i mod kp: the lane mod kp); the least group's is a
  // bound
  float g = m;
  for (int o = a.kp; o < 32; o <<= 1) g = fmaxf(g, __shfl_xor_sync(0xffffffffu, g, o));
  groups[w][lane] = g;
  m = warp_max(m);
  if (lane == 0) red[w][0] = m;
  if (tid == 0) buf_n = 0;
  __syncthreads();
#pragma unroll
  for (int u = 0; u < kTopWarps; ++u) {
    m = fmaxf(m, red[u][0]);
    g = fmaxf(g, groups[u][lane]);
  }
  m = head_max_y(m, a.c2);
  float low;
  if (a.ctas > 0) {
    for (int o = 1; o < a.kp; o <<= 1) g = fminf(g, __shfl_xor_sync(0xffffffffu, g, o));
    low = g;
  } else {
    const uint32_t o = lane < a.kp ? a.bound[static_cast<size_t>(row) * a.kp + lane] : 0xffffffffu;
    low = unord_f32(max(__reduce_min_sync(0xffffffffu, o), ord_f32(-INFINITY)));  // 0: an empty group
  }
  float s = 0.0f, t = 0.0f;
  auto join = [&](const float4& q) {
    if (q.y == 0.0f) return;  // no entries
    const float d = head_max_y(q.x, a.c2) - m, e = exp2f(d);
    s = fmaf(q.y, e, s);
    t = fmaf(fmaf(d, q.y, q.z), e, t);
  };
#pragma unroll
  for (int u = 0; u < HELD; ++u)
    if (tid + u * kTopThreads < a.np) join(held[u]);
  for (int i = tid + HELD * kTopThreads; i < a.np; i += kTopThreads) join(part[i]);
  s = warp_sum(s);
  t = warp_sum(t);
  __syncthreads();
  if (lane == 0) {
    red[w][0] = s;
    red[w][1] = t;
  }

  // ---- the best chunks: keys (maximum, chunk) above kth
  unsigned long long kth = ord_f32(low) > 0 ? (static_cast<unsigned long long>(ord_f32(low)) << 32) - 1 : 0;
  auto push = [&](unsigned long long key) {  // whole warps; the order in buf varies, the set does not
    const uint32_t keep = __ballot_sync(0xffffffffu, key > kth);
    int base = 0;
    if (lane == 0 && keep) base = atomicAdd(&buf_n, __popc(keep));
    base = __shfl_sync(0xffffffffu, base, 0);
    if (key > kth) buf[base + __popc(keep & ((1u << lane) - 1u))] = key;
  };
  auto cut = [&]() {  // all threads: the k largest of buf_n keys to top (in order) and the head of buf
    __syncthreads();
    const int n = buf_n;
    if (tid < kHeadMaxTop) top[tid] = 0;
    __syncthreads();
    for (int i = tid; i < n; i += kTopThreads) {
      const unsigned long long key = buf[i];
      int rank = 0;
#pragma unroll 8
      for (int j = 0; j < n; ++j) rank += buf[j] > key;
      if (rank < a.k) top[rank] = key;
    }
    __syncthreads();
    if (top[a.k - 1] > kth) kth = top[a.k - 1];
    if (tid < a.k) buf[tid] = top[tid];
    if (tid == 0) buf_n = min(n, a.k);
    __syncthreads();
  };
  for (int q0 = 0; q0 < chunks; q0 += kTopPer * kTopThreads) {
    if (q0 > 0) load_maxima(q0);
    int mine = 0;
#pragma unroll
    for (int u = 0; u < kTopPer; ++u) {
      const int q = q0 + u * kTopThreads + tid;
      mine += q < chunks && top_key(cm[u], q) > kth;
    }
    // usually all that reach the bound fit; else (equal maxima) a buffer's half at a time
    mine = __reduce_add_sync(0xffffffffu, mine);
    if (tid == 0) above = buf_n;
    __syncthreads();
    if (lane == 0 && mine) atomicAdd(&above, mine);
    __syncthreads();
    const bool fits = above <= kTopBuf;
#pragma unroll 1
    for (int u = 0; u < kTopPer; ++u) {
      const int q = q0 + u * kTopThreads + tid;
      float c = cm[0];
#pragma unroll
      for (int i = 1; i < kTopPer; ++i) c = u == i ? cm[i] : c;
      if (!fits) {
        // room for what the next push adds, which starts from up to kTopBuf keys of an earlier pass; one
        // decision for the block, read between two barriers since the push adds to buf_n
        __syncthreads();
        const bool full = buf_n > kTopBuf - kTopThreads;
        __syncthreads();
        if (full) cut();
      }
      push(q < chunks ? top_key(c, q) : 0ull);
    }
    __syncthreads();
  }
  cut();

  // ---- their elements
  const unsigned long long mine = lane < a.k ? top[lane] : 0ull;
  unsigned long long key[kHeadMaxTop / kTopWarps];
#pragma unroll
  for (int u = 0; u < kHeadMaxTop / kTopWarps; ++u) {
    const int i = w + u * kTopWarps;
    const unsigned long long ck = __shfl_sync(0xffffffffu, mine, i);
    key[u] = 0;
    if (ck != 0) {
      const int q = static_cast<int>(0xffffffffu - static_cast<uint32_t>(ck));
      int col = q * 32, end = a.V;
      if (a.ctas > 0) {
        const int i0 = q / a.cpp;
        col = hr_first(a.V, i0, a.ctas) + (q - i0 * a.cpp) * 32;
        end = min(a.V, hr_first(a.V, i0 + 1, a.ctas));
      }
      if (col + lane < end) {
        const float z = a.zlog[static_cast<size_t>(row) * a.V + col + lane];
        if (z == z) key[u] = top_key(z, col + lane);
      }
    }
  }
  // the k-th chunk's maximum is the least an element can need
  const unsigned long long least = top[a.k - 1];
  kth = least != 0 ? (least >> 32 << 32) - 1 : 0;
  __syncthreads();
  s = t = 0.0f;
#pragma unroll
  for (int u = 0; u < kTopWarps; ++u) {
    s += red[u][0];
    t += red[u][1];
  }
  const float ls = logf(s);
  if (tid == 0) {
    buf_n = 0;
    a.lse_out[row] = fmaf(m, kLn2, ls);
    if (a.entropy != nullptr) a.entropy[row] = ls - kLn2 * (t / s);
  }
  if (tid < a.n) {
    const size_t at = static_cast<size_t>(row) * a.n + tid;
    const int id = a.ids[at];
    float lp = 0.0f;
    if (id != a.ignore) lp = id >= 0 && id < a.V ? fmaf(a.id_logit[at], a.c2, -m) * kLn2 - ls : NAN;
    a.logprob[at] = lp;
  }
  __syncthreads();
#pragma unroll
  for (int u = 0; u < kHeadMaxTop / kTopWarps; ++u) push(key[u]);
  cut();
  if (row == 0 && tid == 0 && a.live != nullptr) *a.live = 0;
  if (tid < a.k) {
    const unsigned long long best = top[tid];
    const size_t at = static_cast<size_t>(row) * a.k + tid;
    a.top_ids[at] = best != 0 ? static_cast<int32_t>(0xffffffffu - static_cast<uint32_t>(best)) : -1;
    a.top_logprob[at] = best != 0 ? fmaf(unord_f32(static_cast<uint32_t>(best >> 32)), a.c2, -m) * kLn2 - ls : NAN;
  }
}

// The backward from a saved forward prepares the operand of the dX GEMM in place; the GEMM
// multiplies row m of its result by rowf[m] (HeadRowGrad::f).
//   rowf = -scale·C·e^{-lse}: the saved e^z stand, but for tiles that kept 2^{y-tau} (rare: times
//     2^tau) and the given tokens, which become dz/rowf from their fp32 logits.
//   rowf = 1 (an entropy gradient, C small against Σ|c|, an lse that e^z cannot hold): the whole
//     row becomes dz = scale·(Σ c - p·(Σc + g_H·(log p + H))); bound by HBM, 4·V bytes a row.  Here
//     dz is rounded to bf16 a second time and takes log p from the rounded e^z (off by up to 2^-8):
//     the saved buffer has no more, and the GEMM's operand is bf16 in any case.
//   rowf = 0: nothing, the GEMM's row is 0.
// A block takes `per` <= 8 rows, a warp each for their tokens, and writes out its whole rows one
// after the other; more rows a block where there are blocks enough (per = 1 for 13653 rows x 408
// took 71 us, bound by the blocks' latency).  Blocks also clear dX of rows that were left out.
constexpr int kSavedThreads = 256, kSavedRows = kSavedThreads / 32;
__global__ void __launch_bounds__(kSavedThreads)
    head_saved_rows_kernel(const HeadRowArgs a, __nv_bfloat16* expz, const float* taus, int np, int per) {
  griddep_enter();  // the previous kernel in the stream completed (see ptx.cuh)
  __shared__ int sid[kSavedRows][kHeadMaxIds], s_id[kSavedRows][kHeadMaxIds];
  __shared__ float s_c[kSavedRows][kHeadMaxIds], s_z[kSavedRows][kHeadMaxIds];
  __shared__ HeadRowGrad s_g[kSavedRows];
  const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31;
  const int slot0 = blockIdx.x * per, V = a.V;
  const int rows = a.m_dev != nullptr ? *a.m_dev : a.M;
  if (w < per && slot0 + w < a.M) {
    const int slot = slot0 + w;
    if (a.m_dev != nullptr && a.slot_of[slot] < 0) {  // the caller's row of this number was left out
      uint4* d = reinterpret_cast<uint4*>(a.dX + static_cast<size_t>(slot) * a.D);
      for (int i = lane; i < a.D / 8; i += 32) d[i] = make_uint4(0u, 0u, 0u, 0u);
    }
    if (slot < rows) {
      const float* z = a.id_logit + static_cast<size_t>(slot) * a.n;
      const HeadRowGrad g = head_row_tokens<true>(a, a.m_dev != nullptr ? a.rowmap[slot] : slot, lane, sid[w],
                                                  [&](int k, int id, int i, float c) {
                                                    s_id[w][k] = id;
                                                    s_c[w][k] = c;
                                                    s_z[w][k] = z[i];
                                                  });
      if (lane == 0) {
        s_g[w] = g;
        a.rowf[slot] = g.f;
      }
    }
  }
  __syncthreads();
  for (int r = 0; r < per && slot0 + r < rows; ++r) {
    if (s_g[r].f != 1.0f) continue;  // the same for all threads
    const float4 rp = s_g[r].rp;
    __nv_bfloat16* zrow = expz + static_cast<size_t>(slot0 + r) * V;
    const float* tau = taus + static_cast<size_t>(slot0 + r) * np;
    constexpr int U = 4;
    for (int c0 = tid * 8; c0 < V; c0 += kSavedThreads * 8 * U) {
      uint4 x[U];
      float shift[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int col = c0 + u * kSavedThreads * 8;
        if (col < V) {
          x[u] = *reinterpret_cast<const uint4*>(zrow + col);
          shift[u] = tau[col / kHeadTile] - rp.x;
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int col = c0 + u * kSavedThreads * 8;
        if (col >= V) break;
        const uint32_t in[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
        const float es = ex2_approx(shift[u]);
        float d[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float ez = __uint_as_float((j & 1) ? (in[j >> 1] & 0xffff0000u) : (in[j >> 1] << 16));
          float wgt = rp.y;
          if (rp.z != 0.0f && ez > 0.0f) wgt = fmaf(rp.z, lg2_approx(ez) + shift[u], wgt);
          d[j] = -a.scale * ez * es * wgt;
        }
        *reinterpret_cast<uint4*>(zrow + col) = make_uint4(pack_bf16x2(d[0], d[1]), pack_bf16x2(d[2], d[3]),
                                                           pack_bf16x2(d[4], d[5]), pack_bf16x2(d[6], d[7]));
      }
    }
  }
  __syncthreads();
  if (w >= per || slot0 + w >= rows || s_g[w].f == 0.0f) return;  // whole warps
  const float f = s_g[w].f;
  const float4 rp = s_g[w].rp;
  __nv_bfloat16* zrow = expz + static_cast<size_t>(slot0 + w) * V;
  if (f != 1.0f) {
    const float* tau = taus + static_cast<size_t>(slot0 + w) * np;
    constexpr int U = 8;  // loads in flight
    for (int t0 = lane; t0 < np; t0 += 32 * U) {
      float tt[U];
#pragma unroll
      for (int u = 0; u < U; ++u) tt[u] = t0 + 32 * u < np ? tau[t0 + 32 * u] : 0.0f;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (tt[u] == 0.0f) continue;
        const int t = t0 + 32 * u;
        const float es = exp2f(tt[u]);  // at most 2^86.6, an lse of 60
        for (int col = t * kHeadTile; col < min(V, (t + 1) * kHeadTile); ++col)
          zrow[col] = __float2bfloat16_rn(__bfloat162float(zrow[col]) * es);
      }
    }
    __syncwarp();
  }
  for (int i = lane; i < a.n; i += 32) {
    const int id = s_id[w][i];
    if (id == 0x7fffffff || (i > 0 && s_id[w][i - 1] == id)) continue;
    float c = 0.0f;
    for (int j = i; j < a.n && s_id[w][j] == id; ++j) c += s_c[w][j];
    const float lp = fmaf(s_z[w][i], a.c2, -rp.x);
    const float dz = a.scale * (c - exp2f(lp) * (rp.z != 0.0f ? fmaf(rp.z, lp, rp.y) : rp.y));
    zrow[id] = __float2bfloat16_rn(f == 1.0f ? dz : dz / f);
  }
}

}  // namespace lora
