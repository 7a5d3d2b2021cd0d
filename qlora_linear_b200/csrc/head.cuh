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
// A tile (128 vocabulary entries of one row, in one thread) leaves (m, Σe, Σd·e) with
// m = max z, d = z - m, e = e^d.  Both sums stay well conditioned: the entropy of the tile is
// log Σe - Σd·e/Σe, a sum of non-negative terms, and tiles are joined by
// Σe ← e^{m-M}·Σe, Σd·e ← e^{m-M}·(Σd·e + (m - M)·Σe).
//
// The alternatives.  Every 32 columns (a chunk) leave their maximum, and their 32 logits only
// if that reaches a lower bound of the row's k-th largest logit; head_finalize_top_kernel then
// looks at the few chunks that reach the final bound.  The bound: cut what was seen so far into
// kp >= k disjoint groups; the least of the groups' maxima is at most the k-th largest.  It
// never falls, so a chunk that reaches a later bound has been written.  In random order about
// k·log k chunks of the whole vocabulary reach it.
#pragma once

#include "gemm_common.cuh"

namespace lora {

constexpr int kHeadMaxIds = 128;   // given tokens (or teacher entries) a row
constexpr int kHeadMaxTop = 32;    // alternatives a row
constexpr int kHeadTile = 128;     // columns of a partial of the pair kernel

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

struct RowStats {
  float m, s, t;  // max z, Σ e^{z-m}, Σ (z-m)·e^{z-m}
};
// a and b joined (either may be the empty {-inf, 0, 0}).
__device__ __forceinline__ RowStats join_stats(const RowStats& a, const RowStats& b) {
  RowStats o;
  o.m = fmaxf(a.m, b.m);
  const float da = a.m == -INFINITY ? 0.0f : a.m - o.m, db = b.m == -INFINITY ? 0.0f : b.m - o.m;
  const float ea = __expf(da), eb = __expf(db);
  o.s = a.s * ea + b.s * eb;
  o.t = (a.t + da * a.s) * ea + (b.t + db * b.s) * eb;
  return o;
}

// ---------------------------------------------------------------- one accumulator tile
// First pass over a row's nv <= 32·NC accumulator columns at tbase: the chunks' maxima
// (-inf past nv), scaled.  Returns the tile's.
template <int NC>
__device__ __forceinline__ float head_tile_max(uint32_t tbase, int nv, float scale, float (&cm)[NC]) {
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
      cm[c] = fmaxf(a, b) * scale;
      m = fmaxf(m, cm[c]);
    }
  }
  return m;
}

// Second pass: the sums and, of the chunks in `hits`, the logits (zrow != null); expz != null
// keeps e^{z-m} for the backward, in fp16: at most 1, so its 11 bits beat bf16's 8 down to
// 2^-15, and what lies below weighs less in dX than the rounding of the tile's largest entry.
// Full chunks run without a branch: one warp a scheduler hides the latency of exp by the
// instructions of its other columns alone (with a test per pair of columns the pass took three
// times as long).
__device__ __forceinline__ RowStats head_tile_sums(uint32_t tbase, int nv, float scale, bool in, float m, uint32_t hits,
                                                   float* zrow, __half* expz) {
  float s[2] = {0.0f, 0.0f}, t[2] = {0.0f, 0.0f};
#pragma unroll 1
  for (int c = 0; c * 32 < nv; ++c) {
    uint32_t v[32];
    tmem_ld_32x32b_x32(tbase + c * 32, v);
    tmem_ld_wait();
    const int n = nv - c * 32;
    if ((hits >> c) & 1u) {
#pragma unroll
      for (int q = 0; q < 8; ++q)
        if (q * 4 < n)
          *reinterpret_cast<float4*>(zrow + c * 32 + q * 4) =
              make_float4(__uint_as_float(v[4 * q]) * scale, __uint_as_float(v[4 * q + 1]) * scale,
                          __uint_as_float(v[4 * q + 2]) * scale, __uint_as_float(v[4 * q + 3]) * scale);
    }
    if (n >= 32) {
      float e[32];
#pragma unroll
      for (int j = 0; j < 32; ++j) {
        const float d = fmaf(__uint_as_float(v[j]), scale, -m);
        e[j] = __expf(d);
        s[j & 1] += e[j];
        t[j & 1] = fmaf(d, e[j], t[j & 1]);
      }
      if (expz != nullptr && in) {
#pragma unroll
        for (int q = 0; q < 4; ++q)
          *reinterpret_cast<uint4*>(expz + c * 32 + q * 8) =
              make_uint4(pack_f16x2(e[8 * q], e[8 * q + 1]), pack_f16x2(e[8 * q + 2], e[8 * q + 3]),
                         pack_f16x2(e[8 * q + 4], e[8 * q + 5]), pack_f16x2(e[8 * q + 6], e[8 * q + 7]));
      }
    } else {
#pragma unroll
      for (int q = 0; q < 4; ++q)
        if (q * 8 < n) {  // n is a multiple of 8
          float e[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float d = fmaf(__uint_as_float(v[8 * q + j]), scale, -m);
            e[j] = __expf(d);
            s[j & 1] += e[j];
            t[j & 1] = fmaf(d, e[j], t[j & 1]);
          }
          if (expz != nullptr && in)
            *reinterpret_cast<uint4*>(expz + c * 32 + q * 8) = make_uint4(
                pack_f16x2(e[0], e[1]), pack_f16x2(e[2], e[3]), pack_f16x2(e[4], e[5]), pack_f16x2(e[6], e[7]));
        }
    }
    __syncwarp();
  }
  return RowStats{m, s[0] + s[1], t[0] + t[1]};
}

// The logits of the row's given tokens that fall into columns [v0, v0 + nv).  sorted: the
// row's (id, position) by id, e: the first of them at or above v0 (pos: its index).  A register
// cannot be indexed, so the warp reads each wanted column again from TMEM.
__device__ __forceinline__ void head_tile_ids(const HeadArgs& h, uint32_t tbase, int nv, int v0, int row, int pos,
                                              int2 e) {
  const int2* sorted = h.sorted + static_cast<size_t>(row) * h.n;
  while (true) {
    const uint32_t want = __ballot_sync(0xffffffffu, e.x < v0 + nv);
    if (!want) return;
    const int col = __shfl_sync(0xffffffffu, e.x, __ffs(want) - 1) - v0;
    const float z = __uint_as_float(tmem_ld_32x32b_x1(tbase + col)) * h.scale;
    while (e.x - v0 == col) {
      h.id_logit[static_cast<size_t>(row) * h.n + e.y] = z;
      e = ++pos < h.n ? sorted[pos] : make_int2(0x7fffffff, 0);
    }
    __syncwarp();
  }
}

// First entry of the row's sorted tokens at or above v0.
__device__ __forceinline__ int head_first_id(const int2* sorted, int n, int v0) {
  int lo = 0, hi = n;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (sorted[mid].x < v0) lo = mid + 1;
    else hi = mid;
  }
  return lo;
}

// The pair kernel's forward epilogue of one row's columns [nt·128, +128) (all lanes of the warp
// take part).  The bound's groups are the chunks modulo kp, over every tile of the row so far,
// in h.bound: which tiles got there first changes how many chunks are written, never the k best
// of them.
__device__ __forceinline__ void head_fwd_tile(const HeadArgs& h, uint32_t tbase, int nv, int nt, int np, bool in,
                                              int row, int pos, int2 first, int V) {
  constexpr int NC = kHeadTile / 32;
  float cm[NC];
  const float m = head_tile_max<NC>(tbase, nv, h.scale, cm);
  const size_t at = static_cast<size_t>(row) * np + nt;
  uint32_t hits = 0;
  if (h.k > 0 && in) {
    unsigned* bound = h.bound + static_cast<size_t>(row) * h.kp;
    uint32_t low = 0xffffffffu;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const uint32_t o = ord_f32(cm[c]);
      unsigned* b = bound + ((nt * NC + c) & (h.kp - 1));
      if (o > __ldcg(b)) atomicMax(b, o);
    }
    if (h.kp >= 4) {
      for (int j = 0; j < h.kp; j += 4) {
        const uint4 b = __ldcg(reinterpret_cast<const uint4*>(bound + j));
        low = min(min(low, min(b.x, b.y)), min(b.z, b.w));
      }
    } else {
      for (int j = 0; j < h.kp; ++j) low = min(low, __ldcg(bound + j));
    }
#pragma unroll
    for (int c = 0; c < NC; ++c)
      if (ord_f32(cm[c]) >= low && c * 32 < nv) hits |= 1u << c;
    *reinterpret_cast<float4*>(h.cmax + at * NC) = make_float4(cm[0], cm[1], cm[2], cm[3]);
  }
  __syncwarp();
  const size_t col0 = static_cast<size_t>(row) * V + nt * kHeadTile;
  const RowStats st = head_tile_sums(tbase, nv, h.scale, in, m, hits, h.zlog + col0,
                                     h.expz != nullptr ? h.expz + col0 : nullptr);
  if (h.n > 0) head_tile_ids(h, tbase, nv, nt * kHeadTile, row, pos, first);
  if (!in) return;
  h.part[at] = make_float4(st.m, st.s, st.t, 0.0f);
  if (h.expz != nullptr) h.tile_max[at] = st.m;
}

// dz of one accumulator tile of nv <= 128 columns in bf16 (recomputed logits).
// rowp: (lse, Σc + g_H·H, g_H).
__device__ __forceinline__ void head_dlogits_tile(const HeadArgs& h, uint32_t tbase, int nv, int v0, bool in,
                                                  const float4& rp, const int2* sorted, int pos, int2 e,
                                                  __nv_bfloat16* orow) {
#pragma unroll 1
  for (int c = 0; c * 32 < nv; ++c) {
    uint32_t v[32];
    tmem_ld_32x32b_x32(tbase + c * 32, v);
    tmem_ld_wait();
    const int n = min(32, nv - c * 32);
    if (in) {
      float d[32];
      if (rp.z == 0.0f) {
        const float w = -h.scale * rp.y;
#pragma unroll
        for (int j = 0; j < 32; ++j) d[j] = w * __expf(fmaf(__uint_as_float(v[j]), h.scale, -rp.x));
      } else {
#pragma unroll
        for (int j = 0; j < 32; ++j) {
          const float lp = fmaf(__uint_as_float(v[j]), h.scale, -rp.x);
          d[j] = -h.scale * __expf(lp) * fmaf(rp.z, lp, rp.y);
        }
      }
      while (e.x < v0 + c * 32 + n) {
        const int at = e.x - v0 - c * 32;
#pragma unroll
        for (int j = 0; j < 32; ++j)
          if (j == at) d[j] = fmaf(h.scale, __int_as_float(e.y), d[j]);
        e = ++pos < h.n ? sorted[pos] : make_int2(0x7fffffff, 0);
      }
#pragma unroll
      for (int q = 0; q < 4; ++q)
        if (q * 8 < n)
          *reinterpret_cast<uint4*>(orow + c * 32 + q * 8) =
              make_uint4(pack_bf16x2(d[8 * q], d[8 * q + 1]), pack_bf16x2(d[8 * q + 2], d[8 * q + 3]),
                         pack_bf16x2(d[8 * q + 4], d[8 * q + 5]), pack_bf16x2(d[8 * q + 6], d[8 * q + 7]));
    }
    __syncwarp();
  }
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
  float scale;
  const int32_t* ids;      // [M][n]
  const float* teacher;    // distillation: [M][n]
  // forward
  const float4* part;      // [M][np]
  int np;
  const float* id_logit;   // [M][n]
  int k, kp;
  int cpp;                 // chunks a partial
  int few;                 // partials are head_rows_kernel's (col0 of hr_first), else 128 columns each
  const float* cmax;       // [M][np·cpp] chunk maxima (-inf past a partial's last)
  const float* zlog;       // [M][V] logits of the chunks that were kept
  float* logprob;          // [M][n] or null
  float* entropy;          // [M] or null
  float* lse_out;          // [M]
  float* loss;             // distillation: [M]
  int32_t* top_ids;        // [M][k]
  float* top_logprob;      // [M][k]
  // preparation
  int2* sorted;            // [M][n]
  unsigned* bound;         // [M][kp] or null
  float4* rowp;            // backward: [M]
  const float* lse;        // [M]
  const float* ent;        // [M] or null
  const float* dlogprob;   // [M][n] or null
  const float* dentropy;   // [M] or null
  const float* dloss;      // distillation: [M]
};

constexpr int kHeadRowWarps = 4;

// One warp a row.  Sorts the row's tokens by id (by counting the entries before each: n <=
// 128 values in shared memory) with their position (forward) or coefficient (backward);
// ignored and out-of-range entries go last as 0x7fffffff and match no column.  Clears the
// forward's bounds; writes the backward's row coefficients.
template <bool BWD>
__global__ void __launch_bounds__(32 * kHeadRowWarps) head_prep_kernel(const HeadRowArgs a) {
  griddep_enter();  // the previous kernel in the stream completed (see ptx.cuh)
  __shared__ int sid[kHeadRowWarps][kHeadMaxIds];
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row = blockIdx.x * kHeadRowWarps + w;
  if (row >= a.M) return;  // whole warps
  const int32_t* ids = a.ids + static_cast<size_t>(row) * a.n;
  float coef[kHeadPerLane];
  float csum = 0.0f;
  if (BWD) {
    if (a.teacher != nullptr) {
      const bool any = teacher_log_softmax(ids, a.teacher + static_cast<size_t>(row) * a.n, a.n, a.ignore, a.scale,
                                           lane, coef);
      const float g = any ? -a.dloss[row] : 0.0f;
#pragma unroll
      for (int u = 0; u < kHeadPerLane; ++u) coef[u] = any ? g * expf(coef[u]) : 0.0f;
    } else {
#pragma unroll
      for (int u = 0; u < kHeadPerLane; ++u) {
        const int i = lane + 32 * u;
        coef[u] = a.dlogprob != nullptr && i < a.n && ids[i] != a.ignore ? a.dlogprob[static_cast<size_t>(row) * a.n + i]
                                                                       : 0.0f;
      }
    }
#pragma unroll
    for (int u = 0; u < kHeadPerLane; ++u) csum += coef[u];
    csum = warp_sum(csum);
    if (lane == 0) {
      const float gh = a.dentropy != nullptr ? a.dentropy[row] : 0.0f;
      a.rowp[row] = make_float4(a.lse[row], gh != 0.0f ? fmaf(gh, a.ent[row], csum) : csum, gh, 0.0f);
    }
  }
  for (int i = lane; i < a.n; i += 32) {
    const int id = ids[i];
    sid[w][i] = id == a.ignore || id < 0 || id >= a.V ? 0x7fffffff : id;
  }
  __syncwarp();
#pragma unroll
  for (int u = 0; u < kHeadPerLane; ++u) {
    const int i = lane + 32 * u;
    if (i < a.n) {
      const int id = sid[w][i];
      int before = 0;
      for (int j = 0; j < a.n; ++j) before += sid[w][j] < id || (sid[w][j] == id && j < i);
      a.sorted[static_cast<size_t>(row) * a.n + before] = make_int2(id, BWD ? __float_as_int(coef[u]) : i);
    }
  }
  if (!BWD && a.bound != nullptr && lane < a.kp) a.bound[static_cast<size_t>(row) * a.kp + lane] = 0u;
}

// First vocabulary entry of partial i of np of head_rows_kernel: ranges of multiples of 16.
__host__ __device__ __forceinline__ int hr_first(int V, int i, int np) {
  return static_cast<int>(static_cast<long long>((V + 15) / 16) * i / np) * 16;
}

// One warp a row: joins the row's partials (in a fixed order), and from them the
// log-probabilities, the entropy and the distillation loss.
__global__ void __launch_bounds__(32 * kHeadRowWarps) head_finalize_kernel(const HeadRowArgs a) {
  griddep_enter();  // the previous kernel in the stream completed (see ptx.cuh)
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row = blockIdx.x * kHeadRowWarps + w;
  if (row >= a.M) return;  // whole warps
  const float4* part = a.part + static_cast<size_t>(row) * a.np;
  float m = -INFINITY;
  for (int i = lane; i < a.np; i += 32) m = fmaxf(m, part[i].x);
  m = warp_max(m);
  float s = 0.0f, t = 0.0f;
  for (int i = lane; i < a.np; i += 32) {
    const float4 q = part[i];
    const float d = q.x - m, e = expf(d);
    s = fmaf(q.y, e, s);
    t = fmaf(fmaf(d, q.y, q.z), e, t);
  }
  s = warp_sum(s);
  t = warp_sum(t);
  const float ls = logf(s);
  if (lane == 0) {
    a.lse_out[row] = m + ls;
    if (a.entropy != nullptr) a.entropy[row] = ls - t / s;
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
        lp[u] = id >= 0 && id < a.V ? (a.id_logit[static_cast<size_t>(row) * a.n + i] - m) - ls : NAN;
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

// One block a row, with alternatives: as head_finalize_kernel (no loss), then the k best.  The
// chunks that reach the row's bound go to a list, 1024 chunks a round; their logits, as far as
// they beat the k-th key known, to a buffer that is sorted and cut back to k when it fills.
// Buffer order varies from run to run, the k largest keys do not.
constexpr int kTopThreads = 128, kTopBuf = 512, kTopRound = 1024;
__global__ void __launch_bounds__(kTopThreads) head_finalize_top_kernel(const HeadRowArgs a) {
  griddep_enter();  // the previous kernel in the stream completed (see ptx.cuh)
  __shared__ unsigned long long buf[kTopBuf];
  __shared__ int2 list[kTopRound];
  __shared__ float red[4][3];
  __shared__ int list_n, buf_n;
  const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31;
  const int row = blockIdx.x;
  const float4* part = a.part + static_cast<size_t>(row) * a.np;
  float m = -INFINITY, own = -INFINITY;  // own: the largest bound of a partial's own (few rows)
  for (int i = tid; i < a.np; i += kTopThreads) {
    const float4 q = part[i];
    m = fmaxf(m, q.x);
    own = fmaxf(own, q.w);
  }
  // the partials' maxima in groups (i mod kp: the lane mod kp): the least group's is a bound
  float g = m;
  m = warp_max(m);
  own = warp_max(own);
  for (int o = a.kp; o < 32; o <<= 1) g = fmaxf(g, __shfl_xor_sync(0xffffffffu, g, o));
  __shared__ float groups[4][32];
  groups[w][lane] = g;
  if (lane == 0) {
    red[w][0] = m;
    red[w][1] = own;
  }
  if (tid == 0) buf_n = 0;
  __syncthreads();
  m = fmaxf(fmaxf(red[0][0], red[1][0]), fmaxf(red[2][0], red[3][0]));
  own = fmaxf(fmaxf(red[0][1], red[1][1]), fmaxf(red[2][1], red[3][1]));
  float low;
  if (a.few) {
    g = fmaxf(fmaxf(groups[0][lane], groups[1][lane]), fmaxf(groups[2][lane], groups[3][lane]));
    for (int o = 1; o < a.kp; o <<= 1) g = fminf(g, __shfl_xor_sync(0xffffffffu, g, o));
    low = fmaxf(g, own);
  } else {
    uint32_t o = lane < a.kp ? a.bound[static_cast<size_t>(row) * a.kp + lane] : 0xffffffffu;
    low = unord_f32(max(__reduce_min_sync(0xffffffffu, o), ord_f32(-INFINITY)));  // 0: an empty group
  }
  float s = 0.0f, t = 0.0f;
  for (int i = tid; i < a.np; i += kTopThreads) {
    const float4 q = part[i];
    const float d = q.x - m, e = expf(d);
    s = fmaf(q.y, e, s);
    t = fmaf(fmaf(d, q.y, q.z), e, t);
  }
  s = warp_sum(s);
  t = warp_sum(t);
  __syncthreads();
  if (lane == 0) {
    red[w][0] = s;
    red[w][1] = t;
  }
  __syncthreads();
  s = (red[0][0] + red[1][0]) + (red[2][0] + red[3][0]);
  t = (red[0][1] + red[1][1]) + (red[2][1] + red[3][1]);
  const float ls = logf(s);
  if (tid == 0) {
    a.lse_out[row] = m + ls;
    if (a.entropy != nullptr) a.entropy[row] = ls - t / s;
  }
  if (tid < a.n) {
    const size_t at = static_cast<size_t>(row) * a.n + tid;
    const int id = a.ids[at];
    float lp = 0.0f;
    if (id != a.ignore) lp = id >= 0 && id < a.V ? (a.id_logit[at] - m) - ls : NAN;
    a.logprob[at] = lp;
  }

  // ---- the alternatives: keys above kth may be among the k best
  unsigned long long kth = ord_f32(low) > 0 ? (static_cast<unsigned long long>(ord_f32(low)) << 32) - 1 : 0;
  const int chunks = a.np * a.cpp;
  const float* cmax = a.cmax + static_cast<size_t>(row) * chunks;
  const float* zrow = a.zlog + static_cast<size_t>(row) * a.V;
  auto cut = [&](bool last) {  // all threads; buf_n keys -> the k largest, in order
    __syncthreads();
    const int n = buf_n;
    int size = 32;
    while (size < n) size <<= 1;
    for (int i = n + tid; i < size; i += kTopThreads) buf[i] = 0;
    __syncthreads();
    for (int kk = 2; kk <= size; kk <<= 1)
      for (int j = kk >> 1; j > 0; j >>= 1) {
        for (int i = tid; i < size / 2; i += kTopThreads) {
          const int x = ((i & ~(j - 1)) << 1) | (i & (j - 1)), y = x | j;
          const unsigned long long kx = buf[x], ky = buf[y];
          if ((kx < ky) == ((x & kk) == 0)) {
            buf[x] = ky;
            buf[y] = kx;
          }
        }
        __syncthreads();
      }
    if (n >= a.k && buf[a.k - 1] > kth) kth = buf[a.k - 1];
    if (!last) {
      __syncthreads();
      if (tid == 0) buf_n = min(n, a.k);
      __syncthreads();
    }
  };
  for (int q0 = 0; q0 < chunks; q0 += kTopRound) {
    if (tid == 0) list_n = 0;
    __syncthreads();
#pragma unroll
    for (int u = 0; u < kTopRound / kTopThreads; ++u) {
      const int q = q0 + u * kTopThreads + tid;
      if (q < chunks) {
        const float cm = cmax[q];
        if (cm >= low) {
          const int part_i = a.few ? q / a.cpp : 0;
          const int col = a.few ? hr_first(a.V, part_i, a.np) + (q - part_i * a.cpp) * 32 : q * 32;
          if (top_key(cm, col) > kth) list[atomicAdd(&list_n, 1)] = make_int2(q, col);
        }
      }
    }
    __syncthreads();
    const int ln = list_n;
    for (int i0 = 0; i0 < ln;) {
      const int room = min((kTopBuf - buf_n) / 32, ln - i0);  // chunks that fit: at least one
      __syncthreads();
      for (int i = i0 + w; i < i0 + room; i += 4) {
        const int2 e = list[i];
        const int end = a.few ? min(a.V, hr_first(a.V, e.x / a.cpp + 1, a.np)) : a.V;
        unsigned long long key = 0;
        if (e.y + lane < end) key = top_key(zrow[e.y + lane], e.y + lane);
        const uint32_t keep = __ballot_sync(0xffffffffu, key > kth);
        int base = 0;
        if (lane == 0 && keep) base = atomicAdd(&buf_n, __popc(keep));
        base = __shfl_sync(0xffffffffu, base, 0);
        if (key > kth) buf[base + __popc(keep & ((1u << lane) - 1u))] = key;
      }
      i0 += room;
      if (i0 < ln) cut(false);
      else __syncthreads();
    }
    if (buf_n > kTopBuf - 32) cut(false);
  }
  cut(true);
  if (tid < a.k) {
    const unsigned long long key = tid < min(buf_n, kTopBuf) ? buf[tid] : 0ull;
    const size_t at = static_cast<size_t>(row) * a.k + tid;
    a.top_ids[at] = key != 0 ? static_cast<int32_t>(0xffffffffu - static_cast<uint32_t>(key)) : -1;
    a.top_logprob[at] = key != 0 ? (unord_f32(static_cast<uint32_t>(key >> 32)) - m) - ls : NAN;
  }
}

// The backward from a saved forward, in place: e^{z-m} of a tile (fp16) becomes (bf16)
// dz = scale·(Σ c - p·(Σc + g_H·(log p + H))) with p = e^{z-m}·e^{m-lse}.  Streams M·V 16-bit
// values in and out (bound by HBM).  One warp takes 2048 columns of a row, 8 a lane and step.
constexpr int kHeadSpan = 16;  // tiles a warp
__global__ void __launch_bounds__(32 * kHeadRowWarps)
    head_dlogits_saved_kernel(const HeadArgs h, int M, int V, int np) {
  griddep_enter();  // the previous kernel in the stream completed (see ptx.cuh)
  const int lane = threadIdx.x & 31;
  const int spans = (np + kHeadSpan - 1) / kHeadSpan;
  const long long job = static_cast<long long>(blockIdx.x) * kHeadRowWarps + (threadIdx.x >> 5);
  const int row = static_cast<int>(job / spans);
  const int t0 = static_cast<int>(job % spans) * kHeadSpan;
  if (row >= M) return;
  const float4 rp = h.rowp[row];
  const int2* sorted = h.sorted + static_cast<size_t>(row) * h.n;
  int pos = head_first_id(sorted, h.n, t0 * kHeadTile);
  int2 e = pos < h.n ? sorted[pos] : make_int2(0x7fffffff, 0);
  __half* zrow = h.expz + static_cast<size_t>(row) * V;
  const float* tm = h.tile_max + static_cast<size_t>(row) * np;
  constexpr int STEPS = kHeadSpan * kHeadTile / 256;
  uint4 x[STEPS];
  float shift[STEPS];
#pragma unroll
  for (int u = 0; u < STEPS; ++u) {
    const int col = t0 * kHeadTile + u * 256 + lane * 8;
    if (col < V) x[u] = *reinterpret_cast<const uint4*>(zrow + col);
    shift[u] = col < V ? tm[col / kHeadTile] - rp.x : 0.0f;
  }
#pragma unroll
  for (int u = 0; u < STEPS; ++u) {
    const int col = t0 * kHeadTile + u * 256 + lane * 8;
    const uint32_t in[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
    float d[8];
    const float f = __expf(shift[u]);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float ez = __half2float(__ushort_as_half(static_cast<unsigned short>(in[j >> 1] >> ((j & 1) ? 16 : 0))));
      const float p = ez * f;
      float wgt = rp.y;
      if (rp.z != 0.0f && ez > 0.0f) wgt = fmaf(rp.z, __logf(ez) + shift[u], wgt);
      d[j] = -h.scale * p * wgt;
    }
    const int end = t0 * kHeadTile + u * 256 + 256;
    while (e.x < end) {  // the same for every lane
      const int at = e.x - col;
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j == at) d[j] = fmaf(h.scale, __int_as_float(e.y), d[j]);
      e = ++pos < h.n ? sorted[pos] : make_int2(0x7fffffff, 0);
    }
    if (col < V)
      *reinterpret_cast<uint4*>(zrow + col) = make_uint4(pack_bf16x2(d[0], d[1]), pack_bf16x2(d[2], d[3]),
                                                         pack_bf16x2(d[4], d[5]), pack_bf16x2(d[6], d[7]));
  }
}

}  // namespace lora
