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
// A tile (256 vocabulary entries of one row, in one thread) leaves (m, Σe, Σd·e) with
// m = max z, d = z - m, e = e^d.  Both sums stay well conditioned: the entropy of the tile is
// log Σe - Σd·e/Σe, a sum of non-negative terms, and tiles are joined by
// Σe ← e^{m-M}·Σe, Σd·e ← e^{m-M}·(Σd·e + (m - M)·Σe).
#pragma once

#include "gemm_common.cuh"

namespace lora {

constexpr int kHeadMaxIds = 128;   // given tokens (or teacher entries) a row
constexpr int kHeadMaxTop = 32;    // alternatives a row: one warp lane each
constexpr int kHeadListThreads = 128;

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

// The k best keys one thread has seen, unsorted, in shared memory ([slot][thread]: no bank
// conflicts), with the smallest of them once the list is full.
struct TopList {
  unsigned long long* s;  // this thread's column
  int k, cnt, minpos;
  unsigned long long minkey;
  __device__ __forceinline__ void init(unsigned long long* col, int k_) {
    s = col;
    k = k_;
    cnt = 0;
    minpos = 0;
    minkey = 0;
  }
  // Logits below this cannot enter: an equal one has a larger id than the list's.
  __device__ __forceinline__ float enters_from() const {
    if (cnt < k) return -INFINITY;
    return unord_f32(static_cast<uint32_t>(minkey >> 32) + 1u);
  }
  __device__ __forceinline__ void rescan() {
    minkey = s[0];
    minpos = 0;
    for (int i = 1; i < k; ++i) {
      const unsigned long long x = s[i * kHeadListThreads];
      if (x < minkey) {
        minkey = x;
        minpos = i;
      }
    }
  }
  __device__ __forceinline__ void offer(float z, int id) {
    const unsigned long long key = top_key(z, id);
    if (cnt < k) {
      s[cnt * kHeadListThreads] = key;
      if (++cnt == k) rescan();
    } else if (key > minkey) {
      s[minpos * kHeadListThreads] = key;
      rescan();
    }
  }
};

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
// First pass over a row's nv <= 256 accumulator columns at tbase: the largest logit and, for
// the alternatives, a bound.  The columns fall into kp >= k disjoint groups (column mod kp);
// the least of the groups' maxima is at most the kp-th largest logit, so nothing below it is
// among the k best.  `bound` (pair kernel) holds the groups' maxima over every tile of the
// row seen so far, raised by atomic max: which tiles got there first changes how many
// candidates are kept, never which k remain in the end.
__device__ __forceinline__ float head_tile_max(const HeadArgs& h, uint32_t tbase, int nv, bool in, unsigned* bound,
                                               float& lower) {
  float m = -INFINITY;
  lower = -INFINITY;
  if (h.k == 0) {
#pragma unroll 1
    for (int c = 0; c * 32 < nv; ++c) {
      uint32_t v[32];
      tmem_ld_32x32b_x32(tbase + c * 32, v);
      tmem_ld_wait();
      const int n = nv - c * 32;
      if (n >= 32) {
#pragma unroll
        for (int j = 0; j < 32; ++j) m = fmaxf(m, __uint_as_float(v[j]));
      } else {
#pragma unroll
        for (int j = 0; j < 32; ++j)
          if (j < n) m = fmaxf(m, __uint_as_float(v[j]));
      }
    }
    return m * h.scale;
  }
  float g[32];
#pragma unroll
  for (int j = 0; j < 32; ++j) g[j] = -INFINITY;
#pragma unroll 1
  for (int c = 0; c * 32 < nv; ++c) {
    uint32_t v[32];
    tmem_ld_32x32b_x32(tbase + c * 32, v);
    tmem_ld_wait();
    const int n = nv - c * 32;
#pragma unroll
    for (int j = 0; j < 32; ++j)
      if (j < n) g[j] = fmaxf(g[j], __uint_as_float(v[j]));
  }
#pragma unroll
  for (int s = 16; s > 0; s >>= 1)
    if (h.kp <= s) {
#pragma unroll
      for (int j = 0; j < s; ++j) g[j] = fmaxf(g[j], g[j + s]);
    }
  uint32_t low = 0xffffffffu;
#pragma unroll
  for (int j = 0; j < 32; ++j)
    if (j < h.kp) {
      m = fmaxf(m, g[j]);
      uint32_t o = ord_f32(g[j] * h.scale);
      if (bound != nullptr && in) {
        const uint32_t b = __ldcg(bound + j);
        if (o > b) atomicMax(bound + j, o);
        o = max(o, b);
      }
      low = min(low, o);
    }
  lower = unord_f32(low);
  return m * h.scale;
}

// Second pass: the sums, the candidates for the alternatives and (expz != null) e^{z-m} for
// the backward, in fp16: at most 1, so its 11 bits beat bf16's 8 down to 2^-15, and what lies
// below weighs less in dX than the rounding of the tile's largest entry.  Columns that few lanes want (a candidate, below: a given token) are
// read again from TMEM one at a time by the whole warp, since a register cannot be indexed.
__device__ __forceinline__ RowStats head_tile_sums(const HeadArgs& h, uint32_t tbase, int nv, int v0, bool in, float m,
                                                   float lower, TopList& list, __half* expz) {
  float s0 = 0.0f, s1 = 0.0f, t0 = 0.0f, t1 = 0.0f;
#pragma unroll 1
  for (int c = 0; c * 32 < nv; ++c) {
    uint32_t v[32];
    tmem_ld_32x32b_x32(tbase + c * 32, v);
    tmem_ld_wait();
    const int n = nv - c * 32;
    uint32_t mask = 0;
    if (h.k > 0) {
      const float from = in ? fmaxf(lower, list.enters_from()) : INFINITY;
      float cm = -INFINITY;
#pragma unroll
      for (int j = 0; j < 32; ++j)
        if (j < n) cm = fmaxf(cm, __uint_as_float(v[j]));
      if (in && cm * h.scale >= from) {
#pragma unroll
        for (int j = 0; j < 32; ++j)
          if (j < n && __uint_as_float(v[j]) * h.scale >= from) mask |= 1u << j;
      }
      __syncwarp();
    }
#pragma unroll
    for (int j = 0; j < 32; j += 2) {
      if (j < n) {  // nv is even (a multiple of 8)
        const float d0 = __uint_as_float(v[j]) * h.scale - m, d1 = __uint_as_float(v[j + 1]) * h.scale - m;
        const float e0 = __expf(d0), e1 = __expf(d1);
        s0 += e0;
        s1 += e1;
        t0 = fmaf(d0, e0, t0);
        t1 = fmaf(d1, e1, t1);
        v[j >> 1] = pack_f16x2(e0, e1);
      }
    }
    if (expz != nullptr && in) {
#pragma unroll
      for (int q = 0; q < 4; ++q)
        if (q * 8 < n)
          *reinterpret_cast<uint4*>(expz + c * 32 + q * 8) = make_uint4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
    }
    if (h.k > 0) {
      uint32_t want = __reduce_or_sync(0xffffffffu, mask);
      while (want) {
        const int j = __ffs(want) - 1;
        want &= want - 1;
        const float z = __uint_as_float(tmem_ld_32x32b_x1(tbase + c * 32 + j)) * h.scale;
        if ((mask >> j) & 1u) list.offer(z, v0 + c * 32 + j);
        __syncwarp();
      }
    }
  }
  return RowStats{m, s0 + s1, t0 + t1};
}

// The logits of the row's given tokens that fall into columns [v0, v0 + nv).  sorted: the
// row's (id, position) by id, pos: the first of them at or above v0.
__device__ __forceinline__ void head_tile_ids(const HeadArgs& h, uint32_t tbase, int nv, int v0, bool in, int row,
                                              int pos) {
  const int2* sorted = h.sorted + static_cast<size_t>(row) * h.n;
  int2 e = in && pos < h.n ? sorted[pos] : make_int2(0x7fffffff, 0);
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

// The pair kernel's forward epilogue of one tile (all lanes of the warp take part).
__device__ __forceinline__ void head_fwd_tile(const HeadArgs& h, uint32_t tbase, int nv, int nb, int num_n, bool in,
                                              int row, int first_id, unsigned long long* list_col, int ldz) {
  unsigned* bound = h.k > 0 && in ? h.bound + static_cast<size_t>(row) * h.kp : nullptr;
  float lower;
  const float m = head_tile_max(h, tbase, nv, in, bound, lower);
  TopList list;
  list.init(list_col, h.k);
  __half* expz = h.expz != nullptr ? h.expz + static_cast<size_t>(row) * ldz + nb * 256 : nullptr;
  const RowStats st = head_tile_sums(h, tbase, nv, nb * 256, in, m, lower, list, expz);
  if (h.n > 0) head_tile_ids(h, tbase, nv, nb * 256, in, row, first_id);
  if (!in) return;
  const size_t at = static_cast<size_t>(row) * num_n + nb;
  h.part[at] = make_float4(st.m, st.s, st.t, __int_as_float(list.cnt));
  if (h.expz != nullptr) h.tile_max[at] = st.m;
  for (int i = 0; i < list.cnt; ++i) h.cand[at * h.k + i] = list.s[i * kHeadListThreads];
}

// dz of one accumulator tile in bf16 (recomputed logits).  rowp: (lse, Σc + g_H·H, g_H).
__device__ __forceinline__ void head_dlogits_tile(const HeadArgs& h, uint32_t tbase, int nv, int v0, bool in, int row,
                                                  __nv_bfloat16* orow) {
  float4 rp = make_float4(0.f, 0.f, 0.f, 0.f);
  const int2* sorted = h.sorted + static_cast<size_t>(row) * h.n;
  int pos = h.n;
  if (in) {
    rp = h.rowp[row];
    pos = head_first_id(sorted, h.n, v0);
  }
  int2 e = pos < h.n ? sorted[pos] : make_int2(0x7fffffff, 0);
#pragma unroll 1
  for (int c = 0; c * 32 < nv; ++c) {
    uint32_t v[32];
    tmem_ld_32x32b_x32(tbase + c * 32, v);
    tmem_ld_wait();
    const int n = nv - c * 32;
    if (in) {
      float d[32];
#pragma unroll
      for (int j = 0; j < 32; ++j) {
        const float lp = __uint_as_float(v[j]) * h.scale - rp.x;
        const float w = rp.z != 0.0f ? fmaf(rp.z, lp, rp.y) : rp.y;
        d[j] = -h.scale * __expf(lp) * w;
      }
      while (e.x < v0 + c * 32 + n && e.x < v0 + c * 32 + 32) {
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
  const unsigned long long* cand;
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

// Descending bitonic sort of size (a power of two) keys in shared memory by one warp.
__device__ __forceinline__ void warp_sort_desc(unsigned long long* s, int size, int lane) {
  for (int k = 2; k <= size; k <<= 1)
    for (int j = k >> 1; j > 0; j >>= 1) {
      for (int i = lane; i < size / 2; i += 32) {
        const int a = ((i & ~(j - 1)) << 1) | (i & (j - 1)), b = a | j;
        const unsigned long long x = s[a], y = s[b];
        if ((x < y) == ((a & k) == 0)) {
          s[a] = y;
          s[b] = x;
        }
      }
      __syncwarp();
    }
}

// One warp a row: joins the row's partials (in a fixed order), and from them the
// log-probabilities, the entropy, the distillation loss and the alternatives.  The k best
// among the partials' candidates: a bound from the partials' maxima (groups as in
// head_tile_max) drops most of them; the rest pass through a buffer of 256 keys that is
// sorted and cut back to k whenever it fills.
constexpr int kHeadBuf = 256;
__global__ void __launch_bounds__(32 * kHeadRowWarps) head_finalize_kernel(const HeadRowArgs a) {
  griddep_enter();  // the previous kernel in the stream completed (see ptx.cuh)
  __shared__ unsigned long long buf_s[kHeadRowWarps][kHeadBuf];
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row = blockIdx.x * kHeadRowWarps + w;
  if (row >= a.M) return;  // whole warps
  const float4* part = a.part + static_cast<size_t>(row) * a.np;
  float m = -INFINITY;
  for (int i = lane; i < a.np; i += 32) m = fmaxf(m, part[i].x);
  const float lane_max = m;
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
  if (a.k == 0) return;
  // group maxima: lane l holds those of partials l, l + 32, ..., all of group l mod kp
  float g = lane_max;
  for (int o = a.kp; o < 32; o <<= 1) g = fmaxf(g, __shfl_xor_sync(0xffffffffu, g, o));
  for (int o = 1; o < a.kp; o <<= 1) g = fminf(g, __shfl_xor_sync(0xffffffffu, g, o));
  unsigned long long* buf = buf_s[w];
  unsigned long long kth = 0;  // keys up to this one are out
  if (ord_f32(g) > 0) kth = (static_cast<unsigned long long>(ord_f32(g)) << 32) - 1;
  int fill = 0;
  auto cut = [&]() {
    int size = 32;
    while (size < fill) size <<= 1;
    for (int i = fill + lane; i < size; i += 32) buf[i] = 0;
    __syncwarp();
    warp_sort_desc(buf, size, lane);
    if (fill >= a.k) {
      fill = a.k;
      const unsigned long long last = buf[a.k - 1];
      if (last > kth) kth = last;
    }
  };
  for (int i0 = 0; i0 < a.np; i0 += 32) {
    const int i = i0 + lane;
    float4 q = make_float4(-INFINITY, 0.f, 0.f, 0.f);
    if (i < a.np) q = part[i];
    const int cnt = __float_as_int(q.w);
    uint32_t have = __ballot_sync(0xffffffffu, i < a.np && cnt > 0 && q.x >= g);
    while (have) {
      const int src = __ffs(have) - 1;
      have &= have - 1;
      const int n = __shfl_sync(0xffffffffu, cnt, src);
      unsigned long long key = 0;
      if (lane < n) key = a.cand[(static_cast<size_t>(row) * a.np + i0 + src) * a.k + lane];
      const uint32_t keep = __ballot_sync(0xffffffffu, key > kth);
      if (key > kth) buf[fill + __popc(keep & ((1u << lane) - 1u))] = key;
      fill += __popc(keep);
      __syncwarp();
      if (fill > kHeadBuf - 32) cut();
    }
  }
  cut();
  if (lane < a.k) {
    const unsigned long long key = lane < fill ? buf[lane] : 0ull;
    const size_t at = static_cast<size_t>(row) * a.k + lane;
    a.top_ids[at] = key != 0 ? static_cast<int32_t>(0xffffffffu - static_cast<uint32_t>(key)) : -1;
    a.top_logprob[at] = key != 0 ? (unord_f32(static_cast<uint32_t>(key >> 32)) - m) - ls : NAN;
  }
}

// The backward from a saved forward, in place: e^{z-m} of a tile (fp16) becomes (bf16)
// dz = scale·(Σ c - p·(Σc + g_H·(log p + H))) with p = e^{z-m}·e^{m-lse}.  Streams M·V bf16
// values in and out (bound by HBM).  One warp takes 2048 columns of a row, 8 a lane and tile.
constexpr int kHeadSpan = 8;  // tiles a warp
__global__ void __launch_bounds__(32 * kHeadRowWarps)
    head_dlogits_saved_kernel(const HeadArgs h, int M, int V, int num_n) {
  griddep_enter();  // the previous kernel in the stream completed (see ptx.cuh)
  const int lane = threadIdx.x & 31;
  const int spans = (num_n + kHeadSpan - 1) / kHeadSpan;
  const long long job = static_cast<long long>(blockIdx.x) * kHeadRowWarps + (threadIdx.x >> 5);
  const int row = static_cast<int>(job / spans);
  const int nb0 = static_cast<int>(job % spans) * kHeadSpan;
  if (row >= M) return;
  const float4 rp = h.rowp[row];
  const int2* sorted = h.sorted + static_cast<size_t>(row) * h.n;
  int pos = head_first_id(sorted, h.n, nb0 * 256);
  int2 e = pos < h.n ? sorted[pos] : make_int2(0x7fffffff, 0);
  __half* zrow = h.expz + static_cast<size_t>(row) * V;
  const float* tm = h.tile_max + static_cast<size_t>(row) * num_n;
  uint4 x[kHeadSpan];
  float shift[kHeadSpan];
#pragma unroll
  for (int u = 0; u < kHeadSpan; ++u) {
    const int col = (nb0 + u) * 256 + lane * 8;
    if (col < V) x[u] = *reinterpret_cast<const uint4*>(zrow + col);
    shift[u] = nb0 + u < num_n ? tm[nb0 + u] - rp.x : 0.0f;
  }
#pragma unroll
  for (int u = 0; u < kHeadSpan; ++u) {
    const int col = (nb0 + u) * 256 + lane * 8;
    const uint32_t in[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
    float d[8];
    const float f = __expf(shift[u]);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float ez = __half2float(__ushort_as_half(static_cast<unsigned short>(in[j >> 1] >> (j & 1 ? 16 : 0))));
      const float p = ez * f;
      float wgt = rp.y;
      if (rp.z != 0.0f && ez > 0.0f) wgt = fmaf(rp.z, __logf(ez) + shift[u], wgt);
      d[j] = -h.scale * p * wgt;
    }
    const int end = (nb0 + u) * 256 + 256;
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
