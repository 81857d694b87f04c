// Scoring of logits rows: the log-prob of a given token, the entropy of the row's distribution
// and its K most probable tokens with their log-probs, in one pass over the logits.
//
//   log p_v = z_v/tau - log sum_u exp(z_u/tau),   H = -sum_v p_v log p_v
//
// A row is read once from HBM in warp tiles (grpo_vocab.cuh), which gives the log-sum-exp and the
// entropy. For the K largest logits every tile also leaves the maximum of each group of elements
// (a lane's vectors of one tile, or single vectors of a short row). The K-th largest group maximum
// bounds the K-th largest logit from below, as K groups hold an element at least that large. A
// histogram of the group maxima finds that bound up to a bucket, and only the groups that reach it
// are read again: about K of them, from L2. What survives of them is ranked exactly, equal logits by
// index. Any row is served: where the bound lets more than the candidate buffer through (ties, rows
// with fewer than K finite logits), the buffer is cut back to its K best as it fills, which raises
// the bound.
//
// Two kernels, chosen by the number and length of the rows (launch rule at the end of the file):
//  * stream_kernel  many long rows: one persistent CTA per SM whose 12 streaming warps never stop,
//                   while 8 others finish (LSE, bound, ranking) the rows before. 8192 x 151936 bf16,
//                   K = 64: 390 us, 6.39 TB/s, bound by HBM; K = 256: 600 us, and shorter rows (50264: 148 us
//                   at K = 0, 187 at 20, 200 at 37), by the finishing warps: about 8 us a row and group,
//                   against 2.4 us of reading at 50264
//  * row_kernel     few or short rows: one CTA per row, or a cluster that shares its reading
#include <algorithm>
#include <atomic>
#include <cmath>
#include <mutex>

#include "grpo_vocab.cuh"

namespace grpo {

size_t max_smem_optin();

namespace score {

constexpr int kMaxGroups = 5120;            // group maxima kept per row
constexpr int kMaxBlocks = kMaxGroups / 32;  // blocks (of `fold` tiles) per row
constexpr int kBuckets = 256;
constexpr int kListCap = 1024;  // listed groups; more (rows of ties) are walked without a list

struct Args {
  const void* logits;
  int64_t T, V, ld;
  const int64_t* tok_src;
  const int32_t* target;
  const uint8_t* mask;
  float c;  // log2(e) / temperature
  int32_t K;
  float *logp, *entropy;
  int32_t* top_idx;
  float* top_logp;
  int64_t ld_top;
  // the row's cut into tiles, blocks and groups (functions of V): `fold` consecutive tiles form a
  // block (1 but for vocabularies past 160 tiles), a lane's elements of a block a group; `by_vec`:
  // every vector is a group of its own
  int32_t n_tiles, n_blocks, fold, n_groups;
  bool by_vec;
  int32_t n_cta;  // row_kernel: CTAs per row
  int32_t slots;  // stream_kernel: row states
};

// What the reading of a row leaves: per block the softmax partial (m, s, q) and the largest and the
// smallest finite of its group maxima, and the group maxima.
struct RowState {
  float4* part;  // [n_blocks] m, s, q, largest
  float* lo;     // [n_blocks] smallest
  float* gmax;   // [n_groups]
};

// Scratch of the NT threads that finish a row. kCap: candidates; K kept and one round's fit.
template <int NT>
struct Finish {
  static constexpr int kCap = NT < 64 ? 512 : NT * 8;
  static_assert(GRPO_TOPK_MAX + NT * 4 <= kCap && (kCap & (kCap - 1)) == 0, "a round fits; the sort takes a power of two");
  unsigned long long cand[kCap];
  int hist[kBuckets];
  union {
    uint16_t list[kListCap];  // the groups that reach the bound
    uint16_t place[kCap];     // candidates by bucket
  };
  float lse_m, lse_l;
  uint32_t zmin;  // the listed groups' smallest maximum, as an ordered integer
  int bucket, n_list, n_cand;
  int broken;  // stream_kernel: a wait gave up before this row
};

__device__ __forceinline__ uint32_t order_of(float z) {
  const uint32_t b = __float_as_uint(z);
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float of_order(uint32_t o) {
  return __uint_as_float((o & 0x80000000u) ? (o & 0x7FFFFFFFu) : ~o);
}
// Descending order of (logit, then ascending index) as one unsigned key; -0 counts as +0.
__device__ __forceinline__ unsigned long long make_key(float z, uint32_t idx) {
  return ((unsigned long long)order_of(z + 0.f) << 32) | (uint32_t)~idx;
}
__device__ __forceinline__ uint32_t key_idx(unsigned long long k) { return ~(uint32_t)k; }
__device__ __forceinline__ float key_logit(unsigned long long k) { return of_order((uint32_t)(k >> 32)); }

// The log-prob of a logit in a row with shift m and log2 l2 of its sum.
__device__ __forceinline__ float logp_of(float z, float c, float m, float l2) {
  return fmaf(fmaf(z, scale_at(m, c), -m), unit_at(m, c), -l2) * kLn2;
}

// Bucket of a logit in [0, kBuckets): monotone in z.
__device__ __forceinline__ int bucket_of(float z, float lo, float scale) {
  return min(kBuckets - 1, max(0, __float2int_rd((z - lo) * scale)));
}

// The first n candidates sorted in descending order (bitonic, padded with 0: below every key).
template <int NT>
__device__ __noinline__ void sort_candidates(unsigned long long* k, int n, int tid, int bar) {
  int P = 1;
  while (P < n) P <<= 1;
  for (int i = n + tid; i < P; i += NT) k[i] = 0ull;
  for (int size = 2; size <= P; size <<= 1)
    for (int stride = size >> 1; stride > 0; stride >>= 1) {
      named_bar_sync(bar, NT);
      for (int i = tid; i < P / 2; i += NT) {
        const int a = 2 * i - (i & (stride - 1)), b = a + stride;
        const unsigned long long x = k[a], y = k[b];
        if (((a & size) == 0) ? x < y : x > y) {
          k[a] = y;
          k[b] = x;
        }
      }
    }
  named_bar_sync(bar, NT);
}

// A row that is not scored.
__device__ __forceinline__ void write_none(const Args& a, int64_t out, int tid, int nt, float f, float top) {
  if (tid == 0) {
    if (a.logp) a.logp[out] = f;
    if (a.entropy) a.entropy[out] = f;
  }
  for (int i = tid; i < a.K; i += nt) {
    a.top_idx[out * a.ld_top + i] = -1;
    if (a.top_logp) a.top_logp[out * a.ld_top + i] = top;
  }
}

// Readies the scratch for a row; a barrier of the NT threads comes before finish_row.
template <int NT>
__device__ __forceinline__ void finish_reset(Finish<NT>& sh, int tid) {
  for (int i = tid; i < kBuckets; i += NT) sh.hist[i] = 0;
  if (tid == 0) {
    sh.n_list = sh.n_cand = 0;
    sh.zmin = 0xFFFFFFFFu;
  }
}

// The rest of a row after its reading, by NT threads (named barrier `bar`): every one of them
// calls it. zy: the target's logit, y_ok whether the row has that token. `release` runs in every
// thread behind a barrier after which the row state is no longer read.
template <typename T, bool ALIGNED, int NT, typename Release>
__device__ __forceinline__ void finish_row(const Args& a, const T* row, int64_t out, float zy, bool y_ok,
                                           const RowState& st, Finish<NT>& sh, int tid, int bar, Release release) {
  constexpr int E = 16 / (int)sizeof(T);
  constexpr int kCap = Finish<NT>::kCap;
  const int lane = tid & 31, warp = tid >> 5;
  const int64_t V = a.V;
  const int K = a.K;

  // ---- a histogram of the group maxima; every warp finds its range from the blocks' extremes. The
  // maxima of the groups that matter lie within a few tens of the largest; whatever lies below the
  // range (masks) falls into bucket 0 ----
  float blo = 0.f, bsc = 0.f, h = -INFINITY;
  if (K > 0) {
    float l = INFINITY;
    for (int i = lane; i < a.n_blocks; i += 32) {
      h = fmaxf(h, st.part[i].w);
      l = fminf(l, st.lo[i]);
    }
    h = warp_max_f32(h);
    l = -warp_max_f32(-l);
    blo = fmaxf(l, h - 128.f);
    bsc = h > blo ? (kBuckets - 0.5f) / (h - blo) : 0.f;
    // four maxima a load (where their number is no multiple of four, -inf stands behind them)
    const float4* g4 = reinterpret_cast<const float4*>(st.gmax);
#pragma unroll 2
    for (int g = tid; g < (a.n_groups + 3) / 4; g += NT) {
      const float4 z = g4[g];
      atomicAdd(&sh.hist[bucket_of(z.x, blo, bsc)], 1);
      atomicAdd(&sh.hist[bucket_of(z.y, blo, bsc)], 1);
      atomicAdd(&sh.hist[bucket_of(z.z, blo, bsc)], 1);
      atomicAdd(&sh.hist[bucket_of(z.w, blo, bsc)], 1);
    }
  }
  named_bar_sync(bar, NT);
  if (warp == 0) {
    // ---- the row's log-sum-exp, entropy and target ----
    Part r{-INFINITY, 0.f, 0.f};
    for (int i = lane; i < a.n_blocks; i += 32) r = part_join(r, Part{st.part[i].x, st.part[i].y, st.part[i].z});
    r = warp_part<true>(r);
    if (lane == 0) {
      // no distribution: a NaN or +inf logit, or no mass at all
      const bool ok = fabsf(r.m) < INFINITY && r.s > 0.f && r.s < INFINITY;
      const float nan = __int_as_float(0x7fc00000);
      const float l2 = ok ? log2f(r.s) : nan;
      sh.lse_m = r.m;
      sh.lse_l = l2;
      if (a.logp) a.logp[out] = y_ok && ok ? logp_of(zy, a.c, r.m, l2) : nan;
      if (a.entropy) a.entropy[out] = ok ? (l2 - r.q / r.s) * kLn2 : nan;
    }
  }
  if (warp == (NT > 32 ? 1 : 0) && K > 0) {
    // ---- the bucket that the K-th largest group maximum falls into. Lane l counts buckets
    // [8 (31 - l), 8 (31 - l) + 8): lanes in descending bucket order ----
    constexpr int PB = kBuckets / 32;
    int own = 0;
#pragma unroll
    for (int i = 0; i < PB; ++i) own += sh.hist[PB * (31 - lane) + i];
    int pre = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, pre, o);
      if (lane >= o) pre += y;
    }
    const unsigned reach = __ballot_sync(0xffffffffu, pre >= K);
    if (reach == 0) {
      if (lane == 0) sh.bucket = -1;  // fewer groups than K: every element is a candidate
    } else if (lane == __ffs(reach) - 1) {
      int n = pre - own, k = PB * (31 - lane) + PB - 1;
      while ((n += sh.hist[k]) < K) --k;
      sh.bucket = k;
    }
  }
  named_bar_sync(bar, NT);
  const float m = sh.lse_m, l2 = sh.lse_l;
  if (K == 0 || l2 != l2) {
    release();
    if (K > 0)
      for (int i = tid; i < K; i += NT) {
        a.top_idx[out * a.ld_top + i] = -1;
        if (a.top_logp) a.top_logp[out * a.ld_top + i] = l2;
      }
    return;
  }

  // ---- the groups that reach the bucket, and the smallest of their maxima: at least K elements of
  // theirs are no smaller, and no element outside them is as large ----
  const int bmin = sh.bucket;
  // the bucket's lower edge, a little lower against the rounding of bucket_of
  const float edge = bmin > 0 ? blo + ((float)bmin - 0.02f) / bsc : -INFINITY;
  float zl = INFINITY;
  {
    const float4* g4 = reinterpret_cast<const float4*>(st.gmax);
#pragma unroll 2
    for (int g = tid; g < (a.n_groups + 3) / 4; g += NT) {
      const float4 v = g4[g];
      const float z[4] = {v.x, v.y, v.z, v.w};
      if (fmaxf(fmaxf(z[0], z[1]), fmaxf(z[2], z[3])) >= edge) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (z[i] >= edge) {
            zl = fminf(zl, z[i]);
            const int at = atomicAdd(&sh.n_list, 1);
            if (at < kListCap) sh.list[at] = (uint16_t)(4 * g + i);
          }
      }
    }
  }
  zl = -warp_max_f32(-zl);
  if (lane == 0) atomicMin(&sh.zmin, order_of(zl));
  named_bar_sync(bar, NT);
  const bool listed = sh.n_list <= kListCap;
  const uint32_t n_list = listed ? (uint32_t)sh.n_list : (uint32_t)a.n_groups;
  const float zthr = bmin < 0 ? -INFINITY : of_order(sh.zmin);
  release();

  // ---- the listed groups read again (without a list: all of them), a vector at a time: every
  // element at or above the bound is a candidate ----
  const uint32_t vpg = a.by_vec ? 1u : (uint32_t)kTileVecs * (uint32_t)a.fold;
  const uint32_t n_vec = n_list * vpg;  // at most the row's vectors and a block
  auto vec_at = [&](uint32_t i) -> int64_t {
    uint32_t li = i, k = 0;
    if (!a.by_vec) {
      li = a.fold == 1 ? i / kTileVecs : i / vpg;
      k = i - li * vpg;
    }
    const uint32_t g = listed ? sh.list[li] : li;
    if (a.by_vec) return (int64_t)g;
    return ((int64_t)(g >> 5) * a.fold + k / kTileVecs) * (32 * kTileVecs) + ((k >> 2) & 1u) * 128 + (g & 31u) * 4 + (k & 3u);
  };
  unsigned long long floor_key = 0ull;  // K candidates at least as good are in the buffer
  auto offer = [&](int64_t e, float z) {
    const unsigned long long key = make_key(z, (uint32_t)e);
    if (key > floor_key) {
      const int at = atomicAdd(&sh.n_cand, 1);
      if (at < kCap) sh.cand[at] = key;
    }
  };
  // first all at once, kBatch vectors a thread in flight; the buffer holds their candidates but for
  // rows full of ties or masks. Thread i takes vector i % 8 of its groups' tiles.
  constexpr int kBatch = 4;
  static_assert(kTileVecs == 8 && NT % kTileVecs == 0, "vectors by threads");
  const uint32_t n_unit = a.by_vec ? n_list : n_list * (uint32_t)a.fold;
  const uint32_t step = a.by_vec ? NT : NT / kTileVecs, k_at = ((tid >> 2) & 1u) * 128u + (tid & 3u);
  for (uint32_t u0 = a.by_vec ? tid : tid / kTileVecs; u0 < n_unit; u0 += step * kBatch) {
    uint4 x[kBatch];
    uint32_t j[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const uint32_t u = u0 + i * step, li = a.fold == 1 ? u : u / (uint32_t)a.fold;
      const uint32_t ninf = sizeof(T) == 2 ? 0xFF80FF80u : 0xFF800000u;
      x[i] = make_uint4(ninf, ninf, ninf, ninf);
      j[i] = INT32_MAX;  // a vector past every row
      if (u < n_unit) {
        const uint32_t g = listed ? sh.list[li] : li;
        j[i] = g;
        if (!a.by_vec) j[i] = ((g >> 5) * (uint32_t)a.fold + (u - li * (uint32_t)a.fold)) * (32u * kTileVecs) + (g & 31u) * 4u + k_at;
        x[i] = load_vec<T, ALIGNED>(row, j[i], V);
      }
    }
    uint32_t hit = 0;
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      float z[E];
      vec_floats<T>(x[i], z);
      if (vec_max<T>(x[i]) >= zthr) {
#pragma unroll
        for (int k = 0; k < E; ++k) hit |= (z[k] >= zthr ? 1u : 0u) << (i * E + k);
      }
    }
    for (; hit; hit &= hit - 1) {
      const uint32_t b = (uint32_t)__ffs(hit) - 1u, i = b / E;
      const int64_t e = (int64_t)(i & 2u ? (i & 1u ? j[3] : j[2]) : (i & 1u ? j[1] : j[0])) * E + b % E;
      if (e < V) offer(e, elem_f32(row + e));
    }
    if (*static_cast<volatile int*>(&sh.n_cand) > kCap) break;  // it only grows: the rounds below start over
  }
  named_bar_sync(bar, NT);
  int n = sh.n_cand;
  if (n > kCap) {
    // again in rounds of half vectors, keeping the K best whenever the next round might not fit
    named_bar_sync(bar, NT);
    if (tid == 0) sh.n_cand = 0;
    named_bar_sync(bar, NT);
    constexpr uint32_t kParts = E / 4;
    for (uint32_t u0 = 0; u0 < n_vec * kParts; u0 += NT) {
      const uint32_t u = u0 + tid;
      if (u < n_vec * kParts) {
        const int64_t e0 = vec_at(u / kParts) * E + (u % kParts) * 4;
        for (int64_t e = e0; e < e0 + 4 && e < V; ++e) {
          const float z = elem_f32(row + e);
          if (z >= zthr) offer(e, z);
        }
      }
      named_bar_sync(bar, NT);
      n = sh.n_cand;
      if (n > kCap - NT * 4) {
        sort_candidates<NT>(sh.cand, n, tid, bar);
        floor_key = sh.cand[K - 1];
        if (tid == 0) sh.n_cand = K;
      }
      named_bar_sync(bar, NT);
    }
    n = sh.n_cand;
  }

  // ---- rank the candidates and write the K best ----
  auto write = [&](int r, unsigned long long key) {
    a.top_idx[out * a.ld_top + r] = (int32_t)key_idx(key);
    if (a.top_logp) a.top_logp[out * a.ld_top + r] = logp_of(key_logit(key), a.c, m, l2);
  };
  if (n <= NT) {  // each against all
    if (tid < n) {
      const unsigned long long key = sh.cand[tid];
      int r = 0;
#pragma unroll 8
      for (int j = 0; j < n; ++j) r += sh.cand[j] > key;
      if (r < K) write(r, key);
    }
    return;
  }
  // into buckets by their logits (bucket 255 first), then each against those of its bucket. (Sorting a
  // row's 300 candidates for K = 256 took twice the time of reading the row, 17,000 cycles.)
  const float clo = fmaxf(zthr, h - 128.f), csc = h > clo ? (kBuckets - 0.5f) / (h - clo) : 0.f;
  auto bucket = [&](unsigned long long key) { return bucket_of(key_logit(key), clo, csc); };
  for (int i = tid; i < kBuckets; i += NT) sh.hist[i] = 0;
  named_bar_sync(bar, NT);
  for (int i = tid; i < n; i += NT) atomicAdd(&sh.hist[bucket(sh.cand[i])], 1);
  named_bar_sync(bar, NT);
  if (warp == 0) {  // each bucket's first place
    constexpr int PB = kBuckets / 32;
    int c[PB], own = 0;
#pragma unroll
    for (int i = 0; i < PB; ++i) own += c[i] = sh.hist[PB * (31 - lane) + i];
    int pre = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, pre, o);
      if (lane >= o) pre += y;
    }
    pre -= own;
#pragma unroll
    for (int i = PB - 1; i >= 0; --i) {
      sh.hist[PB * (31 - lane) + i] = pre;
      pre += c[i];
    }
  }
  named_bar_sync(bar, NT);
  static_assert(kCap <= 65536, "16-bit places");
  for (int i = tid; i < n; i += NT) sh.place[atomicAdd(&sh.hist[bucket(sh.cand[i])], 1)] = (uint16_t)i;
  named_bar_sync(bar, NT);
  for (int i = tid; i < n; i += NT) {
    const unsigned long long key = sh.cand[i];
    const int b = bucket(key), first = b == kBuckets - 1 ? 0 : sh.hist[b + 1], end = sh.hist[b];
    if (first >= K) continue;
    int r = first;
    for (int j = first; j < end; ++j) r += sh.cand[sh.place[j]] > key;
    if (r < K) write(r, key);
  }
}

// ------------------------------------------------------------------------------------------
// Few or short rows: one CTA per row. SPLIT: a cluster of CTAs shares the row's reading; the rest is
// the work of its first CTA, in whose shared memory the others leave their results.
// ------------------------------------------------------------------------------------------
constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCtas = 16;  // CTAs that may share a row

struct RowShared {
  uint8_t ring[kWarps][2][kSlotBytes];  // 128-byte aligned: the first member
  Finish<kThreads> fin;
  alignas(16) float gmax[kMaxGroups];
  float4 part[kMaxBlocks];
  float lo[kMaxBlocks];
  uint64_t full[kWarps][2];  // the tile in the slot has landed
  int abort;
};

template <typename T, bool ALIGNED, bool SPLIT>
__global__ void __launch_bounds__(kThreads, 2) row_kernel(Args a) {
  extern __shared__ __align__(128) uint8_t smem_raw[];
  RowShared& sh = *reinterpret_cast<RowShared*>(smem_raw);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int n_cta = SPLIT ? a.n_cta : 1, rank = SPLIT ? (int)cluster_ctarank() : 0;
  const int64_t row_i = SPLIT ? blockIdx.x / n_cta : blockIdx.x;
  const int64_t V = a.V;
  const T* row = static_cast<const T*>(a.logits) + row_i * a.ld;
  const int off = ALIGNED ? 0 : row_off(row);
  const int64_t out = a.tok_src ? a.tok_src[row_i] : row_i;
  if (out < 0) return;  // a padding row
  if (a.mask && a.mask[out] == 0) {
    if (rank == 0) write_none(a, out, tid, kThreads, 0.f, -INFINITY);
    return;
  }

  // this warp's blocks, tile by tile, two tiles in flight
  const int n_warps = n_cta * kWarps;
  volatile int* s_abort = &sh.abort;
  if (tid == 0) sh.abort = 0;
  if (lane == 0) {
    mbar_init(&sh.full[warp][0], 1);
    mbar_init(&sh.full[warp][1], 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  __syncwarp();
  int b = rank * kWarps + warp, f = 0;    // the tile to reduce: block b, its f-th
  int fb = b, ff = 0, slot = 0, fslot = 0;  // the tile to fetch, and the slots of both
  uint32_t ph = 0;
  auto next_tile = [&](int& nb, int& nf) {
    if (++nf == a.fold || nb * a.fold + nf >= a.n_tiles) {
      nf = 0;
      nb += n_warps;
    }
  };
  auto fetch = [&] {
    if (fb >= a.n_blocks) return;
    fetch_tile<T>(sh.ring[warp][fslot], row, off, fb * a.fold + ff, a.n_tiles, V, lane, &sh.full[warp][fslot]);
    fslot ^= 1;
    next_tile(fb, ff);
  };
  fetch();
  fetch();
  finish_reset(sh.fin, tid);
  if (a.by_vec && tid < 3 && a.n_groups + tid < kMaxGroups) sh.gmax[a.n_groups + tid] = -INFINITY;
  int32_t y = -1;
  if (a.logp) y = a.target[out];
  const bool y_ok = y >= 0 && (int64_t)y < V;
  const float zy = y_ok && rank == 0 && tid == 0 ? elem_f32(row + y) : 0.f;
  if (SPLIT)
    cluster_sync_all();  // the first CTA runs: its shared memory may be written
  else
    __syncthreads();
  auto put = [&](float* dst, float v) {
    if (SPLIT)
      st_dsmem_f32(mapa_u32(smem_u32(dst), 0u), v);
    else
      *dst = v;
  };
  const LaneOffsets lo4(lane);
  Part p{-INFINITY, 0.f, 0.f};
  float gm = -INFINITY, lo = INFINITY;
  while (b < a.n_blocks) {
    if (__all_sync(0xffffffffu, mbar_wait_bounded(&sh.full[warp][slot], (ph >> slot) & 1u, s_abort))) ph ^= 1u << slot;
    uint4 x[kTileVecs];
    read_tile<T, ALIGNED>(smem_u32(sh.ring[warp][slot]), off, lo4, x);
    __syncwarp();  // every lane has read the slot
    fetch();
    slot ^= 1;
    const int tile = b * a.fold + f;
    const bool last = f + 1 == a.fold || tile + 1 == a.n_tiles;  // of its block
    const float lm = tile_lane_max<T>(x);
    gm = f == 0 ? lm : max_nan(gm, lm);
    if (a.by_vec && a.K > 0) {
#pragma unroll
      for (int u = 0; u < kTileVecs; ++u) {
        const int g = tile * (32 * kTileVecs) + tile_vec(lane, u);
        if (g < a.n_groups) {
          const float vm = vec_max<T>(x[u]);
          put(&sh.gmax[g], vm);
          if (vm > -INFINITY) lo = fminf(lo, vm);
        }
      }
    }
    const Part tp = tile_part<T, true>(x, warp_max_nan(lm), a.c);
    p = f == 0 ? tp : part_join(p, tp);
    if (last) {
      if (!a.by_vec) {
        put(&sh.gmax[b * 32 + lane], gm);
        lo = gm > -INFINITY ? gm : INFINITY;
      }
      const float bh = warp_max_f32(gm), bl = -warp_max_f32(-lo);
      if (lane == 0) {
        put(&sh.part[b].x, p.m);
        put(&sh.part[b].y, *s_abort ? __int_as_float(0x7fc00000) : p.s);  // a wait gave up: no result
        put(&sh.part[b].z, p.q);
        put(&sh.part[b].w, bh);
        put(&sh.lo[b], bl);
      }
      lo = INFINITY;
    }
    next_tile(b, f);
  }
  // a wait gave up: let the copies still in flight land before the CTA's memory goes away (bounded; a
  // slot without a copy runs into the limit)
  if (*s_abort && lane == 0)
    for (int i = 0; i < 2; ++i) {
      const uint64_t t0 = global_timer_ns();
      while (!mbar_try_wait(&sh.full[warp][i], (ph >> i) & 1u) && global_timer_ns() - t0 < 1000000000ull) {}
    }
  if (SPLIT) {
    cluster_sync_all();
    if (rank != 0) return;
  } else {
    __syncthreads();
  }
  const RowState st{sh.part, sh.lo, sh.gmax};
  finish_row<T, ALIGNED, kThreads>(a, row, out, zy, y_ok, st, sh.fin, tid, 1, [] {});
}

template <typename T, bool ALIGNED, bool SPLIT>
int launch_row(const Args& a, cudaStream_t st) {
  auto kern = row_kernel<T, ALIGNED, SPLIT>;
  int dev = 0;
  GRPO_CUDA_TRY(cudaGetDevice(&dev));
  {
    static std::mutex mu;
    static bool ready[64] = {};
    std::lock_guard<std::mutex> lock(mu);
    if (dev < 0 || dev >= 64 || !ready[dev]) {
      GRPO_CUDA_TRY(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(RowShared)));
      if (SPLIT) GRPO_CUDA_TRY(cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1));
      if (dev >= 0 && dev < 64) ready[dev] = true;
    }
  }
  if (!SPLIT) {
    kern<<<(unsigned)a.T, kThreads, sizeof(RowShared), st>>>(a);
    GRPO_CUDA_TRY(cudaGetLastError());
    return GRPO_OK;
  }
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = a.n_cta;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.gridDim = dim3((unsigned)(a.T * a.n_cta), 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = sizeof(RowShared);
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  GRPO_CUDA_TRY(cudaLaunchKernelEx(&cfg, kern, a));
  return GRPO_OK;
}

// ------------------------------------------------------------------------------------------
// Many long rows: a persistent CTA per SM. Warps 0..11 stream: the tiles of the CTA's rows, in row
// order, go round-robin over them (a block is one tile here). Each warp has two slots of shared memory:
// bulk copies fetch its next two tiles while it reduces this one; the tiles of a row that is not 16-byte
// aligned are shifted as they are read from their slot. A row's results go to one of a.slots row states. Every streaming warp passes every row, also where
// none of the tiles is its own: before it enters a row it waits until the row's state was handed back
// (mbarrier freed), and it arrives on the state's other mbarrier (done) when it leaves it. So rows
// are done in order, and both barriers' phases follow the rows one by one: a phase bit is never a
// whole round off as long as there are at least as many states as finishing groups. The other warps
// finish rows, kFinishGroups groups in turn, and hand the state back. So the loads never wait for a
// row's end. Masked and padding rows are skipped by every warp alike.
// ------------------------------------------------------------------------------------------
constexpr int kStreamWarps = 12;
constexpr int kFinishThreads = 128;
constexpr int kFinishGroups = 2;
constexpr int kStreamThreads = kStreamWarps * 32 + kFinishGroups * kFinishThreads;
constexpr int kMinSlots = 3, kMaxSlots = 8;
static_assert(kFinishGroups <= kMinSlots, "the phases' order");
struct StreamShared {
  Finish<kFinishThreads> fin[kFinishGroups];
  uint64_t full[kStreamWarps][2];  // the tile in the slot has landed
  uint64_t done[kMaxSlots];        // every streaming warp has left the row
  uint64_t freed[kMaxSlots];       // the row state may be rewritten
  int abort;
};

// Floats of a row state: five per block, then the group maxima.
__host__ __device__ constexpr int state_floats(int n_blocks) { return 4 * n_blocks + (n_blocks + 3) / 4 * 4 + 32 * n_blocks; }

__device__ __forceinline__ RowState row_state(float* base, int slot, int n_blocks) {
  float* p = base + (size_t)slot * state_floats(n_blocks);
  return {reinterpret_cast<float4*>(p), p + 4 * n_blocks, p + 4 * n_blocks + (n_blocks + 3) / 4 * 4};
}

__host__ __device__ constexpr size_t stream_head_bytes() { return (sizeof(StreamShared) + 127) / 128 * 128; }

__host__ __device__ constexpr size_t stream_state_bytes(int slots, int n_blocks) {
  return ((size_t)slots * state_floats(n_blocks) * 4 + 127) / 128 * 128;
}

// A warp's walk over its tiles of the CTA's read rows, with the next row's index and mask loads in
// flight. row = T at the end.
struct TileWalk {
  const Args& a;
  int32_t row, next;
  bool next_read;
  int n;  // read rows before this one
  int t;  // tile of the row
  __device__ TileWalk(const Args& args, int warp) : a(args), row(-1), n(-1), t(warp) {
    next = (int32_t)blockIdx.x;
    look();
    step();
    settle();
  }
  __device__ __forceinline__ void look() {
    next_read = false;
    if (next < a.T) {
      const int64_t src = a.tok_src ? a.tok_src[next] : next;
      next_read = src >= 0 && (!a.mask || a.mask[src] != 0);
    }
  }
  __device__ __forceinline__ int32_t after(int32_t r) const {
    const int64_t s = (int64_t)r + gridDim.x;
    return s < a.T ? (int32_t)s : (int32_t)a.T;
  }
  __device__ __forceinline__ void step() {  // to the next read row
    while (next < a.T && !next_read) {
      next = after(next);
      look();
    }
    row = next;
    ++n;
    if (next < a.T) {
      next = after(next);
      look();
    }
  }
  __device__ __forceinline__ void settle() {
    while (t >= a.n_tiles && row < a.T) {
      t -= a.n_tiles;
      step();
    }
  }
};

template <typename T, bool ALIGNED>
__global__ void __launch_bounds__(kStreamThreads, 1) stream_kernel(Args a) {
  extern __shared__ __align__(128) uint8_t smem_raw[];
  StreamShared& sh = *reinterpret_cast<StreamShared*>(smem_raw);
  float* states = reinterpret_cast<float*>(smem_raw + stream_head_bytes());  // [slots] row states
  uint8_t* ring = smem_raw + stream_head_bytes() + stream_state_bytes(a.slots, a.n_blocks);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t V = a.V;
  volatile int* s_abort = &sh.abort;
  if (tid == 0) {
    for (int w = 0; w < kStreamWarps; ++w)
      for (int s = 0; s < 2; ++s) mbar_init(&sh.full[w][s], 1);
    for (int s = 0; s < kMaxSlots; ++s) {
      mbar_init(&sh.done[s], kStreamWarps);
      mbar_init(&sh.freed[s], 1);
    }
    sh.abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  __syncthreads();

  if (warp < kStreamWarps) {
    TileWalk walk(a, warp);  // the tile to fetch next
    // its row, the row's offset, and the address of the aligned vectors that hold it
    const T* row = nullptr;
    const uint8_t* src = nullptr;
    int off = 0;
    auto locate = [&] {
      if (walk.row >= a.T) return;
      row = static_cast<const T*>(a.logits) + (int64_t)walk.row * a.ld;
      off = ALIGNED ? 0 : row_off(row);
      src = reinterpret_cast<const uint8_t*>(row) + (int64_t)walk.t * kTileBytes - off;
    };
    locate();
    uint8_t* mine = ring + (size_t)warp * 2 * kSlotBytes;
    const uint32_t mine32 = smem_u32(mine);
    const LaneOffsets lo4(lane);
    // a tile in flight: its number in the row (-1: none), the read row, the row's offset
    struct Flight {
      int t, n, off;
    };
    auto fetch = [&](int s) -> Flight {
      if (walk.row >= a.T) return {-1, walk.n, 0};
      const Flight f{walk.t, walk.n, off};
      uint64_t* bar = &sh.full[warp][s];
      uint8_t* slot = mine + s * kSlotBytes;
      if ((f.t == 0 && off) || f.t >= a.n_tiles - 2) {
        fetch_tile<T>(slot, row, off, f.t, a.n_tiles, V, lane, bar);
      } else if (lane == 0) {
        const uint32_t bytes = kTileBytes + (off ? 16u : 0u);
        mbar_arrive_expect_tx(bar, bytes);
        bulk_g2s(slot, src, bytes, bar);
      }
      walk.t += kStreamWarps;
      src += kStreamWarps * kTileBytes;
      if (walk.t >= a.n_tiles) {
        walk.settle();
        locate();
      }
      return f;
    };
    bool ok = true;
    int at = 0, at_slot = 0, at_round = 0;  // the read row this warp is in, its state, rows that used it before
    RowState st = row_state(states, 0, a.n_blocks);
    auto pass_to = [&](int n, bool end) {  // on to read row n (end: there is none)
      while (at < n && ok) {
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.done[at_slot]);
        ++at;
        if (++at_slot == a.slots) {
          at_slot = 0;
          ++at_round;
        }
        if (at_round > 0 && !(end && at == n))
          ok = __all_sync(0xffffffffu, mbar_wait_bounded(&sh.freed[at_slot], (uint32_t)(at_round - 1) & 1u, s_abort));
      }
      if (__any_sync(0xffffffffu, *s_abort)) ok = false;
      st = row_state(states, at_slot, a.n_blocks);
    };
    Flight cur = fetch(0), nxt = fetch(1);
    __syncwarp();
    uint32_t ph = 0;  // bit s: the phase of slot s
    int s = 0;
    pass_to(cur.n, cur.t < 0);
    while (cur.t >= 0 && ok) {
      // (a wait that gives up is seen in pass_to: the rows from here on are marked as broken)
      if (mbar_wait_bounded(&sh.full[warp][s], (ph >> s) & 1u, s_abort)) ph ^= 1u << s;
      uint4 x[kTileVecs];
      read_tile<T, ALIGNED>(mine32 + s * kSlotBytes, cur.off, lo4, x);
      __syncwarp();  // every lane has read the slot
      const Flight after = fetch(s);
      const float lm = tile_lane_max<T>(x);
      const float hi = warp_max_nan(lm);
      const Part p = tile_part<T, true>(x, hi, a.c);
      const float lo = -warp_max_f32(lm > -INFINITY ? -lm : -INFINITY);
      st.gmax[cur.t * 32 + lane] = lm;
      if (lane == 0) {
        st.part[cur.t] = make_float4(p.m, p.s, p.q, hi);
        st.lo[cur.t] = lo;
      }
      cur = nxt;
      nxt = after;
      s ^= 1;
      if (cur.n != at) pass_to(cur.n, cur.t < 0);
    }
    // a wait gave up: let the copies still in flight land before the CTA's memory goes away
    // (bounded; a slot without a copy runs into the limit)
    if (*s_abort && lane == 0)
      for (int i = 0; i < 2; ++i) {
        const uint64_t t0 = global_timer_ns();
        while (!mbar_try_wait(&sh.full[warp][i], (ph >> i) & 1u) && global_timer_ns() - t0 < 1000000000ull) {}
      }
  } else {
    const int group = (warp - kStreamWarps) / (kFinishThreads / 32);
    const int gt = tid - kStreamWarps * 32 - group * kFinishThreads;
    const int bar = 1 + group;
    Finish<kFinishThreads>& fin = sh.fin[group];
    // the row to finish next, its target and the target's logit loaded ahead of it
    int n = 0, seen = 0;  // read rows and rows so far
    int64_t r = blockIdx.x;
    struct Ahead {
      int64_t row, out;
      int32_t y;
      float zy;
      int k;
    };
    auto look = [&]() -> Ahead {
      for (; r < a.T; r += gridDim.x, ++seen) {
        const int64_t out = a.tok_src ? a.tok_src[r] : r;
        if (out < 0) continue;
        if (a.mask && a.mask[out] == 0) {
          if (seen % kFinishGroups == group) write_none(a, out, gt, kFinishThreads, 0.f, -INFINITY);
          continue;
        }
        const int k = n++;
        if (k % kFinishGroups != group) continue;
        Ahead h{r, out, -1, 0.f, k};
        if (a.logp && gt == 0) {
          h.y = a.target[out];
          if (h.y >= 0 && (int64_t)h.y < V) h.zy = elem_f32(static_cast<const T*>(a.logits) + r * a.ld + h.y);
        }
        r += gridDim.x;
        ++seen;
        return h;
      }
      return Ahead{a.T, 0, -1, 0.f, 0};
    };
    Ahead cur = look();
    while (cur.row < a.T) {
      finish_reset(fin, gt);
      const int slot = cur.k % a.slots;
      if (gt < 32) {  // the group's first warp waits, the others at the barrier
        const bool ok = mbar_wait_bounded(&sh.done[slot], (uint32_t)(cur.k / a.slots) & 1u, s_abort);
        if (gt == 0) fin.broken = !ok || *s_abort;
      }
      const Ahead nxt = look();
      named_bar_sync(bar, kFinishThreads);
      const T* row = static_cast<const T*>(a.logits) + cur.row * a.ld;
      if (fin.broken) {  // the pipeline broke: this row has no result
        write_none(a, cur.out, gt, kFinishThreads, __int_as_float(0x7fc00000), __int_as_float(0x7fc00000));
      } else {
        const RowState st = row_state(states, slot, a.n_blocks);
        finish_row<T, ALIGNED, kFinishThreads>(a, row, cur.out, cur.zy,
                                               cur.y >= 0 && (int64_t)cur.y < V, st, fin, gt, bar, [&] {
                                                 if (gt == 0) mbar_arrive(&sh.freed[slot]);
                                               });
      }
      named_bar_sync(bar, kFinishThreads);  // the scratch is rewritten for the group's next row
      cur = nxt;
    }
  }
}

// Shared memory of the streaming kernel.
size_t stream_smem(const Args& a) {
  return stream_head_bytes() + stream_state_bytes(a.slots, a.n_blocks) +
         (size_t)kStreamWarps * 2 * kSlotBytes;
}

template <typename T, bool ALIGNED>
int launch_stream(const Args& a, cudaStream_t st) {
  auto kern = stream_kernel<T, ALIGNED>;
  const size_t smem = stream_smem(a);
  int dev = 0;
  GRPO_CUDA_TRY(cudaGetDevice(&dev));
  {
    static std::mutex mu;
    static size_t limit[64] = {};
    std::lock_guard<std::mutex> lock(mu);
    if (dev < 0 || dev >= 64 || smem > limit[dev]) {
      GRPO_CUDA_TRY(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem));
      if (dev >= 0 && dev < 64) limit[dev] = smem;
    }
  }
  kern<<<(unsigned)std::min<int64_t>(a.T, sm_count()), kStreamThreads, smem, st>>>(a);
  GRPO_CUDA_TRY(cudaGetLastError());
  return GRPO_OK;
}

template <typename T>
int dispatch(Args& a, bool aligned, cudaStream_t st) {
  // Up to three rows per SM: row_kernel, with few of them a cluster sharing each row's reading, as many
  // CTAs as the SMs hold at once and as have a block per warp. Short rows (under 16 tiles) and rows past
  // the streaming kernel's states: row_kernel. All others: stream_kernel. K = 20, row_kernel and
  // stream_kernel: 229 x 50264 bf16 12.4 and 14.4 us, 300 x 151936 21.0 and 22.8, 460 x 50264 22.4 and 20.6,
  // 2048 x 151936 128 and 106, 8192 x 32776 228 and 165. 64 x 151936 fp32 by four CTAs a row 15.6 us, by one
  // 21.9.
  const int64_t sms = sm_count();
  if (a.T > 3 * sms && a.fold == 1 && !a.by_vec) {
    a.slots = kMaxSlots;
    while (a.slots > kMinSlots && stream_smem(a) > max_smem_optin()) --a.slots;
    if (stream_smem(a) <= max_smem_optin())
      return aligned ? launch_stream<T, true>(a, st) : launch_stream<T, false>(a, st);
  }
  a.n_cta = 1;
  while (a.n_cta < kMaxCtas && 2 * a.n_cta * a.T <= 2 * sms && a.n_cta * kWarps < a.n_blocks) a.n_cta *= 2;
  if (a.n_cta > 1) return aligned ? launch_row<T, true, true>(a, st) : launch_row<T, false, true>(a, st);
  return aligned ? launch_row<T, true, false>(a, st) : launch_row<T, false, false>(a, st);
}

}  // namespace score
}  // namespace grpo

using namespace grpo;

extern "C" GRPO_API int grpo_token_topk_logprobs(const void* logits, int32_t dtype, int64_t T, int64_t V, int64_t ld,
                                                 const int64_t* tok_src, const int32_t* target, const uint8_t* mask,
                                                 float temperature, int32_t K, float* logp_tok, float* entropy_tok,
                                                 int32_t* top_idx, float* top_logp, int64_t ld_top, void* stream) {
  if (dtype != GRPO_DTYPE_F32 && dtype != GRPO_DTYPE_BF16) return GRPO_ERR_UNSUPPORTED;
  if (T < 0 || V < 1 || ld < V || V > (int64_t)INT32_MAX || T > (int64_t)INT32_MAX) return GRPO_ERR_INVALID;
  if (K < 0 || K > GRPO_TOPK_MAX || K > V) return GRPO_ERR_INVALID;
  if (!(temperature > 0.f) || !std::isfinite(temperature)) return GRPO_ERR_INVALID;
  const double cd = 1.4426950408889634 / (double)temperature;
  const float c = (float)cd;
  if (!(c < 0x1p126f) || c < 1.1754944e-38f) return GRPO_ERR_INVALID;  // (its powers of two are float32 numbers)
  if (K > 0 && ld_top < K) return GRPO_ERR_INVALID;
  if (T == 0) return GRPO_OK;
  if (!logits || (logp_tok && !target) || (K > 0 && !top_idx)) return GRPO_ERR_INVALID;
  const size_t es = dtype == GRPO_DTYPE_F32 ? 4 : 2;
  if (reinterpret_cast<uintptr_t>(logits) % es) return GRPO_ERR_INVALID;

  score::Args a{};
  a.logits = logits;
  a.T = T;
  a.V = V;
  a.ld = ld;
  a.tok_src = tok_src;
  a.target = target;
  a.mask = mask;
  a.c = c;
  a.K = K;
  a.logp = logp_tok;
  a.entropy = entropy_tok;
  a.top_idx = top_idx;
  a.top_logp = top_logp;
  a.ld_top = ld_top;
  const int64_t vecs = (V * (int64_t)es + 15) / 16;
  const int64_t tiles = (vecs + 32 * kTileVecs - 1) / (32 * kTileVecs);
  // every vector a group where they are few: a short row then has groups enough for a tight bound
  a.by_vec = tiles < 16;  // at most 16 * 256 vectors
  a.fold = (int32_t)((tiles + score::kMaxBlocks - 1) / score::kMaxBlocks);
  a.n_tiles = (int32_t)tiles;
  a.n_blocks = (int32_t)((tiles + a.fold - 1) / a.fold);
  a.n_groups = a.by_vec ? (int32_t)vecs : a.n_blocks * 32;
  const bool aligned = (reinterpret_cast<uintptr_t>(logits) & 15u) == 0 && (ld * es) % 16 == 0;
  const cudaStream_t st = as_stream(stream);
  return dtype == GRPO_DTYPE_BF16 ? score::dispatch<__nv_bfloat16>(a, aligned, st)
                                  : score::dispatch<float>(a, aligned, st);
}
