// Scoring of logits rows: the log-prob of a given token, the entropy of the row's distribution
// and its K most probable tokens with their log-probs, in one pass over the logits.
//
//   log p_v = z_v/tau - log sum_u exp(z_u/tau),   H = -sum_v p_v log p_v
//
// One CTA takes a row and reads it once from HBM in warp tiles (grpo_vocab.cuh), which gives the
// log-sum-exp and the entropy. For the K largest logits every tile also leaves the maximum of
// each group of elements (a lane's vectors of one tile, or single vectors of a short row). The
// K-th largest group maximum bounds the K-th largest logit from below, as K groups hold an
// element at least that large. A histogram of the group maxima finds that bound (rounded down
// to a bucket), and only the groups that reach it are read again: about K of them, from L2. What
// survives of them is ranked exactly, equal logits by index. Any row is served: where the bound
// lets more than the candidate buffer through (ties, rows with fewer than K finite logits), the
// buffer is cut back to its K best as it fills, which raises the bound.
#include <algorithm>
#include <cmath>
#include <mutex>

#include "grpo_vocab.cuh"

namespace grpo {
namespace score {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxGroups = 5120;     // group maxima kept per row
constexpr int kBuckets = 256;
constexpr int kUnit = 4;             // elements a thread tests per round of the second reading
constexpr int kCap = 2048;           // candidate buffer: K kept + one round's kThreads * kUnit
constexpr int kRankMax = 256;        // candidates ranked by counting; more are sorted

static_assert(GRPO_TOPK_MAX + kThreads * kUnit <= kCap, "a round's candidates fit beside the kept K");
static_assert((kCap & (kCap - 1)) == 0, "the sort takes a power of two");

struct Args {
  const void* logits;
  int64_t V, ld;
  const int64_t* tok_src;
  const int32_t* target;
  const uint8_t* mask;
  float c;  // log2(e) / temperature
  int32_t K;
  float *logp, *entropy;
  int32_t* top_idx;
  float* top_logp;
  int64_t ld_top;
  // the row's cut into tiles and groups (functions of V): `fold` consecutive tiles form a
  // block, a lane's elements of a block a group; `by_vec`: every vector is a group of its own
  int32_t n_blocks, fold, n_groups;
  bool by_vec;
};

struct Shared {
  unsigned long long cand[kCap];
  float gmax[kMaxGroups];
  uint16_t list[kMaxGroups];
  float pm[kMaxGroups / 32], ps[kMaxGroups / 32], pq[kMaxGroups / 32];
  int hist[kBuckets];
  float whi[kWarps], wlo[kWarps];
  float lse_m, lse_l, s_lo, s_scale;
  int bucket, n_list, n_cand;
};

// Descending order of (logit, then ascending index) as one unsigned key; -0 counts as +0.
__device__ __forceinline__ unsigned long long make_key(float z, uint32_t idx) {
  const uint32_t b = __float_as_uint(z + 0.f);
  const uint32_t o = (b & 0x80000000u) ? ~b : (b | 0x80000000u);
  return ((unsigned long long)o << 32) | (uint32_t)~idx;
}
__device__ __forceinline__ uint32_t key_idx(unsigned long long k) { return ~(uint32_t)k; }
__device__ __forceinline__ float key_logit(unsigned long long k) {
  const uint32_t o = (uint32_t)(k >> 32);
  return __uint_as_float((o & 0x80000000u) ? (o & 0x7FFFFFFFu) : ~o);
}

// Bucket of a logit in [0, kBuckets): monotone in z.
__device__ __forceinline__ int bucket_of(float z, float lo, float scale) {
  return min(kBuckets - 1, max(0, __float2int_rd((z - lo) * scale)));
}

// The first n candidates sorted in descending order (bitonic, padded with 0: below every key).
__device__ __forceinline__ void sort_candidates(unsigned long long* k, int n, int tid) {
  int P = 1;
  while (P < n) P <<= 1;
  for (int i = n + tid; i < P; i += kThreads) k[i] = 0ull;
  for (int size = 2; size <= P; size <<= 1)
    for (int stride = size >> 1; stride > 0; stride >>= 1) {
      __syncthreads();
      for (int i = tid; i < P / 2; i += kThreads) {
        const int a = 2 * i - (i & (stride - 1)), b = a + stride;
        const unsigned long long x = k[a], y = k[b];
        if (((a & size) == 0) ? x < y : x > y) {
          k[a] = y;
          k[b] = x;
        }
      }
    }
  __syncthreads();
}

template <typename T, bool ALIGNED>
__global__ void __launch_bounds__(kThreads) topk_kernel(Args a) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  Shared& sh = *reinterpret_cast<Shared*>(smem_raw);
  constexpr int E = 16 / (int)sizeof(T);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t row_i = blockIdx.x;
  const int64_t out = a.tok_src ? a.tok_src[row_i] : row_i;
  if (out < 0) return;  // a padding row
  const int32_t K = a.K;
  if (a.mask && a.mask[out] == 0) {
    if (tid == 0) {
      if (a.logp) a.logp[out] = 0.f;
      if (a.entropy) a.entropy[out] = 0.f;
    }
    for (int i = tid; i < K; i += kThreads) {
      a.top_idx[out * a.ld_top + i] = -1;
      if (a.top_logp) a.top_logp[out * a.ld_top + i] = -INFINITY;
    }
    return;
  }
  const int64_t V = a.V;
  const T* row = static_cast<const T*>(a.logits) + row_i * a.ld;
  if (tid == 0) sh.n_list = sh.n_cand = 0;
  for (int i = tid; i < kBuckets; i += kThreads) sh.hist[i] = 0;

  // ---- one reading: softmax partials and group maxima ----
  float hi = -INFINITY, lo = INFINITY;  // largest and smallest group maximum of this lane
  for (int b = warp; b < a.n_blocks; b += kWarps) {
    Part p{-INFINITY, 0.f, 0.f};
    float gm = -INFINITY;
    for (int f = 0; f < a.fold; ++f) {
      const int64_t tile = (int64_t)b * a.fold + f;
      if (tile * tile_elems<T>() >= V) break;
      uint4 x[kTileVecs];
      load_tile<T, ALIGNED>(row, tile, V, lane, x);
      const float lm = tile_lane_max<T>(x);
      gm = max_nan(gm, lm);
      const Part tp = tile_part<T, true>(x, lm, a.c);
      p = f == 0 ? tp : part_join(p, tp);
      if (a.by_vec && K > 0) {
#pragma unroll
        for (int u = 0; u < kTileVecs; ++u) {
          const int g = (int)tile * (32 * kTileVecs) + u * 32 + lane;
          if (g < a.n_groups) {
            const float vm = vec_max<T>(x[u]);
            sh.gmax[g] = vm;
            lo = fminf(lo, vm);
          }
        }
      }
    }
    hi = fmaxf(hi, gm);
    if (!a.by_vec && b * 32 + lane < a.n_groups) {
      sh.gmax[b * 32 + lane] = gm;
      lo = fminf(lo, gm);
    }
    if (lane == 0) {
      sh.pm[b] = p.m;
      sh.ps[b] = p.s;
      sh.pq[b] = p.q;
    }
  }
  hi = warp_max_f32(hi);
  lo = -warp_max_f32(-lo);
  if (lane == 0) {
    sh.whi[warp] = hi;
    sh.wlo[warp] = lo;
  }
  __syncthreads();

  // ---- the row's log-sum-exp, entropy and target (warp 0); the histogram's range (warp 1) ----
  if (warp == 0) {
    Part p{-INFINITY, 0.f, 0.f};
    for (int b = lane; b < a.n_blocks; b += 32) p = part_join(p, Part{sh.pm[b], sh.ps[b], sh.pq[b]});
    p = warp_part(p);
    if (lane == 0) {
      // no distribution: a NaN or +inf logit, or no mass at all
      const bool ok = fabsf(p.m) < INFINITY && p.s > 0.f && p.s < INFINITY;
      const float nan = __int_as_float(0x7fc00000);
      const float l2 = ok ? log2f(p.s) : nan;
      sh.lse_m = p.m;
      sh.lse_l = l2;
      if (a.logp) {
        const int32_t y = a.target[out];
        const bool in = y >= 0 && (int64_t)y < V;
        a.logp[out] = in && ok ? (fmaf(elem_f32(row + y), a.c, -p.m) - l2) * kLn2 : nan;
      }
      if (a.entropy) a.entropy[out] = ok ? (l2 - p.q / p.s) * kLn2 : nan;
    }
  } else if (warp == 1) {
    float h = lane < kWarps ? sh.whi[lane] : -INFINITY, l = lane < kWarps ? sh.wlo[lane] : INFINITY;
    h = warp_max_f32(h);
    l = -warp_max_f32(-l);
    if (lane == 0) {
      // the maxima of the groups that matter lie within a few tens of the largest; whatever
      // lies below the range (masks) falls into bucket 0
      l = fmaxf(l, h - 128.f);
      sh.s_lo = l;
      sh.s_scale = h > l ? (kBuckets - 0.5f) / (h - l) : 0.f;
    }
  }
  if (K == 0) return;
  __syncthreads();
  const float m = sh.lse_m, l2 = sh.lse_l;
  if (l2 != l2) {
    for (int i = tid; i < K; i += kThreads) {
      a.top_idx[out * a.ld_top + i] = -1;
      if (a.top_logp) a.top_logp[out * a.ld_top + i] = l2;
    }
    return;
  }

  // ---- the bucket that the K-th largest group maximum falls into ----
  const float blo = sh.s_lo, bsc = sh.s_scale;
  for (int g = tid; g < a.n_groups; g += kThreads) atomicAdd(&sh.hist[bucket_of(sh.gmax[g], blo, bsc)], 1);
  __syncthreads();
  if (warp == 0) {
    // lane l counts buckets [8 (31 - l), 8 (31 - l) + 8): lanes in descending bucket order
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
      if (lane == 0) sh.bucket = 0;  // fewer groups than K: every element is a candidate
    } else if (lane == __ffs(reach) - 1) {
      int n = pre - own, b = PB * (31 - lane) + PB - 1;
      while ((n += sh.hist[b]) < K) --b;
      sh.bucket = b;
    }
  }
  __syncthreads();
  const int bmin = sh.bucket;
  for (int g = tid; g < a.n_groups; g += kThreads)
    if (bucket_of(sh.gmax[g], blo, bsc) >= bmin) sh.list[atomicAdd(&sh.n_list, 1)] = (uint16_t)g;
  __syncthreads();

  // ---- the listed groups read again: every element that reaches the bucket is a candidate ----
  const int units_per_vec = E / kUnit;
  const int vecs_per_group = a.by_vec ? 1 : kTileVecs * a.fold;
  const int64_t units = (int64_t)sh.n_list * vecs_per_group * units_per_vec;
  unsigned long long floor_key = 0ull;  // keys of K candidates at least as good are in the buffer
  for (int64_t u0 = 0; u0 < units; u0 += kThreads) {
    const int64_t u = u0 + tid;
    if (u < units) {
      const int part = (int)(u % units_per_vec);
      const int64_t v = u / units_per_vec;
      const int g = sh.list[v / vecs_per_group];
      const int k = (int)(v % vecs_per_group);
      const int64_t j = a.by_vec ? g
                                 : ((int64_t)(g / 32) * a.fold + k / kTileVecs) * (32 * kTileVecs) +
                                       (k % kTileVecs) * 32 + (g & 31);
      const int64_t e0 = j * E + part * kUnit;
#pragma unroll
      for (int i = 0; i < kUnit; ++i) {
        if (e0 + i >= V) break;
        const float z = elem_f32(row + e0 + i);
        if (bucket_of(z, blo, bsc) < bmin) continue;
        const unsigned long long key = make_key(z, (uint32_t)(e0 + i));
        if (key > floor_key) sh.cand[atomicAdd(&sh.n_cand, 1)] = key;
      }
    }
    __syncthreads();
    const int n = sh.n_cand;
    if (n > kCap - kThreads * kUnit) {  // the next round may not fit: keep the K best
      sort_candidates(sh.cand, n, tid);
      floor_key = sh.cand[K - 1];
      if (tid == 0) sh.n_cand = K;
      __syncthreads();
    }
  }

  // ---- rank the candidates and write the K best ----
  const int n = sh.n_cand;
  auto put = [&](int r, unsigned long long key) {
    a.top_idx[out * a.ld_top + r] = (int32_t)key_idx(key);
    if (a.top_logp) a.top_logp[out * a.ld_top + r] = (fmaf(key_logit(key), a.c, -m) - l2) * kLn2;
  };
  if (n <= kRankMax) {
    for (int i = tid; i < n; i += kThreads) {
      const unsigned long long key = sh.cand[i];
      int r = 0;
      for (int j = 0; j < n; ++j) r += sh.cand[j] > key;
      if (r < K) put(r, key);
    }
  } else {
    sort_candidates(sh.cand, n, tid);
    for (int i = tid; i < K; i += kThreads) put(i, sh.cand[i]);
  }
}

template <typename T, bool ALIGNED>
int launch(const Args& a, int64_t T_rows, cudaStream_t st) {
  auto kern = topk_kernel<T, ALIGNED>;
  int dev = 0;
  GRPO_CUDA_TRY(cudaGetDevice(&dev));
  {
    static std::mutex mu;
    static bool ready[64] = {};
    std::lock_guard<std::mutex> lock(mu);
    if (dev < 0 || dev >= 64 || !ready[dev]) {
      GRPO_CUDA_TRY(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(Shared)));
      if (dev >= 0 && dev < 64) ready[dev] = true;
    }
  }
  kern<<<(unsigned)T_rows, kThreads, sizeof(Shared), st>>>(a);
  GRPO_CUDA_TRY(cudaGetLastError());
  return GRPO_OK;
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
  if (!std::isfinite(c) || c < 1.1754944e-38f) return GRPO_ERR_INVALID;
  if (K > 0 && ld_top < K) return GRPO_ERR_INVALID;
  if (T == 0) return GRPO_OK;
  if (!logits || (logp_tok && !target) || (K > 0 && !top_idx)) return GRPO_ERR_INVALID;
  const size_t es = dtype == GRPO_DTYPE_F32 ? 4 : 2;
  if (reinterpret_cast<uintptr_t>(logits) % es) return GRPO_ERR_INVALID;

  score::Args a{};
  a.logits = logits;
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
  // every vector a group where they fit: a short row then has groups enough for a tight bound
  a.by_vec = vecs <= score::kMaxGroups;
  a.fold = a.by_vec ? 1 : (int32_t)((tiles * 32 + score::kMaxGroups - 1) / score::kMaxGroups);
  a.n_blocks = (int32_t)((tiles + a.fold - 1) / a.fold);
  a.n_groups = a.by_vec ? (int32_t)vecs : a.n_blocks * 32;
  const bool aligned = (reinterpret_cast<uintptr_t>(logits) & 15u) == 0 && (ld * es) % 16 == 0;
  const cudaStream_t st = as_stream(stream);
  if (dtype == GRPO_DTYPE_BF16)
    return aligned ? score::launch<__nv_bfloat16, true>(a, T, st) : score::launch<__nv_bfloat16, false>(a, T, st);
  return aligned ? score::launch<float, true>(a, T, st) : score::launch<float, false>(a, T, st);
}
