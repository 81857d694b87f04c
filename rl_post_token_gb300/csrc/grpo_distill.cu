// Distillation of a student's logits rows from a teacher's top tokens, loss and dlogits in one
// call (formulas in grpo_distill.cuh).
//
// One CTA takes a row: it sorts the teacher's list by token, reads the row once for its softmax
// sums (warp tiles, grpo_vocab.cuh; the tail kinds leave the listed tokens out of the tiles' sums
// and add them singly), forms the token's loss with one thread per list entry, and reads the
// row again, from L2, to write dlogits. 304 KB x 152 rows in flight fit L2.
#include <algorithm>
#include <cmath>
#include <mutex>

#include "grpo_distill.cuh"
#include "grpo_vocab.cuh"

namespace grpo {
namespace distill {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxBlocks = 160;  // softmax partials kept per row

struct Args {
  const void* logits;
  int64_t T, V, ld;
  const int64_t* tok_src;
  const int32_t* top_idx;
  const float* top_logp;
  int64_t ld_top;
  int32_t K;
  const uint8_t* mask;
  const float* w_tok;
  float c;      // log2(e) / temperature
  float scale;  // grad_scale / temperature
  void* dlogits;
  int64_t ld_out;
  float* loss_tok;
  grpo_step_acc* acc;
  int32_t n_blocks, fold;  // `fold` consecutive tiles per kept partial (a function of V)
};

struct Shared {
  int32_t sorted[GRPO_TOPK_MAX];  // the listed tokens in ascending order
  float pm[kMaxBlocks], ps[kMaxBlocks];
  double red[2][kWarps];
  int bad, n_listed;
};

// Sum of a value over the block (fixed tree); every thread gets it. Calls alternate `buf`.
__device__ __forceinline__ double block_sum(double v, double* red, int lane, int warp) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (lane == 0) red[warp] = v;
  __syncthreads();
  double s = 0.0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) s += red[w];
  return s;
}

__device__ __forceinline__ float block_max(float v, double* red, int lane, int warp) {
  v = warp_max_f32(v);
  if (lane == 0) red[warp] = (double)v;
  __syncthreads();
  double m = red[0];
#pragma unroll
  for (int w = 1; w < kWarps; ++w) m = fmax(m, red[w]);
  return (float)m;
}

// The elements of this lane's tile vectors that are on the sorted list, as a bit mask (bit
// u E + i: element i of vector u).
template <typename T>
__device__ __forceinline__ uint64_t listed_bits(const int32_t* sorted, int n, int64_t tile, int lane) {
  constexpr int E = 16 / (int)sizeof(T), TE = tile_elems<T>();
  const int64_t e0 = tile * TE;
  int lo = 0, hi = n;
  while (lo < hi) {  // first entry at or after the tile's start
    const int mid = (lo + hi) / 2;
    if ((int64_t)sorted[mid] < e0)
      lo = mid + 1;
    else
      hi = mid;
  }
  uint64_t bits = 0;
  for (; lo < n; ++lo) {
    const int64_t d = (int64_t)sorted[lo] - e0;
    if (d >= TE) break;
    const int j = (int)d / E;  // vector of the tile: lane and u as tile_vec has them
    const int l = (j >> 2) & 31, u = (j >> 7) * 4 + ((j - (l >> 1)) & 3);
    if (l == lane) bits |= 1ull << (u * E + (int)d % E);
  }
  return bits;
}

// The listed elements of the vectors set to -inf.
template <typename T>
__device__ __forceinline__ void drop_listed(uint4 (&x)[kTileVecs], uint64_t bits) {
  constexpr int E = 16 / (int)sizeof(T);
#pragma unroll
  for (int u = 0; u < kTileVecs; ++u) {
    const uint32_t b = (uint32_t)(bits >> (u * E)) & ((1u << E) - 1u);
    if (b) {
      uint32_t w[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
#pragma unroll
      for (int i = 0; i < E; ++i)
        if (b >> i & 1u) {
          if constexpr (sizeof(T) == 2)
            w[i / 2] = i & 1 ? (w[i / 2] & 0x0000FFFFu) | 0xFF800000u : (w[i / 2] & 0xFFFF0000u) | 0x0000FF80u;
          else
            w[i] = 0xFF800000u;
        }
      x[u] = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
}

template <typename T>
__device__ __forceinline__ void put_elem(T* p, float v) {
  if constexpr (sizeof(T) == 2)
    *p = __float2bfloat16_rn(v);
  else
    *p = v;
}

template <typename T, int KIND, bool ALIGNED>
__global__ void __launch_bounds__(kThreads) distill_kernel(Args a) {
  __shared__ Shared sh;
  constexpr int E = 16 / (int)sizeof(T);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t V = a.V, nvec = (V + E - 1) / E;
  for (int64_t row_i = blockIdx.x; row_i < a.T; row_i += gridDim.x) {
    const int64_t src = a.tok_src ? a.tok_src[row_i] : row_i;
    const T* row = static_cast<const T*>(a.logits) + row_i * a.ld;
    T* dz = a.dlogits ? static_cast<T*>(a.dlogits) + row_i * a.ld_out : nullptr;
    const bool valid = src >= 0 && a.mask[src] != 0;
    float mult = 0.f, M = 0.f;   // dz_v = mult 2^(z_v c - M) outside the list
    float corr = 0.f;            // dz of this thread's list entry
    int32_t tok = -1;            // its token
    if (tid == 0) atomicAdd(reinterpret_cast<unsigned long long*>(&a.acc->n_tokens), 1ull);
    if (!valid) {
      if (tid == 0 && src >= 0) a.loss_tok[src] = 0.f;
    } else {
      // ---- the teacher's list: one thread per entry ----
      float tlp = -INFINITY, z = -INFINITY;
      if (tid < a.K) {
        tok = a.top_idx[src * a.ld_top + tid];
        if (tok != -1) tlp = a.top_logp[src * a.ld_top + tid];
      }
      if (tid == 0) sh.bad = sh.n_listed = 0;
      if (tid < GRPO_TOPK_MAX) sh.sorted[tid] = tok;
      __syncthreads();
      const bool listed = tok != -1;
      bool bad = listed && (tok < 0 || (int64_t)tok >= V || tlp != tlp || tlp == INFINITY);
      int rank = 0;
      if (listed)
        for (int k = 0; k < a.K; ++k) {
          const int32_t o = sh.sorted[k];
          bad |= o == tok && k != tid;  // a token listed twice
          rank += o != -1 && o < tok;
        }
      if (listed && !bad) z = elem_f32(row + tok);
      const unsigned nl = __popc(__ballot_sync(0xffffffffu, listed));
      if (lane == 0 && nl) atomicAdd(&sh.n_listed, (int)nl);
      if (bad) atomicOr(&sh.bad, 1);
      __syncthreads();
      if (listed && !bad) sh.sorted[rank] = tok;
      const bool row_bad = sh.bad != 0;
      const int n_listed = sh.n_listed;
      Teacher te{0.f, 0.f, 0.f};
      float q = 0.f;
      {
        // the list's mass: in 64 bits, as q_R = 1 - Q cancels
        const bool use = listed && !row_bad;
        float mx = 0.f;  // FORWARD_TOPK takes the list up to a constant
        if (KIND == GRPO_DISTILL_FORWARD_TOPK) {
          mx = block_max(use ? tlp : -INFINITY, sh.red[1], lane, warp);
          if (mx == -INFINITY) mx = 0.f;
        }
        const double qd = use ? exp((double)tlp - (double)mx) : 0.0;
        const double Q = block_sum(qd, sh.red[0], lane, warp);
        if (KIND == GRPO_DISTILL_FORWARD_TOPK) {
          te.log_norm = (float)((double)mx + log(Q));
          q = Q > 0.0 ? (float)(qd / Q) : 0.f;
          te.q_all = Q > 0.0 ? 1.f : 0.f;
        } else {
          const double qr = 1.0 - Q;
          q = (float)qd;
          const bool none = n_listed >= V;
          if (KIND == GRPO_DISTILL_FORWARD_TAIL)
            te.q_rest = qr < kTailMin || none ? 0.f : (float)qr;
          else
            te.q_rest = (float)fmax(qr, kTailMin);
          te.q_all = (float)(Q + (double)te.q_rest);
        }
      }

      // ---- the row's softmax sums ----
      constexpr bool TAIL = KIND != GRPO_DISTILL_FORWARD_TOPK;
      for (int b = warp; b < a.n_blocks; b += kWarps) {
        Part p{-INFINITY, 0.f, 0.f};
        for (int f = 0; f < a.fold; ++f) {
          const int64_t tile = (int64_t)b * a.fold + f;
          if (tile * tile_elems<T>() >= V) break;
          uint4 x[kTileVecs];
#pragma unroll
          for (int u = 0; u < kTileVecs; ++u)
            x[u] = load_vec<T, ALIGNED>(row, tile * (32 * kTileVecs) + tile_vec(lane, u), V);
          const float tm = warp_max_nan(tile_lane_max<T>(x)) * a.c;
          if (TAIL) drop_listed<T>(x, row_bad ? 0ull : listed_bits<T>(sh.sorted, n_listed, tile, lane));
          const Part tp = tile_part<T, false>(x, tm, a.c);
          p = f == 0 ? tp : part_join(p, tp);
        }
        if (lane == 0) {
          sh.pm[b] = p.m;
          sh.ps[b] = p.s;
        }
      }
      __syncthreads();
      Part p{-INFINITY, 0.f, 0.f};
      for (int b = lane; b < a.n_blocks; b += 32) p = part_join(p, Part{sh.pm[b], sh.ps[b], 0.f});
      p = warp_part(p);
      M = p.m;

      // ---- the token's loss and gradient coefficients ----
      const float t = fmaf(z, a.c, -M);  // log2 of the entry's share before normalisation
      const bool in = listed && !bad;
      const float e = in ? ex2(t) : 0.f;
      const float S = TAIL ? p.s + (float)block_sum((double)e, sh.red[1], lane, warp) : p.s;
      const bool ok = !row_bad && fabsf(M) < INFINITY && S > 0.f && S < INFINITY;
      const float l2s = log2f(S), inv = 1.f / S;
      const float lp = in ? (t - l2s) * kLn2 : 0.f;
      const float pk = e * inv;
      const float pr = TAIL ? p.s * inv : 0.f;
      float term = 0.f;
      if (KIND == GRPO_DISTILL_REVERSE_TAIL)
        term = in && pk > 0.f ? pk * (lp - tlp) : 0.f;
      else
        term = in && q > 0.f ? q * ((tlp - te.log_norm) - lp) : 0.f;
      float loss = (float)block_sum((double)term, sh.red[0], lane, warp);
      float alpha;
      if (KIND == GRPO_DISTILL_FORWARD_TOPK) {
        alpha = te.q_all;
        corr = te.q_all != 0.f ? pk - q : 0.f;
      } else if (KIND == GRPO_DISTILL_FORWARD_TAIL) {
        const float ratio = te.q_rest > 0.f ? te.q_rest / pr : 0.f;
        if (te.q_rest > 0.f) loss += te.q_rest * logf(ratio);
        alpha = te.q_all - ratio;
        corr = fmaf(te.q_all, pk, -q);
      } else {
        const bool tail = pr > 0.f && n_listed < V;
        const float fr = tail ? logf(pr / te.q_rest) : 0.f;
        if (tail) loss = fmaf(pr, fr, loss);
        alpha = tail ? fr - loss : 0.f;
        corr = pk > 0.f ? pk * ((lp - tlp) - loss) : 0.f;
      }
      if (!ok) loss = alpha = corr = __int_as_float(0x7fc00000);
      const float g = a.w_tok ? a.scale * a.w_tok[src] : a.scale;
      corr *= g;
      mult = alpha * g * inv;
      if (!ok) M = 0.f;
      if (tid == 0) {
        a.loss_tok[src] = loss;
        atomicAdd(reinterpret_cast<unsigned long long*>(&a.acc->n_valid), 1ull);
        if (!isfinite(loss) || !isfinite(alpha * g))
          atomicAdd(reinterpret_cast<unsigned long long*>(&a.acc->n_nonfinite), 1ull);
      }
      if (bad) tok = -1;
    }
    if (dz) {
      // ---- dlogits: the dense part, then the list's entries over it ----
      for (int64_t j = tid; j < nvec; j += kThreads) {
        float f[E];
        if (mult == 0.f) {
#pragma unroll
          for (int i = 0; i < E; ++i) f[i] = 0.f;
        } else {
          vec_floats<T>(load_vec<T, ALIGNED>(row, j, V), f);
#pragma unroll
          for (int i = 0; i < E; ++i) f[i] = mult * ex2(fmaf(f[i], a.c, -M));
        }
        if (ALIGNED && (j + 1) * E <= V) {
          if constexpr (sizeof(T) == 2)
            __stcs(reinterpret_cast<uint4*>(dz) + j,
                   make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                              pack_bf16x2(f[6], f[7])));
          else
            __stcs(reinterpret_cast<float4*>(dz) + j, make_float4(f[0], f[1], f[2], f[3]));
        } else {
#pragma unroll
          for (int i = 0; i < E; ++i)
            if (j * E + i < V) put_elem(dz + j * E + i, f[i]);
        }
      }
      __syncthreads();
      if (tok >= 0) put_elem(dz + tok, corr);
    }
    __syncthreads();  // sh is rewritten by the next row
  }
}

template <typename T, int KIND, bool ALIGNED>
int launch(const Args& a, cudaStream_t st) {
  const int64_t grid = std::min<int64_t>(a.T, (int64_t)sm_count() * 2);
  distill_kernel<T, KIND, ALIGNED><<<(unsigned)grid, kThreads, 0, st>>>(a);
  GRPO_CUDA_TRY(cudaGetLastError());
  return GRPO_OK;
}

template <typename T, int KIND>
int launch_aligned(const Args& a, bool aligned, cudaStream_t st) {
  return aligned ? launch<T, KIND, true>(a, st) : launch<T, KIND, false>(a, st);
}

template <typename T>
int dispatch(const Args& a, int32_t kind, bool aligned, cudaStream_t st) {
  if (kind == GRPO_DISTILL_FORWARD_TOPK) return launch_aligned<T, GRPO_DISTILL_FORWARD_TOPK>(a, aligned, st);
  if (kind == GRPO_DISTILL_FORWARD_TAIL) return launch_aligned<T, GRPO_DISTILL_FORWARD_TAIL>(a, aligned, st);
  return launch_aligned<T, GRPO_DISTILL_REVERSE_TAIL>(a, aligned, st);
}

}  // namespace distill
}  // namespace grpo

using namespace grpo;

extern "C" GRPO_API int grpo_distill_topk_fwd_bwd(const void* logits, int32_t dtype, int64_t T, int64_t V, int64_t ld,
                                                  const int64_t* tok_src, const int32_t* top_idx,
                                                  const float* top_logp, int64_t ld_top, int32_t K,
                                                  const uint8_t* mask, int32_t kind, float temperature,
                                                  const float* w_tok, float grad_scale, void* dlogits, int64_t ld_out,
                                                  float* loss_tok, grpo_step_acc* acc, void* stream) {
  if (dtype != GRPO_DTYPE_F32 && dtype != GRPO_DTYPE_BF16) return GRPO_ERR_UNSUPPORTED;
  if (kind != GRPO_DISTILL_FORWARD_TOPK && kind != GRPO_DISTILL_FORWARD_TAIL && kind != GRPO_DISTILL_REVERSE_TAIL)
    return GRPO_ERR_INVALID;
  if (T < 0 || V < 1 || ld < V || V > (int64_t)INT32_MAX || T > (int64_t)INT32_MAX || !acc) return GRPO_ERR_INVALID;
  if (K < 1 || K > GRPO_TOPK_MAX || ld_top < K) return GRPO_ERR_INVALID;
  if (dlogits && ld_out < V) return GRPO_ERR_INVALID;
  if (!(temperature > 0.f) || !std::isfinite(temperature) || !std::isfinite(grad_scale)) return GRPO_ERR_INVALID;
  const float c = (float)(1.4426950408889634 / (double)temperature);
  if (!std::isfinite(c) || c < 1.1754944e-38f) return GRPO_ERR_INVALID;
  if (T == 0) return GRPO_OK;
  if (!logits || !top_idx || !top_logp || !mask || !loss_tok) return GRPO_ERR_INVALID;
  const size_t es = dtype == GRPO_DTYPE_F32 ? 4 : 2;
  const uintptr_t in = reinterpret_cast<uintptr_t>(logits), out = reinterpret_cast<uintptr_t>(dlogits);
  if (in % es || out % es) return GRPO_ERR_INVALID;
  // dlogits is written while other rows of the logits are still to be read
  if (dlogits && in < out + ((T - 1) * ld_out + V) * es && out < in + ((T - 1) * ld + V) * es) return GRPO_ERR_INVALID;

  distill::Args a{};
  a.logits = logits;
  a.T = T;
  a.V = V;
  a.ld = ld;
  a.tok_src = tok_src;
  a.top_idx = top_idx;
  a.top_logp = top_logp;
  a.ld_top = ld_top;
  a.K = K;
  a.mask = mask;
  a.w_tok = w_tok;
  a.c = c;
  a.scale = (float)((double)grad_scale / (double)temperature);
  a.dlogits = dlogits;
  a.ld_out = ld_out;
  a.loss_tok = loss_tok;
  a.acc = acc;
  const int64_t tiles = (V * (int64_t)es + 4095) / 4096;
  a.fold = (int32_t)((tiles + distill::kMaxBlocks - 1) / distill::kMaxBlocks);
  a.n_blocks = (int32_t)((tiles + a.fold - 1) / a.fold);
  const bool aligned = ((in | out) & 15u) == 0 && (ld * es) % 16 == 0 && (!dlogits || (ld_out * es) % 16 == 0);
  const cudaStream_t st = as_stream(stream);
  return dtype == GRPO_DTYPE_BF16 ? distill::dispatch<__nv_bfloat16>(a, kind, aligned, st)
                                  : distill::dispatch<float>(a, kind, aligned, st);
}
