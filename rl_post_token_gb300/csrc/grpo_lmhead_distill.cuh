#pragma once
// Kernels of the LM-head form of the distillation loss (FORWARD_TOPK, formulas in
// grpo_distill.cuh): the vocabulary's softmax partials, the recompute and the two gradient products
// are the LM-head GEMMs (grpo_lmhead_gemm.cuh); what is left per token is its list.
//
//  lse_kernel   the token's (shift, sum) from its vocabulary tiles' partials
//  list_kernel  z = h . W[i_k] for every list entry, the token's loss, and the entries' gradients
//  fix_kernel   the entries' gradients put over the dense dlogits p_v of a recomputed chunk
//
// The K dot products of a token read K rows of W (K H 2 bytes: 256 KB at K = 64, H = 2048), a few
// percent of the step's GEMM time. They replace a pick-up in the GEMM's epilogue, which would test
// every column of every tile against the token's list.
#include "grpo_distill.cuh"

namespace grpo {
namespace lmhead {

constexpr int kLseWarps = 16;

// A block takes 32 tokens (lane = token: a partial's load is one 128-byte line), its warps every
// 16th tile in order; warp 0 joins the warps' in order. idx / live_n: the compact order of a pass A
// that skipped the masked tokens (row i holds token idx[i]), or NULL.
__global__ void __launch_bounds__(kLseWarps * 32) lse_kernel(int64_t T, int n_col_tiles, const float* part_m,
                                                             const float* part_s, const int32_t* idx,
                                                             const int32_t* live_n, float* m_out, float* s_out) {
  __shared__ float wm[kLseWarps][32], ws[kLseWarps][32];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int64_t i = (int64_t)blockIdx.x * 32 + lane;
  const bool on = i < T && (!idx || i < (int64_t)*live_n);
  MS t{-INFINITY, 0.f};
  if (on)
#pragma unroll 4
    for (int c = w; c < n_col_tiles; c += kLseWarps) t = ms2_combine(t, MS{part_m[(int64_t)c * T + i], part_s[(int64_t)c * T + i]});
  wm[w][lane] = t.m;
  ws[w][lane] = t.s;
  __syncthreads();
  if (w == 0 && on) {
    MS tot{wm[0][lane], ws[0][lane]};
#pragma unroll
    for (int k = 1; k < kLseWarps; ++k) tot = ms2_combine(tot, MS{wm[k][lane], ws[k][lane]});
    const int64_t tok = idx ? (int64_t)idx[i] : i;
    m_out[tok] = tot.m;
    s_out[tok] = tot.s;
  }
}

struct ListArgs {
  int64_t T, V;
  int H;
  const __nv_bfloat16 *h, *W;
  const int32_t* top_idx;
  const float* top_logp;
  int64_t ld_top;
  int K;
  const uint8_t* mask;
  const float* w_tok;
  float scale;
  const float *m, *s;  // [T] the token's softmax shift and sum (log2 units)
  float *lse2, *coef;  // [T] out: what the recompute's epilogue takes
  float* corr;         // [T][K] out: the entries' dlogits
  float* loss_tok;
  grpo_step_acc* acc;
};

constexpr int kListThreads = 256;

__device__ __forceinline__ float dot8(const uint4& a, const uint4& b, float acc) {
  const uint32_t x[4] = {a.x, a.y, a.z, a.w}, y[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    acc = fmaf(bf16_lo(x[i]), bf16_lo(y[i]), acc);
    acc = fmaf(bf16_hi(x[i]), bf16_hi(y[i]), acc);
  }
  return acc;
}

__device__ __forceinline__ float list_sum(float v, float* red, int lane, int warp) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (lane == 0) red[warp] = v;
  __syncthreads();
  float s = 0.f;
#pragma unroll
  for (int w = 0; w < kListThreads / 32; ++w) s += red[w];
  __syncthreads();
  return s;
}

// One block per token: its warps take the list's dot products (h from shared memory), then thread
// k holds entry k.
__global__ void __launch_bounds__(kListThreads) list_kernel(ListArgs a) {
  extern __shared__ __align__(16) uint8_t smem[];
  uint4* sh_h = reinterpret_cast<uint4*>(smem);  // [H / 8]
  __shared__ int32_t sh_tok[GRPO_TOPK_MAX];
  __shared__ float sh_z[GRPO_TOPK_MAX], red[kListThreads / 32];
  __shared__ int sh_bad;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t t = blockIdx.x;
  const int K = a.K;
  if (tid == 0) atomicAdd(reinterpret_cast<unsigned long long*>(&a.acc->n_tokens), 1ull);
  if (a.mask[t] == 0) {
    if (tid == 0) {
      a.loss_tok[t] = 0.f;
      a.coef[t] = 0.f;
      a.lse2[t] = 0.f;
    }
    return;
  }
  int32_t tok = -1;
  float tlp = -INFINITY;
  if (tid < K) {
    tok = a.top_idx[t * a.ld_top + tid];
    if (tok != -1) tlp = a.top_logp[t * a.ld_top + tid];
  }
  sh_tok[tid] = tok;
  if (tid == 0) sh_bad = 0;
  const int nvec = a.H >> 3;
  for (int j = tid; j < nvec; j += kListThreads) sh_h[j] = __ldg(reinterpret_cast<const uint4*>(a.h + t * a.H) + j);
  __syncthreads();
  const bool listed = tok != -1;
  bool bad = listed && (tok < 0 || (int64_t)tok >= a.V || tlp != tlp || tlp == INFINITY);
  if (listed)
    for (int k = 0; k < K; ++k) bad |= sh_tok[k] == tok && k != tid;
  if (bad) atomicOr(&sh_bad, 1);
  for (int k = warp; k < K; k += kListThreads / 32) {
    const int32_t v = sh_tok[k];
    if (v < 0 || (int64_t)v >= a.V) continue;  // warp-uniform
    const uint4* wr = reinterpret_cast<const uint4*>(a.W + (int64_t)v * a.H);
    float d0 = 0.f, d1 = 0.f;
    int j = lane;
#pragma unroll 4
    for (; j + 32 < nvec; j += 64) {
      d0 = dot8(sh_h[j], __ldg(wr + j), d0);
      d1 = dot8(sh_h[j + 32], __ldg(wr + j + 32), d1);
    }
    if (j < nvec) d0 = dot8(sh_h[j], __ldg(wr + j), d0);
    d0 += d1;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) d0 += __shfl_xor_sync(0xffffffffu, d0, o);
    if (lane == 0) sh_z[k] = d0;
  }
  __syncthreads();
  const bool row_bad = sh_bad != 0;
  const bool use = listed && !row_bad;
  // the list renormalised (it may carry any constant)
  float mx = warp_max_f32(use ? tlp : -INFINITY);
  if (lane == 0) red[warp] = mx;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kListThreads / 32; ++w) mx = fmaxf(mx, red[w]);
  __syncthreads();
  const float mq = mx == -INFINITY ? 0.f : mx;
  const float qe = use ? expf(tlp - mq) : 0.f;
  const float Q = list_sum(qe, red, lane, warp);
  const float q = Q > 0.f ? qe / Q : 0.f;
  const float m = a.m[t], s = a.s[t];
  const float l2s = log2f(s), lse2 = m + l2s;
  // as in the LM-head loss, a row past the vouched logit range counts as non-finite
  const bool ok = !row_bad && s > 0.f && s < INFINITY && fabsf(lse2) <= kLseMax * kLog2e;
  const float u = use ? fmaf(sh_z[tid], kLog2e, -m) - l2s : 0.f;  // log2 p_k
  const float loss = list_sum(q > 0.f ? q * (((tlp - mq) - logf(Q)) - u * kLn2) : 0.f, red, lane, warp);
  const float nan = __int_as_float(0x7fc00000);
  const float g = a.w_tok ? a.scale * a.w_tok[t] : a.scale;
  const float coef = !ok ? nan : Q > 0.f ? g : 0.f;
  if (tid < K) a.corr[t * K + tid] = !ok ? nan : use && Q > 0.f ? g * (ex2(u) - q) : 0.f;
  if (tid == 0) {
    const float l = ok ? loss : nan;
    a.loss_tok[t] = l;
    a.coef[t] = coef;
    a.lse2[t] = lse2;
    atomicAdd(reinterpret_cast<unsigned long long*>(&a.acc->n_valid), 1ull);
    if (!isfinite(l) || !isfinite(coef)) atomicAdd(reinterpret_cast<unsigned long long*>(&a.acc->n_nonfinite), 1ull);
  }
}

// The list entries of the live tokens that fall into the chunk's columns [v0, v0 + vc), over the
// dense dlogits the recompute has just written. Thread = (compact row, entry).
__global__ void __launch_bounds__(256) fix_kernel(const int32_t* live_n, const int32_t* row_idx, const int32_t* top_idx,
                                                  int64_t ld_top, int K, const float* corr, __nv_bfloat16* dz,
                                                  int64_t ldz, int64_t v0, int64_t vc) {
  const int64_t n = (int64_t)*live_n * K;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
    const int64_t r = i / K, t = row_idx[r];
    const int k = (int)(i - r * K);
    const int64_t c = (int64_t)top_idx[t * ld_top + k] - v0;
    if (c >= 0 && c < vc) dz[r * ldz + c] = __float2bfloat16_rn(corr[t * K + k]);
  }
}

}  // namespace lmhead
}  // namespace grpo
