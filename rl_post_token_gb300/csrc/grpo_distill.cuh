#pragma once
// Distillation from a teacher's top tokens: the arithmetic of one token's list. With the student's
// p = softmax(z/tau), the teacher's list S of (token i_k, log q_k), Q = sum q_k, P = sum_S p,
// q_R = 1 - Q and p_R = 1 - P:
//
//   FORWARD_TOPK  L = sum_k qh_k (log qh_k - log p_k), qh = q/Q
//   FORWARD_TAIL  L = sum_k q_k (log q_k - log p_k) + q_R (log q_R - log p_R)
//   REVERSE_TAIL  L = sum_k p_k f_k + p_R f_R,  f_k = log p_k - log q_k, f_R = log p_R - log q_R
//
// and dL/d(z_v/tau) = alpha p_v outside S and corr_k on S:
//
//   FORWARD_TOPK  alpha = 1                      corr_k = p_k - qh_k
//   FORWARD_TAIL  alpha = Q + q_R - q_R/p_R      corr_k = (Q + q_R) p_k - q_k
//   REVERSE_TAIL  alpha = f_R - L                corr_k = p_k (f_k - L)
//
// p_R is summed over the tokens outside S, never formed as 1 - P: a confident student leaves a
// remainder that 1 - P would round away.
#include "grpo_vocab.cuh"

namespace grpo {
namespace distill {

// A teacher remainder below 2^-24 cannot be told from the rounding of its float32 log-probs:
// FORWARD_TAIL counts it as none, REVERSE_TAIL takes this value in its logarithm.
constexpr double kTailMin = 5.9604644775390625e-08;

constexpr int kPerLane = GRPO_TOPK_MAX / 32;  // list entries a lane of the list's warp holds

template <typename F>
__device__ __forceinline__ F warp_sum(F v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// The row's partial (without q) from those of its blocks: get(i) gives block i's (m, s). Lane l joins
// blocks l, l + 32, ... in order.
template <typename G>
__device__ __forceinline__ Part join_blocks(int n, int lane, G get) {
  float m = -INFINITY, s = 0.f;
  for (int i = lane; i < n; i += 32) {
    const float2 b = get(i);
    const float M = fmaxf(m, b.x);
    // (where nothing has mass yet the sums are added as they are: 0, or the NaN of a NaN block)
    s = M == -INFINITY ? s + b.y : fmaf(s, ex2(m - M), b.y * ex2(b.x - M));
    m = M;
  }
  return warp_part<false>(Part{m, s, 0.f});
}

// One token's list, entry 32 j + lane in slot j of the lane. The warp holds it from the loads to the
// gradients.
template <typename T, int KIND>
struct List {
  int32_t tok[kPerLane];  // -1: unused
  float tlp[kPerLane], z[kPerLane], q[kPerLane];
  float log_norm;  // FORWARD_TOPK: log of the list's mass, its log-probs taken from their largest
  float q_rest;    // q_R (tail kinds), floored as above; 0 where nothing lies outside the list
  float q_all;     // FORWARD_TOPK: 1, or 0 without a list; FORWARD_TAIL: Q + q_R
  int n;           // tokens listed
  bool bad;        // a token twice or outside the vocabulary, a NaN or +inf log-prob

  // Loads the list and the listed logits and writes the tokens to sh_tok [GRPO_TOPK_MAX] (unused
  // entries -1; all of them if the list is bad).
  __device__ __forceinline__ void load(const int32_t* top_idx, const float* top_logp, int K, const T* row, int64_t V,
                                       int32_t* sh_tok, int lane) {
    bool b = false;
    n = 0;
#pragma unroll
    for (int j = 0; j < kPerLane; ++j) {
      tok[j] = -1;
      tlp[j] = z[j] = -INFINITY;
      if (32 * j < K && 32 * j + lane < K) {
        tok[j] = top_idx[32 * j + lane];
        tlp[j] = top_logp[32 * j + lane];
      }
    }
#pragma unroll
    for (int j = 0; j < kPerLane; ++j) {
      if (32 * j < K) {  // warp-uniform, here and below
        const bool in = tok[j] >= 0 && (int64_t)tok[j] < V;
        if (in) z[j] = elem_f32(row + tok[j]);
        if (tok[j] == -1) tlp[j] = -INFINITY;
        b |= tok[j] != -1 && (!in || tlp[j] != tlp[j] || tlp[j] == INFINITY);
        n += __popc(__ballot_sync(0xffffffffu, tok[j] != -1));
      }
      sh_tok[32 * j + lane] = tok[j];
    }
    __syncwarp();
    // every entry against the entries before it
#pragma unroll
    for (int j = 0; j < kPerLane; ++j)
      if (32 * j < K) {
        const int k = 32 * j + lane;
#pragma unroll 2
        for (int k0 = 0; k0 < 32 * j + 32; k0 += 4) {
          const int4 o = *reinterpret_cast<const int4*>(sh_tok + k0);
          b |= tok[j] != -1 && ((o.x == tok[j] && k0 < k) || (o.y == tok[j] && k0 + 1 < k) ||
                                (o.z == tok[j] && k0 + 2 < k) || (o.w == tok[j] && k0 + 3 < k));
        }
      }
    bad = __any_sync(0xffffffffu, b);
    __syncwarp();
    if (bad) {
#pragma unroll
      for (int j = 0; j < kPerLane; ++j) sh_tok[32 * j + lane] = tok[j] = -1;
      __syncwarp();
    }
    log_norm = q_rest = 0.f;
    if constexpr (KIND == GRPO_DISTILL_FORWARD_TOPK) {  // takes the list up to a constant
      float mx = -INFINITY;
#pragma unroll
      for (int j = 0; j < kPerLane; ++j) mx = fmaxf(mx, tok[j] != -1 ? tlp[j] : -INFINITY);
      mx = warp_max_f32(mx);
      const float shift = mx == -INFINITY ? 0.f : mx;
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < kPerLane; ++j) {
        q[j] = 0.f;
        if (32 * j < K) {
          q[j] = tok[j] != -1 ? expf(tlp[j] - shift) : 0.f;
          sum += q[j];
        }
      }
      const float Q = warp_sum(sum), inv = Q > 0.f ? 1.f / Q : 0.f;
      // log(q/Q) is formed as (log q - shift) - log Q: exact differences of the list's values
#pragma unroll
      for (int j = 0; j < kPerLane; ++j) {
        q[j] *= inv;
        tlp[j] -= shift;
      }
      log_norm = logf(Q);
      q_all = Q > 0.f ? 1.f : 0.f;
    } else {
      // the list's mass in 64 bits, as q_R = 1 - Q cancels
      double sum = 0.0;
#pragma unroll
      for (int j = 0; j < kPerLane; ++j) {
        q[j] = 0.f;
        if (32 * j < K) {
          const double qd = tok[j] != -1 ? exp((double)tlp[j]) : 0.0;
          sum += qd;
          q[j] = (float)qd;
        }
      }
      const double Q = warp_sum(sum), qr = 1.0 - Q;
      if (KIND == GRPO_DISTILL_FORWARD_TAIL)
        q_rest = qr < kTailMin || n >= V ? 0.f : (float)qr;
      else
        q_rest = (float)fmax(qr, kTailMin);
      q_all = (float)(Q + (double)q_rest);
    }
  }

  // The token's loss and gradients from the row's partial p (the tail kinds': without the listed
  // tokens). dlogits are mult 2^(z c - shift) outside the list and sh_corr on it; g: the gradient
  // scale. A row without a distribution or with a bad list has NaN for all of them.
  __device__ __forceinline__ void finish(Part p, float c, float g, int64_t V, int K, float* sh_corr, int lane,
                                         float& loss, float& shift, float& mult, bool& finite) {
    constexpr bool TAIL = KIND != GRPO_DISTILL_FORWARD_TOPK;
    float t[kPerLane], e[kPerLane];
    float se = 0.f;
#pragma unroll
    for (int j = 0; j < kPerLane; ++j) {
      t[j] = e[j] = 0.f;
      if (32 * j < K) {
        t[j] = fmaf(z[j], c, -p.m);
        e[j] = tok[j] != -1 ? ex2(t[j]) : 0.f;
        if (TAIL) se += e[j];
      }
    }
    const float S = TAIL ? p.s + warp_sum(se) : p.s;
    const bool ok = !bad && fabsf(p.m) < INFINITY && S > 0.f && S < INFINITY;
    const float l2s = log2f(S), inv = 1.f / S, pr = TAIL ? p.s * inv : 0.f;
    float sum = 0.f;
    float f[kPerLane];  // REVERSE_TAIL: log p - log q
#pragma unroll
    for (int j = 0; j < kPerLane; ++j) {
      f[j] = 0.f;
      if (32 * j >= K) continue;
      const float lp = (t[j] - l2s) * kLn2, pk = e[j] * inv;
      float term;
      if (KIND == GRPO_DISTILL_REVERSE_TAIL) {
        f[j] = pk > 0.f ? lp - tlp[j] : 0.f;
        term = pk > 0.f ? pk * f[j] : 0.f;
      } else {
        term = tok[j] != -1 && q[j] > 0.f ? q[j] * ((tlp[j] - log_norm) - lp) : 0.f;
      }
      sum += term;
    }
    loss = warp_sum(sum);
    float alpha;
    if (KIND == GRPO_DISTILL_FORWARD_TOPK) {
      alpha = q_all;
    } else if (KIND == GRPO_DISTILL_FORWARD_TAIL) {
      const float ratio = q_rest > 0.f ? q_rest / pr : 0.f;
      if (q_rest > 0.f) loss += q_rest * logf(ratio);
      alpha = q_all - ratio;
    } else {
      const bool tail = pr > 0.f && n < V;
      const float fr = tail ? logf(pr / q_rest) : 0.f;
      if (tail) loss = fmaf(pr, fr, loss);
      alpha = tail ? fr - loss : 0.f;
    }
    const float nan = __int_as_float(0x7fc00000);
    if (!ok) loss = alpha = nan;
#pragma unroll
    for (int j = 0; j < kPerLane; ++j)
      if (32 * j < K) {
        const float pk = e[j] * inv;
        float corr;
        if (KIND == GRPO_DISTILL_FORWARD_TOPK)
          corr = q_all != 0.f ? pk - q[j] : 0.f;
        else if (KIND == GRPO_DISTILL_FORWARD_TAIL)
          corr = fmaf(q_all, pk, -q[j]);
        else
          corr = pk > 0.f ? pk * (f[j] - loss) : 0.f;
        sh_corr[32 * j + lane] = ok ? corr * g : nan;
      }
    shift = ok ? p.m : 0.f;
    mult = ok ? alpha * g * inv : nan;
    finite = isfinite(loss) && isfinite(alpha * g);
  }
};

}  // namespace distill
}  // namespace grpo
