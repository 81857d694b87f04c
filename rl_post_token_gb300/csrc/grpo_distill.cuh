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

template <typename F>
__device__ __forceinline__ F warp_sum(F v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// The row's partial (without q) from those of its n blocks: get(i) gives block i's (m, s). Lane l sums
// blocks l, l + 32, ... in order, rescaled to the row's largest shift.
template <typename G>
__device__ __forceinline__ Part join_blocks(int n, int lane, G get) {
  float m = -INFINITY, bad = 0.f;
#pragma unroll 4
  for (int i = lane; i < n; i += 32) {
    const float2 b = get(i);
    m = fmaxf(m, b.x);
    bad += b.x != b.x ? b.x : 0.f;  // a NaN block
  }
  m = warp_max_f32(m);
  float s = bad;
  const float shift = m == -INFINITY ? 0.f : m;
#pragma unroll 4
  for (int i = lane; i < n; i += 32) {
    const float2 b = get(i);
    s = fmaf(b.y, ex2(b.x - shift), s);
  }
  return {m, warp_sum(s), 0.f};
}

// One token's list, entry 32 j + lane in slot j < J of the lane (K <= 32 J). The warp holds it from the
// loads to the gradients. Instances of J = 2 and 8 slots: the small one keeps a list of up to 64
// tokens without spilling.
template <typename T, int KIND, int J>
struct List {
  int32_t tok[J];  // -1: unused
  float tlp[J], z[J], q[J];
  float log_norm;  // FORWARD_TOPK: log of the list's mass, its log-probs taken from their largest
  float q_rest;    // q_R (tail kinds), floored as above; 0 where nothing lies outside the list
  float q_all;     // FORWARD_TOPK: 1, or 0 without a list; FORWARD_TAIL: Q + q_R
  int n;           // tokens listed
  bool bad;        // a token twice or outside the vocabulary, a NaN or +inf log-prob

  // Loads the list and the listed logits and writes the tokens to sh_tok [32 J] (unused entries
  // -1; all of them if the list is bad).
  __device__ __forceinline__ void load(const int32_t* top_idx, const float* top_logp, int K, const T* row, int64_t V,
                                       int32_t* sh_tok, int lane) {
    bool b = false;
    n = 0;
#pragma unroll
    for (int j = 0; j < J; ++j) {
      tok[j] = -1;
      tlp[j] = z[j] = -INFINITY;
      if (32 * j < K && 32 * j + lane < K) {
        tok[j] = top_idx[32 * j + lane];
        tlp[j] = top_logp[32 * j + lane];
      }
    }
#pragma unroll
    for (int j = 0; j < J; ++j) {
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
    for (int j = 0; j < J; ++j)
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
      for (int j = 0; j < J; ++j) sh_tok[32 * j + lane] = tok[j] = -1;
      __syncwarp();
    }
    log_norm = q_rest = 0.f;
    if constexpr (KIND == GRPO_DISTILL_FORWARD_TOPK) {  // takes the list up to a constant
      float mx = -INFINITY;
#pragma unroll
      for (int j = 0; j < J; ++j) mx = fmaxf(mx, tok[j] != -1 ? tlp[j] : -INFINITY);
      mx = warp_max_f32(mx);
      const float shift = mx == -INFINITY ? 0.f : mx;
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < J; ++j) {
        q[j] = 0.f;
        if (32 * j < K) {
          q[j] = tok[j] != -1 ? expf(tlp[j] - shift) : 0.f;
          sum += q[j];
        }
      }
      const float Q = warp_sum(sum), inv = Q > 0.f ? 1.f / Q : 0.f;
      // log(q/Q) is formed as (log q - shift) - log Q: exact differences of the list's values
#pragma unroll
      for (int j = 0; j < J; ++j) {
        q[j] *= inv;
        tlp[j] -= shift;
      }
      log_norm = logf(Q);
      q_all = Q > 0.f ? 1.f : 0.f;
    } else {
      // the list's mass in 64 bits, as q_R = 1 - Q cancels
      double sum = 0.0;
#pragma unroll
      for (int j = 0; j < J; ++j) {
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

  // From stats on z holds t = z c - shift (log2 of the entry's share before the normalisation).
  float l2s, inv, pr, alpha, loss;
  bool ok;

  // The row's part of dlogits from its partial p (the tail kinds': without the listed tokens):
  // dlogits are mult 2^(z c - shift) outside the list. g: the gradient scale. A row without a
  // distribution or with a bad list has NaN throughout.
  __device__ __forceinline__ void stats(Part p, float c, float g, int64_t V, int K, float& out_shift, float& out_mult) {
    constexpr bool TAIL = KIND != GRPO_DISTILL_FORWARD_TOPK;
    float se = 0.f;
#pragma unroll
    for (int j = 0; j < J; ++j) {
      if (32 * j < K) {
        z[j] = fmaf(z[j], c, -p.m);
        if (TAIL && tok[j] != -1) se += ex2(z[j]);
      }
    }
    const float S = TAIL ? p.s + warp_sum(se) : p.s;
    ok = !bad && fabsf(p.m) < INFINITY && S > 0.f && S < INFINITY;
    inv = 1.f / S;
    pr = TAIL ? p.s * inv : 0.f;
    l2s = log2f(S);
    if constexpr (KIND == GRPO_DISTILL_FORWARD_TOPK) {
      alpha = q_all;
    } else if constexpr (KIND == GRPO_DISTILL_FORWARD_TAIL) {
      alpha = q_all - (q_rest > 0.f ? q_rest / pr : 0.f);
    } else {
      sum_loss(V, K);
      const bool tail = pr > 0.f && n < V;
      const float fr = tail ? logf(pr / q_rest) : 0.f;
      if (tail) loss = fmaf(pr, fr, loss);
      alpha = tail ? fr - loss : 0.f;
    }
    if (!ok) alpha = __int_as_float(0x7fc00000);
    out_shift = ok ? p.m : 0.f;
    out_mult = ok ? alpha * g * inv : alpha;
  }

  // The student's probability of the entry in slot j.
  __device__ __forceinline__ float share(int j) const { return tok[j] != -1 ? ex2(z[j]) * inv : 0.f; }

  // The list's terms of the loss.
  __device__ __forceinline__ void sum_loss(int64_t V, int K) {
    float sum = 0.f;
#pragma unroll
    for (int j = 0; j < J; ++j) {
      if (32 * j >= K) continue;
      const float lp = (z[j] - l2s) * kLn2, pk = share(j);
      if (KIND == GRPO_DISTILL_REVERSE_TAIL)
        sum += pk > 0.f ? pk * (lp - tlp[j]) : 0.f;
      else
        sum += tok[j] != -1 && q[j] > 0.f ? q[j] * ((tlp[j] - log_norm) - lp) : 0.f;
    }
    loss = warp_sum(sum);
  }

  // The token's loss (after stats).
  __device__ __forceinline__ float token_loss(int64_t V, int K, float g, bool& finite) {
    if constexpr (KIND != GRPO_DISTILL_REVERSE_TAIL) {
      sum_loss(V, K);
      if (KIND == GRPO_DISTILL_FORWARD_TAIL && q_rest > 0.f) loss += q_rest * logf(q_rest / pr);
    }
    if (!ok) loss = __int_as_float(0x7fc00000);
    finite = isfinite(loss) && isfinite(alpha * g);
    return loss;
  }

  // dlogits of the entry in slot j (after stats and, for REVERSE_TAIL, which needs the loss, too).
  __device__ __forceinline__ float entry_grad(int j, float g) const {
    const float pk = share(j);
    float corr;
    if (KIND == GRPO_DISTILL_FORWARD_TOPK)
      corr = q_all != 0.f ? pk - q[j] : 0.f;
    else if (KIND == GRPO_DISTILL_FORWARD_TAIL)
      corr = fmaf(q_all, pk, -q[j]);
    else
      corr = pk > 0.f ? pk * (((z[j] - l2s) * kLn2 - tlp[j]) - loss) : 0.f;
    return ok ? corr * g : __int_as_float(0x7fc00000);
  }
};

}  // namespace distill
}  // namespace grpo
