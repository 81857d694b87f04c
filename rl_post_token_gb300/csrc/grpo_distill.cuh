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
// remainder that 1 - P would round away. It may even lie below the float32 range as a share of the row
// (every token outside 88 nats or more below the largest), where q_R log p_R and q_R p_v/p_R are ordinary
// numbers. So FORWARD_TAIL keeps the sum outside against its own shift m_R = max z c over the tokens
// outside, s_R = sum 2^(z c - m_R):
//
//   log2 p_R = (m_R - m) + log2 s_R - log2 S,   alpha p_v = (Q p_R + q_R p_R - q_R) 2^(z c - m_R) / s_R
#include "grpo_vocab.cuh"

namespace grpo {
namespace distill {

// A teacher remainder below 2^-24 cannot be told from the rounding of its float32 log-probs:
// FORWARD_TAIL counts it as none, REVERSE_TAIL takes this value in its logarithm.
constexpr double kTailMin = 5.9604644775390625e-08;
// Where the student has no mass outside the list, a remainder makes the loss infinite, or as large as a finite
// mask. A teacher that has none either (both rows restricted to the same few tokens) lists log-probs whose
// masses sum to 1 only up to their errors: sum q |d log q| <= 2^-22 + 39 2^-24 of the scoring call's row sum,
// 2 log2(V) 2^-24 ln2 and 2^-23 (|log q| + |z - max|/tau) on average, 6e-6 in all. So where every token
// outside is 2^126 times less probable than the row's most probable, FORWARD_TAIL counts a remainder below
// 2^-16 as none.
constexpr float kTailNone = 1.52587890625e-05f;

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

// K rounded up to whole warps: the entries that a list takes in shared memory.
__host__ __device__ __forceinline__ int padded_list(int K) { return (K + 31) & ~31; }

// A list's entries in shared memory (16-byte aligned), unused ones with token -1.
struct Entries {
  int32_t* tok;
  float *tlp,  // log q
      *z,      // the student's logit; from token_loss (tail kinds: stats) on z c - shift, log2 of its share
      *q;      // the teacher's probability (FORWARD_TOPK: of the renormalised list)
  int32_t* seen;  // the tokens hashed, 2 places for each, to find one that is listed twice
  static constexpr int kWords = 6;
  __device__ Entries(void* mem, int padded)
      : tok(static_cast<int32_t*>(mem)), tlp(static_cast<float*>(mem) + padded), z(tlp + padded), q(z + padded),
        seen(static_cast<int32_t*>(mem) + 4 * padded) {}
};

// One token's list, held by one warp from the loads to the gradients. The entries stay in shared memory,
// lane l working on entries l, l + 32, ... (in registers, 8 a lane spilled and 2 a lane were no faster).
template <typename T, int KIND>
struct List {
  const Entries en;
  const int K, padded, lane;  // padded: K rounded up to whole warps
  const int64_t V;
  float log_norm;  // FORWARD_TOPK: log of the list's mass, its log-probs taken from their largest
  float q_rest;    // q_R (tail kinds), floored as above; FORWARD_TAIL: 0 where the list is all or nothing
  float q_all;     // FORWARD_TOPK: 1, or 0 without a list; FORWARD_TAIL: Q + q_R
  int n;           // tokens listed
  bool bad;        // a token twice or outside the vocabulary, a NaN or +inf log-prob
  float z_max;                        // the largest listed logit (NaN if one is)
  float pm, cz, sum, inv, pr;         // from stats on; cz: the scale that goes with the shift pm
  float unit, tau_c;                  // from its t to log2 units; log2(e)/tau
  float alpha;                        // (FORWARD_TAIL: alpha p_R)
  float rest_m, rest_s, rest_inv;     // FORWARD_TAIL: the shift of the sum outside the list, the sum and its inverse
  float l2s, loss;                    // from token_loss on (REVERSE_TAIL: from stats)
  bool ok;

  static constexpr bool TAIL = KIND != GRPO_DISTILL_FORWARD_TOPK;

  __device__ List(const Entries& entries, int k, int64_t v, int l) : en(entries), K(k), padded(padded_list(k)), lane(l), V(v) {}

  // Loads the list and the listed logits. A bad list is left without tokens.
  __device__ __forceinline__ void load(const int32_t* top_idx, const float* top_logp, const T* row) {
    bool b = false;
    n = 0;
    float mx = -INFINITY;
    z_max = -INFINITY;
    // a token listed twice is found by hashing (all pairs of 256 tokens took longer than their row:
    // 8192 x 151936 bf16, K = 256: 1120 us, so 954)
    const uint32_t places = 2u * (uint32_t)padded;
    for (int k = lane; k < 2 * padded; k += 32) en.seen[k] = -1;
    __syncwarp();
#pragma unroll 2
    for (int k = lane; k < padded; k += 32) {
      int32_t tok = -1;
      float tlp = -INFINITY, z = -INFINITY;
      if (k < K) {
        tok = top_idx[k];
        tlp = top_logp[k];
      }
      const bool in = tok >= 0 && (int64_t)tok < V;
      if (in) {
        z = elem_f32(row + tok);
        uint32_t h = __umulhi((uint32_t)tok * 2654435769u, places);  // (2^32 over the golden ratio)
        for (;;) {  // ends: there are more places than tokens
          const int32_t old = atomicCAS(&en.seen[h], -1, tok);
          if (old == -1) break;
          if (old == tok) {
            b = true;
            break;
          }
          h = h + 1 == places ? 0 : h + 1;
        }
      }
      if (tok == -1) tlp = -INFINITY;
      b |= tok != -1 && (!in || tlp != tlp || tlp == INFINITY);
      n += __popc(__ballot_sync(0xffffffffu, tok != -1));
      mx = fmaxf(mx, tlp);
      z_max = max_nan(z_max, z);
      en.tok[k] = tok;
      en.tlp[k] = tlp;
      en.z[k] = z;
    }
    bad = __any_sync(0xffffffffu, b);
    if (TAIL) z_max = bad ? -INFINITY : warp_max_nan(z_max);  // (a bad list has no tokens)
    __syncwarp();
    log_norm = q_rest = 0.f;
    if constexpr (!TAIL) {  // takes the list up to a constant
      mx = warp_max_f32(bad ? -INFINITY : mx);
      const float shift = mx == -INFINITY ? 0.f : mx;
      float sum = 0.f;
      for (int k = lane; k < padded; k += 32) {
        if (bad) en.tok[k] = -1;
        // log(q/Q) will be formed as (log q - shift) - log Q: exact differences of the list's values
        const float d = en.tlp[k] - shift, q = en.tok[k] != -1 ? expf(d) : 0.f;
        en.tlp[k] = d;
        en.q[k] = q;
        sum += q;
      }
      const float Q = warp_sum(sum), scale = Q > 0.f ? 1.f / Q : 0.f;
      for (int k = lane; k < padded; k += 32) en.q[k] *= scale;
      log_norm = logf(Q);
      q_all = Q > 0.f ? 1.f : 0.f;
    } else {
      // the list's mass in 64 bits, as q_R = 1 - Q cancels
      double sum = 0.0;
#pragma unroll 1
      for (int k = lane; k < padded; k += 32) {
        if (bad) en.tok[k] = -1;
        const double q = en.tok[k] != -1 ? exp((double)en.tlp[k]) : 0.0;
        en.q[k] = (float)q;
        sum += q;
      }
      const double Q = warp_sum(sum), qr = 1.0 - Q;
      if (KIND == GRPO_DISTILL_FORWARD_TAIL)
        q_rest = qr < kTailMin || n >= V || n == 0 ? 0.f : (float)qr;  // (no list: loss and gradient 0)
      else
        q_rest = (float)fmax(qr, kTailMin);
      q_all = (float)(Q + (double)q_rest);
    }
  }

  // The row's part of dlogits from its partial p (the tail kinds': without the listed tokens):
  // dlogits are mult 2^(z c - shift) outside the list. g: the gradient scale. A row without a
  // distribution or with a bad list has NaN throughout, one that needs a remainder and has none of it
  // (FORWARD_TAIL, nothing outside with mass) an infinite loss.
  __device__ __forceinline__ void stats(Part p, float c, float g, float& shift, float& mult) {
    pm = p.m;
    tau_c = c;
    float S = p.s;
    if constexpr (TAIL) {
      rest_m = p.m;
      rest_s = p.s;
      rest_inv = 1.f / rest_s;
      pm = max_nan(pm, shift_of(z_max, c));  // to the largest of all logits
      if (p.m != -INFINITY) p.s *= ex2(p.m - pm);
      p.m = pm;
      cz = scale_at(pm, c);
      float se = 0.f;
#pragma unroll 4
      for (int k = lane; k < padded; k += 32) {
        const float t = fmaf(en.z[k], cz, -pm);
        en.z[k] = t;
        if (en.tok[k] != -1) se += ex2(t);
      }
      S = p.s + warp_sum(se);
    }
    if (!TAIL) cz = scale_at(pm, c);
    unit = unit_at(pm, c);
    ok = !bad && fabsf(p.m) < INFINITY && S > 0.f && S < INFINITY;
    inv = 1.f / S;
    pr = TAIL ? p.s * inv : 0.f;
    sum = S;
    if constexpr (KIND == GRPO_DISTILL_FORWARD_TOPK) {
      alpha = q_all;
    } else if constexpr (KIND == GRPO_DISTILL_FORWARD_TAIL) {
      if (rest_m - pm < -126.f && q_rest < kTailNone) {
        q_all -= q_rest;
        q_rest = 0.f;
      }
      alpha = rest_m != -INFINITY ? fmaf(q_all, pr, -q_rest) : q_rest > 0.f ? -INFINITY : 0.f;
    } else {
      l2s = log2f(S);
      sum_loss();
      const bool tail = pr > 0.f && n < V && n > 0;
      const float fr = tail ? logf(pr / q_rest) : 0.f;
      if (tail) loss = fmaf(pr, fr, loss);
      alpha = tail ? fr - loss : 0.f;
    }
    if (!ok) alpha = __int_as_float(0x7fc00000);
    shift = ok ? p.m : 0.f;
    mult = ok ? alpha * g * inv : alpha;
    if (KIND == GRPO_DISTILL_FORWARD_TAIL && ok && rest_m != -INFINITY) {
      shift = rest_m;
      mult = alpha * g * rest_inv;
    }
  }

  // The student's probability of entry k.
  __device__ __forceinline__ float share(int k) const { return en.tok[k] != -1 ? ex2(en.z[k]) * inv : 0.f; }

  // The list's terms of the loss.
  __device__ __forceinline__ void sum_loss() {
    float part = 0.f;
#pragma unroll 4
    for (int k = lane; k < padded; k += 32) {
      const float lp = fmaf(en.z[k], unit, -l2s) * kLn2;
      if (KIND == GRPO_DISTILL_REVERSE_TAIL) {
        const float pk = share(k);
        part += pk > 0.f ? pk * (lp - en.tlp[k]) : 0.f;
      } else {
        const float q = en.q[k];
        part += q > 0.f ? q * ((en.tlp[k] - log_norm) - lp) : 0.f;  // (q = 0 without a token)
      }
    }
    loss = warp_sum(part);
  }

  // The token's loss (after stats, which does what the other warps wait for).
  __device__ __forceinline__ float token_loss(float g, bool& finite) {
    if constexpr (KIND != GRPO_DISTILL_REVERSE_TAIL) {
      l2s = log2f(sum);
      if (!TAIL)
        for (int k = lane; k < padded; k += 32) en.z[k] = fmaf(en.z[k], cz, -pm);
      sum_loss();
      // the quotient where p_R is far from the end of the range: the logarithms of the sums cancel
      if (KIND == GRPO_DISTILL_FORWARD_TAIL && q_rest > 0.f) {
        if (pr > 0x1p-100f) {
          loss += q_rest * logf(q_rest / pr);
        } else {
          // m_R - m, exact where both have the far scale
          const float gap =
              is_far(pm) && is_far(rest_m) ? (rest_m - pm) * unit : rest_m * unit_at(rest_m, tau_c) - pm * unit;
          loss += q_rest * (logf(q_rest) - (gap + (log2f(rest_s) - l2s)) * kLn2);
        }
      }
    }
    if (!ok) loss = __int_as_float(0x7fc00000);
    finite = isfinite(loss) && isfinite(alpha * g);
    return loss;
  }

  // dlogits of entry k (after token_loss).
  __device__ __forceinline__ float entry_grad(int k, float g) const {
    const float pk = share(k);
    float corr;
    if (KIND == GRPO_DISTILL_FORWARD_TOPK)
      corr = q_all != 0.f ? pk - en.q[k] : 0.f;
    else if (KIND == GRPO_DISTILL_FORWARD_TAIL)
      corr = fmaf(q_all, pk, -en.q[k]);
    else
      corr = pk > 0.f ? pk * ((fmaf(en.z[k], unit, -l2s) * kLn2 - en.tlp[k]) - loss) : 0.f;
    return ok ? corr * g : __int_as_float(0x7fc00000);
  }
};

}  // namespace distill
}  // namespace grpo
