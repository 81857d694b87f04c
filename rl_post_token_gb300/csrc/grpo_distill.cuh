#pragma once
// Distillation from a teacher's top tokens: the arithmetic of one token, shared by the row kernel
// and the LM-head variant. With the student's p = softmax(z/tau), the teacher's list S of
// (token i_k, log q_k), Q = sum q_k, P = sum_S p, q_R = 1 - Q and p_R = 1 - P:
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
#include "grpo_common.cuh"

namespace grpo {
namespace distill {

// A teacher remainder below 2^-24 cannot be told from the rounding of its float32 log-probs:
// FORWARD_TAIL counts it as none, REVERSE_TAIL takes this value in its logarithm.
constexpr double kTailMin = 5.9604644775390625e-08;

// What the slots of one token need of the teacher's whole list.
struct Teacher {
  float log_norm;  // FORWARD_TOPK: log Q; 0 otherwise
  float q_rest;    // q_R (tail kinds), floored as above; 0 where nothing lies outside the list
  float q_all;     // FORWARD_TAIL: Q + q_R
};

}  // namespace distill
}  // namespace grpo
