#pragma once
// Epilogues of the softmax cross entropy from hidden states (included by grpo_lmhead_gemm.cuh, whose
// kernel they belong to). Per token with x = h W^T, z = x or c tanh(x / c), lse = ln sum_v e^z_v:
//
//   L         = (1 - eps) (lse - z_y) + eps (lse - mean_v z_v) + lambda lse^2
//   dL/dx_v   = ((1 + 2 lambda lse) p_v - (1 - eps) [v = y] - eps / V) (1 - (z_v / c)^2)
//
// A tile's epilogue must end before the next tile's products (256 x 256 x H: 4 H clocks of the tensor
// pipe); per element it takes one exponential and, with the cap, one or two more and a reciprocal.

namespace grpo {
namespace lmhead {

__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// t = tanh(u) and d = 1 - t^2. For |u| <= 1 the fifth convergent of Lambert's continued fraction,
// u (945 + 105 u^2 + u^4) / (945 + 420 u^2 + 15 u^4), off by less than 6e-8 of its value there (the
// exponential's form would lose the leading bits of a small u to cancellation); above it
// e = exp(2 |u|), t = 1 - 2 / (1 + e), d = 4 e / (1 + e)^2. The exponent stops at 127: the reciprocal is
// flushed to 0 there, so that t is 1 and d is 0 (they are within 2^-124 of it).
__device__ __forceinline__ void tanh_pair(float u, float& t, float& d) {
  const float a = fabsf(u), q = u * u;
  const bool small = a <= 1.f;
  const float w = a * (2.f * kLog2e);
  const float e = ex2(w > 127.f ? 127.f : w);  // a NaN stays one
  const float r = rcp_approx(small ? fmaf(q, fmaf(q, 15.f, 420.f), 945.f) : 1.f + e);
  const float ts = u * fmaf(q, q + 105.f, 945.f) * r;
  const float tl = copysignf(fmaf(-2.f, r, 1.f), u);
  t = small ? ts : tl;
  d = small ? fmaf(-ts, ts, 1.f) : 4.f * (e * r) * r;
}

// Softmax partials of one 256-column tile, the sum of its logits (with label smoothing) and the target
// logit. The columns past the vocabulary count as -inf, and add nothing to the sum.
template <bool CAP>
__device__ __forceinline__ void epi_ce_partials(const GemmArgs& g, uint32_t taddr, int64_t row, bool rok, int ct) {
  const int64_t c0 = (int64_t)ct * BN;
  const int64_t tok = (rok && g.row_idx) ? (int64_t)g.row_idx[row] : row;
  const int32_t y = rok ? g.target[tok] : -1;
  const bool own = y >= c0 && y < c0 + BN;
  MS acc{-INFINITY, 0.f};
  float zy = 0.f, zsum = 0.f;
#pragma unroll 1
  for (int c = 0; c < BN / 32; ++c) {
    float v[32];
    tmem_ld32(taddr + c * 32, v);
    const int64_t cb = c0 + c * 32;
    if (cb >= g.V) continue;  // warp-uniform
    if constexpr (CAP) {
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        float t, d;
        tanh_pair(v[i] * g.inv_cap, t, d);
        v[i] = g.cap * t;
      }
    }
    if (own && y >= cb && y < cb + 32) {
#pragma unroll
      for (int i = 0; i < 32; ++i)
        if (cb + i == y) zy = v[i];
    }
    const bool tail = cb + 32 > g.V;
    if (g.part_s2) {
      float s[32];
#pragma unroll
      for (int i = 0; i < 32; ++i) s[i] = !tail || cb + i < g.V ? v[i] : 0.f;
      zsum += tree_sum<32>(s);
    }
    if (tail) {
#pragma unroll
      for (int i = 0; i < 32; ++i)
        if (cb + i >= g.V) v[i] = -INFINITY;
    }
    lazy_online2<32>(acc, v);
  }
  if (rok) {
    g.part_m[(int64_t)ct * g.M + row] = acc.m;
    g.part_s[(int64_t)ct * g.M + row] = acc.s;
    if (g.part_s2) g.part_s2[(int64_t)ct * g.M + row] = zsum;
    if (own) g.zy[tok] = zy;
  }
}

// bf16 dlogits of one tile (with respect to x), staged in shared memory and written by TMA stores as
// those of the policy loss (epi_dlogits). The products with W and h take them as bf16: the operands'
// type of the tensor cores at their full rate, half a step (2^-9 of the largest of a binade) per entry.
template <bool CAP>
__device__ __forceinline__ void epi_ce_dlogits(const GemmArgs& g, const CUtensorMap* map_c, uint32_t taddr,
                                               int64_t row, bool rok, int ct, int64_t warp_row0, int64_t rows_store,
                                               uint32_t stage_buf, int lane) {
  const int64_t c0 = (int64_t)ct * BN;
  const int64_t tok = (rok && g.row_idx) ? (int64_t)g.row_idx[row] : row;
  const int32_t y = rok ? g.target[tok] : -1;
  const float sw = rok ? g.coef[tok] : 0.f;  // s w
  const float l2 = rok ? g.lse2[tok] : 0.f, cp = rok ? g.ea[tok] : 0.f;
  const float ce = sw * g.ce_smooth, cy = sw * g.ce_hot;
  const bool live = sw != 0.f;
  const uint32_t swz = (uint32_t)((lane >> 1) & 3);
#pragma unroll 1
  for (int c = 0; c < BN / 32; ++c) {
    float v[32];
    tmem_ld32(taddr + c * 32, v);
    const int64_t cb = c0 + c * 32;
    // warp-uniform: past the vocabulary, or all 32 rows past the rows to be written
    if (cb >= g.V || warp_row0 >= rows_store) continue;
    uint32_t w[16];
    if (live) {
      const bool hit = y >= cb && y < cb + 32;
      if constexpr (CAP) {
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          float t, d;
          tanh_pair(v[i] * g.inv_cap, t, d);
          const float p = ex2(fmaf(g.cap * t, kLog2e, -l2));
          v[i] = (fmaf(cp, p, -ce) - (cb + i == y ? cy : 0.f)) * d;
        }
      } else {
#pragma unroll
        for (int i = 0; i < 32; i += 2) {
          const float2 p = ex2_pair(v[i], v[i + 1], l2);
          v[i] = fmaf(cp, p.x, -ce);
          v[i + 1] = fmaf(cp, p.y, -ce);
        }
        if (hit) {
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (cb + i == y) v[i] -= cy;
        }
      }
#pragma unroll
      for (int i = 0; i < 16; ++i) w[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i) w[i] = 0u;
    }
    const uint32_t buf = stage_buf + (uint32_t)(c & 1) * EPI_BUF_BYTES;
    if (lane == 0) bulk_wait_read<1>();  // the store issued from this buffer two groups ago has read it
    __syncwarp();
    const uint32_t rb = buf + (uint32_t)lane * 64u;
#pragma unroll
    for (int q = 0; q < 4; ++q)
      asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(rb + (((uint32_t)q ^ swz) << 4)), "r"(w[4 * q]),
                   "r"(w[4 * q + 1]), "r"(w[4 * q + 2]), "r"(w[4 * q + 3])
                   : "memory");
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) {
      tma_store2d(map_c, buf, (int)(cb - g.v0), (int)warp_row0);
      bulk_commit();
    }
  }
}

// One output tile of d_h or dW: out[row][n0 .. n0 + 256) = (add ? add : 0) + D as float or, rounded once,
// bf16; with g.C set, the float sums of run `run` to it instead (g.accumulate: added to it). Columns past N are skipped (N is a
// multiple of 8). The shared-memory transposition of epi_store_f32: a warp's access covers 4 rows.
__device__ __forceinline__ void epi_ce_store(const GemmArgs& g, int run, uint32_t taddr, int64_t row, bool rok,
                                             int64_t n0, uint32_t buf, int lane) {
  float* part = g.C ? g.C + run * g.split_stride : nullptr;
  const float* add = part ? (g.accumulate ? part : nullptr) : g.add;
  // the row of out (d_h over the compact tokens: the token's), -1 past the rows
  const int crow = !rok ? -1 : g.row_idx && !part ? g.row_idx[row] : (int)row;
  const int64_t row0 = row - lane;
  const uint32_t put = buf + (uint32_t)lane * 128u, sw = (uint32_t)(lane & 7);
#pragma unroll 1
  for (int c = 0; c < BN / 32; ++c) {
    float v[32];
    tmem_ld32(taddr + c * 32, v);
    const int64_t col = n0 + c * 32;
    if (col >= g.N) continue;  // warp-uniform
    __syncwarp();              // the group before has been read
#pragma unroll
    for (int q = 0; q < 8; ++q)
      asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(put + (((uint32_t)q ^ sw) << 4)), "f"(v[4 * q]),
                   "f"(v[4 * q + 1]), "f"(v[4 * q + 2]), "f"(v[4 * q + 3])
                   : "memory");
    __syncwarp();
    const int64_t at = col + (lane & 7) * 4;  // lane: columns at .. at + 3 of rows lane / 8 + 4 i
    const bool in = at < g.N;
    float4 o[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      o[i] = make_float4(0.f, 0.f, 0.f, 0.f);
      const int64_t r = i * 4 + (lane >> 3);
      const bool on = __shfl_sync(0xffffffffu, crow, (int)r) >= 0 && in;
      if (add && on) o[i] = *reinterpret_cast<const float4*>(add + (row0 + r) * g.ldc + at);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int r = i * 4 + (lane >> 3), cr = __shfl_sync(0xffffffffu, crow, r);
      float4 d;
      asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                   : "=f"(d.x), "=f"(d.y), "=f"(d.z), "=f"(d.w)
                   : "r"(buf + (uint32_t)r * 128u + (((uint32_t)(lane & 7) ^ (uint32_t)(r & 7)) << 4))
                   : "memory");
      if (cr < 0 || !in) continue;
      const int64_t to = cr * g.ldc + at;
      d = make_float4(o[i].x + d.x, o[i].y + d.y, o[i].z + d.z, o[i].w + d.w);
      if (part)
        *reinterpret_cast<float4*>(part + to) = d;
      else if (g.out_bf16)
        *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(g.out) + to) =
            make_uint2(pack_bf16x2(d.x, d.y), pack_bf16x2(d.z, d.w));
      else
        *reinterpret_cast<float4*>(static_cast<float*>(g.out) + to) = d;
    }
  }
}

}  // namespace lmhead
}  // namespace grpo
