#pragma once
// Epilogues of the softmax cross entropy from hidden states (included by grpo_lmhead_gemm.cuh, whose
// kernel they belong to). Per token with x = h W^T, z = x or c tanh(x / c), lse = ln sum_v e^z_v:
//
//   L         = (1 - eps) (lse - z_y) + eps (lse - mean_v z_v) + lambda lse^2
//   dL/dx_v   = ((1 + 2 lambda lse) p_v - (1 - eps) [v = y] - eps / V) (1 - (z_v / c)^2)
//
// A tile's epilogue must end before the next tile's products (256 x 256 x H on a pair of SMs: about 9 H
// clocks; with the cap the epilogue is the longer one below H = 2000 or so); per element it takes one exponential
// and, with the cap, another and a reciprocal. Eight warps share it, two to each quarter of the accumulator's
// lanes: `half` is the columns' half that is a warp's.

namespace grpo {
namespace lmhead {

__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// t = tanh(u) and d = 1 - t^2. For |u| <= 1 the fifth convergent of Lambert's continued fraction,
// u (945 + 105 u^2 + u^4) / (945 + 420 u^2 + 15 u^4), off by less than 7e-8 of its value there (the
// exponential's form would lose the leading bits of a small u to cancellation); above it
// e = exp(2 |u|), t = 1 - 2 / (1 + e), d = 4 e / (1 + e)^2. The exponent stops at 127: the reciprocal is
// flushed to 0 there, so that t is 1 and d is 0 (they are within 2^-124 of it).
__device__ __forceinline__ void tanh_pair(float u, float& t, float& d) {
  // (explicit roundings: the bits of soft_cap32's packed form, whatever the compiler would contract)
  const float a = fabsf(u), q = __fmul_rn(u, u);
  const bool small = a <= 1.f;
  const float w = a * (2.f * kLog2e);
  const float e = ex2(w > 127.f ? 127.f : w);  // a NaN stays one
  const float r = rcp_approx(small ? fmaf(q, fmaf(q, 15.f, 420.f), 945.f) : 1.f + e);
  const float ts = __fmul_rn(__fmul_rn(u, fmaf(q, __fadd_rn(q, 105.f), 945.f)), r);
  const float tl = copysignf(fmaf(-2.f, r, 1.f), u);
  t = small ? ts : tl;
  d = small ? fmaf(-ts, ts, 1.f) : 4.f * (e * r) * r;
}

// tanh_pair of 32 logits x / c: z = c t in v, d in dz. Where no |x / c| of the warp's rows is above 1 -- the
// cap's ordinary range -- by the convergent alone, two at a time. An infinite x, which the cap would make an
// ordinary c, becomes NaN (x - x): its token counts as non-finite.
template <bool DERIV>
__device__ __forceinline__ void soft_cap32(float (&v)[32], float (&dz)[DERIV ? 32 : 1], float cap, float inv_cap) {
  float top = 0.f;
#pragma unroll
  for (int i = 0; i < 32; ++i) top = fmaxf(top, fabsf(v[i]));
  if (__all_sync(0xffffffffu, top * inv_cap <= 1.f)) {  // (a NaN logit stays one either way)
    const float2 k = make_float2(inv_cap, inv_cap), c0 = make_float2(945.f, 945.f);
#pragma unroll
    for (int i = 0; i < 32; i += 2) {
      const float2 u = __fmul2_rn(make_float2(v[i], v[i + 1]), k), q = __fmul2_rn(u, u);
      const float2 den = __ffma2_rn(q, __ffma2_rn(q, make_float2(15.f, 15.f), make_float2(420.f, 420.f)), c0);
      const float2 num = __fmul2_rn(u, __ffma2_rn(q, __fadd2_rn(q, make_float2(105.f, 105.f)), c0));
      const float2 t = __fmul2_rn(num, make_float2(rcp_approx(den.x), rcp_approx(den.y)));
      if constexpr (DERIV) {
        const float2 d = __ffma2_rn(make_float2(-t.x, -t.y), t, make_float2(1.f, 1.f));
        dz[i] = d.x;
        dz[i + 1] = d.y;
      }
      v[i] = cap * t.x;
      v[i + 1] = cap * t.y;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      float t, d;
      tanh_pair(__fmul_rn(v[i], inv_cap), t, d);
      if constexpr (DERIV) dz[i] = d;
      v[i] = fmaf(cap, t, v[i] - v[i]);
    }
  }
}

// The tensor cores round a running sum towards zero at every accumulation (Fasi, Higham, Mikaitis, Pranesh,
// "Numerical behavior of NVIDIA tensor cores", 2021), which takes a share of it each time, so of a product of
// length K a share in proportion to K: in the mean over dense normal operands, centred or not, 0.79 (K = 256), 0.87,
// 0.93, 1.00 (4096), 1.03, 1.06 and 1.07 (32768) times 2^-30 K. Given back, gain = 2^-30 K: the log-probs of 512
// tokens, V = 60000, K = 2048, are then 3.6e-7 of their size from 64 bits, 1.1e-6 without it. A product that is
// exact (few entries that are not 0, or small integers) loses nothing, and the gain is then its error: it stops
// at 2^-17 (K = 8192), where it stays below 1e-5 of a logit, the bar of the log-probs, for those, and what it
// leaves of a dense one's share does up to K = 16384. (Below H = 1000, where the epilogue is the longer part of a
// tile, it costs 2%.)
constexpr int kGainMaxH = 8192;
__device__ __forceinline__ void give_back(float (&v)[32], float gain) {
  const float2 g = make_float2(gain, gain);
#pragma unroll
  for (int i = 0; i < 32; i += 2) {
    const float2 x = make_float2(v[i], v[i + 1]), r = __ffma2_rn(x, g, x);
    v[i] = r.x;
    v[i + 1] = r.y;
  }
}

// Gives a tile's accumulator back to the MMA issuer, once a warp has loaded its last columns: before it
// computes on them and stores. Both arrives release, as the other epilogues' do: the issuer's acquire then has
// all 32 lanes' accumulator loads before it, the other lanes' by way of __syncwarp.
struct AccRelease {
  uint32_t remote;  // the even CTA's barrier as a cluster address, or 0: `local`
  uint64_t* local;
  int lane;
  __device__ __forceinline__ void operator()() const {
    fence_before();
    __syncwarp();
    if (lane == 0) {
      if (remote)
        mbar_arrive_remote(remote);
      else
        mbar_arrive(local);
    }
  }
};

// 3-D TMA tile store, plain or as a float addition (every element gets one addition per launch: the order
// of the sums is that of the launches).
__device__ __forceinline__ void tma_store3d(const CUtensorMap* map, uint32_t src, int x, int y, int z, bool add) {
  if (add)
    asm volatile("cp.reduce.async.bulk.tensor.3d.global.shared::cta.add.tile.bulk_group [%0, {%2, %3, %4}], [%1];"
                 ::"l"(reinterpret_cast<uint64_t>(map)), "r"(src), "r"(x), "r"(y), "r"(z)
                 : "memory");
  else
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4}], [%1];"
                 ::"l"(reinterpret_cast<uint64_t>(map)), "r"(src), "r"(x), "r"(y), "r"(z)
                 : "memory");
}

// One staged box: lane's 64 bytes (32 bf16 or 16 floats of its row) in the 64-byte swizzle, then the store.
// `box` counts a warp's boxes over all its tiles: its BUFS (1 or 2) buffers are used in turn whatever a tile
// leaves out.
template <int BUFS>
__device__ __forceinline__ void put_box(const CUtensorMap* map, uint32_t stage_buf, uint32_t& box, int lane, const uint32_t (&w)[16], int x,
                                        int y, int z, bool add) {
  const uint32_t buf = stage_buf + (box++ & (BUFS - 1u)) * EPI_BUF_BYTES;
  if (lane == 0) bulk_wait_read<BUFS - 1>();  // the last store from this buffer has read it
  __syncwarp();
  const uint32_t rb = (buf + (uint32_t)lane * 64u) | ((uint32_t)((lane >> 1) & 3) << 4);
#pragma unroll
  for (int q = 0; q < 4; ++q)
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(rb ^ ((uint32_t)q << 4)), "r"(w[4 * q]),
                 "r"(w[4 * q + 1]), "r"(w[4 * q + 2]), "r"(w[4 * q + 3])
                 : "memory");
  fence_proxy_async_smem();
  __syncwarp();
  if (lane == 0) {
    tma_store3d(map, buf, x, y, z, add);
    bulk_commit();
  }
}

// Softmax partials of one 256-column tile, the sum of its logits (with label smoothing) and the target
// logit. The columns past the vocabulary count as -inf, and add nothing to the sum. The second half's warp
// hands its row's three numbers to the first's through `join` (its row's place there, one of two in turn);
// the two warps meet at named barrier `bar` once a tile, so that the place is written again only after the
// other has read it and met once more. With g.keep the products are stored too (map_c).
template <bool CAP>
__device__ __forceinline__ void epi_ce_partials(const GemmArgs& g, const CUtensorMap* map_c, uint32_t taddr, int64_t row,
                                                bool rok, int ct, int half, float* join, int bar, int64_t warp_row0,
                                                int64_t rows, uint32_t stage_buf, uint32_t& box, int lane,
                                                const AccRelease& release) {
  const int V = (int)g.V, c0 = ct * BN;
  const int64_t tok = (rok && g.row_idx) ? (int64_t)g.row_idx[row] : row;
  const int y = rok ? g.target[tok] : -1;
  MS acc{-INFINITY, 0.f};
  float zy = 0.f, zsum = 0.f;
  float2 odd = make_float2(0.f, 0.f);  // NaN once a logit is infinite: -inf would leave no trace in the sums
  bool got = false;
#pragma unroll 1
  for (int c = half * (BN / 64); c < (half + 1) * (BN / 64); ++c) {
    float v[32];
    tmem_ld32(taddr + c * 32, v);
    if (c == (half + 1) * (BN / 64) - 1) release();
    const int cb = c0 + c * 32;
    if (cb >= V) continue;  // warp-uniform
    give_back(v, g.gain);
    if (g.keep && warp_row0 < rows) {  // the logits without their cap, for the dlogits
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        if (cb + b * 16 >= V) break;
        uint32_t w[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) w[i] = __float_as_uint(v[b * 16 + i]);
        put_box<1>(map_c, stage_buf, box, lane, w, cb + b * 16, (int)warp_row0, 0, false);
      }
    }
    if constexpr (CAP) {
      float none[1];
      soft_cap32<false>(v, none, g.cap, g.inv_cap);
    } else {
      // (a column past the vocabulary is 0, or NaN with an infinite hidden state, whose logits are all non-finite)
#pragma unroll
      for (int i = 0; i < 32; i += 2) odd = __ffma2_rn(make_float2(v[i], v[i + 1]), make_float2(0.f, 0.f), odd);
    }
    const uint32_t k = (uint32_t)y - (uint32_t)cb;  // (a target outside the vocabulary meets no column below V)
    if (k < 32) {
      got = true;
#pragma unroll
      for (uint32_t i = 0; i < 32; ++i)
        if (i == k) zy = v[i];
    }
    if (cb + 32 > V) {  // warp-uniform
      if (g.part_s2) {
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < 32; ++i) s += i < V - cb ? v[i] : 0.f;
        zsum += s;
      }
#pragma unroll
      for (int i = 0; i < 32; ++i)
        if (i >= V - cb) v[i] = -INFINITY;
    } else if (g.part_s2) {
      float s[32];
#pragma unroll
      for (int i = 0; i < 32; ++i) s[i] = v[i];
      zsum += tree_sum<32>(s);
    }
    lazy_online2<32>(acc, v);
  }
  // (with an ordinary shift: the joining drops a sum whose shift is -inf, as that of a tile with nothing else is)
  const float bad = acc.s + (odd.x + odd.y);
  if (isnan(bad)) acc = MS{0.f, bad};
  if (got) g.zy[tok] = zy;
  if (half) {
    join[0] = acc.m;
    join[1] = acc.s;
    join[2] = zsum;
  }
  asm volatile("bar.sync %0, 64;" ::"r"(bar) : "memory");
  if (half) return;
  acc = ms2_combine(acc, MS{join[0], join[1]});
  if (rok) {
    g.part_m[(int64_t)ct * g.M + row] = acc.m;
    g.part_s[(int64_t)ct * g.M + row] = acc.s;
    if (g.part_s2) g.part_s2[(int64_t)ct * g.M + row] = zsum + join[2];
  }
}

// bf16 dlogits of one tile (with respect to x, without the uniform grad_scale), staged in shared memory and
// written by TMA stores as those of the policy loss (epi_dlogits). The products with W and h take them as
// bf16, the operands' type at the tensor cores' full rate: half a step (2^-8) per entry. grad_scale is
// applied to the float sums: an unlikely target's entry is then next to -1 and loses nothing, where scaled
// by 1/N every such entry would be rounded the same way (0.3% of the gradients' length at N = 4117).
template <bool CAP>
__device__ __forceinline__ void epi_ce_dlogits(const GemmArgs& g, const CUtensorMap* map_c, uint32_t taddr,
                                               int64_t row, bool rok, int ct, int half, int64_t warp_row0,
                                               int64_t rows_store, uint32_t stage_buf, uint32_t& box, int lane,
                                               const AccRelease& release) {
  const int V = (int)g.V, c0 = ct * BN;
  const int64_t tok = (rok && g.row_idx) ? (int64_t)g.row_idx[row] : row;
  const int y = rok ? g.target[tok] : -1;
  const float sw = rok ? g.coef[tok] : 0.f;  // w
  const float l2 = rok ? g.lse2[tok] : 0.f, cp = rok ? g.ea[tok] : 0.f;
  const float ce = sw * g.ce_smooth, cy = sw * g.ce_hot;
  const bool live = sw != 0.f;
  const uint32_t swz = (uint32_t)((lane >> 1) & 3);
#pragma unroll 1
  for (int c = half * (BN / 64); c < (half + 1) * (BN / 64); ++c) {
    float v[32];
    tmem_ld32(taddr + c * 32, v);
    if (c == (half + 1) * (BN / 64) - 1) release();
    const int cb = c0 + c * 32;
    // warp-uniform: past the vocabulary, or all 32 rows past the rows to be written
    if (cb >= V || warp_row0 >= rows_store) continue;
    uint32_t w[16];
    if (__any_sync(0xffffffffu, live)) {
      const uint32_t k = (uint32_t)y - (uint32_t)cb;
      give_back(v, g.gain);
      float d[CAP ? 32 : 1];
      if constexpr (CAP) soft_cap32<true>(v, d, g.cap, g.inv_cap);
#pragma unroll
      for (int i = 0; i < 32; i += 2) {
        const float2 p = __ffma2_rn(make_float2(cp, cp), ex2_pair(v[i], v[i + 1], l2), make_float2(-ce, -ce));
        v[i] = p.x;
        v[i + 1] = p.y;
      }
      if (k < 32) {
#pragma unroll
        for (uint32_t i = 0; i < 32; ++i)
          if (i == k) v[i] -= cy;
      }
      if constexpr (CAP) {
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] *= d[i];
      }
#pragma unroll
      for (int i = 0; i < 16; ++i) w[i] = live ? pack_bf16x2(v[2 * i], v[2 * i + 1]) : 0u;
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i) w[i] = 0u;
    }
    const uint32_t buf = stage_buf + (box++ & 1u) * EPI_BUF_BYTES;
    if (lane == 0) bulk_wait_read<1>();  // the store before the last, from this buffer, has read it
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

// One output tile of d_h (its float sums: rows are compact, run `run` the map's third extent) or dW: the
// product times `scale`, as float or, rounded once, bf16. The map's extents clip the rows and columns.
__device__ __forceinline__ void epi_ce_store(const CUtensorMap* map, uint32_t taddr, int64_t warp_row0, int64_t M, int64_t N,
                                             int n0, int run, int half, float scale, bool bf16, bool add, uint32_t buf,
                                             uint32_t& box, int lane, const AccRelease& release) {
#pragma unroll 1
  for (int c = half * (BN / 64); c < (half + 1) * (BN / 64); ++c) {
    float v[32];
    tmem_ld32(taddr + c * 32, v);
    if (c == (half + 1) * (BN / 64) - 1) release();
    const int col = n0 + c * 32;
    if (col >= N || warp_row0 >= M) continue;  // warp-uniform
    uint32_t w[16];
    if (bf16) {
#pragma unroll
      for (int i = 0; i < 16; ++i) w[i] = pack_bf16x2(v[2 * i] * scale, v[2 * i + 1] * scale);
      put_box<2>(map, buf, box, lane, w, col, (int)warp_row0, run, false);
    } else {
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        if (col + b * 16 >= N) break;
#pragma unroll
        for (int i = 0; i < 16; ++i) w[i] = __float_as_uint(v[b * 16 + i] * scale);
        put_box<2>(map, buf, box, lane, w, col + b * 16, (int)warp_row0, run, add);
      }
    }
  }
}

}  // namespace lmhead
}  // namespace grpo
