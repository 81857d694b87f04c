#pragma once
// Both gradient products of one vocabulary piece in one persistent launch:
//
//   d_h  (+)= dz W_c     [T, H], reduced over the piece's vc columns in `split` runs of K blocks
//   dW_c  =  dz^T h      [vc, H], reduced over the tokens
//
// on the tiles, ring and accumulators of grpo_lmhead_gemm.cuh (A = dz K-major or MN-major, B = W_c or h
// MN-major). One launch for both: alone, d_h has few tiles with a long reduction (16 tiles of 256 x 256 at
// 1024 tokens and H = 1024, for 76 pairs of SMs; 128 at 4096 and 2048, two rounds of which the second is 68%
// full), while dW's many short ones fill whatever is left.
#include "grpo_lmhead_gemm.cuh"

namespace grpo {
namespace lmhead {

struct BwdArgs {
  int64_t T, H, vc;
  int with_dh, with_dw, split;
  int a_rows;  // rows of dz that a d_h unit loads (see CeCall)
  int dh_accumulate, dw_accumulate, dw_bf16;
  float dw_scale;
  const int32_t* live_n;  // the unmasked tokens' count (compact rows), or NULL: T
  grpo_step_acc* acc;
};

struct BwdUnit {
  int dw, mu, nu, run, k0, k1;
};

// The units of worker p of P. d_h's units go round by round; the workers that the last round leaves out
// (from r1 on) take `lead` dW units each, about what a d_h unit takes, before the others join in.
struct BwdPlan {
  int n_nt, n_mu1, n1, n2, kb1, kb2, split, P, p, c1, r1, lead;

  __device__ __forceinline__ BwdPlan(const BwdArgs& a, int cg, int P_, int p_) : P(P_), p(p_) {
    const int64_t nl = a.live_n ? (int64_t)*a.live_n : a.T;
    n_nt = (int)((a.H + BN - 1) / BN);
    n_mu1 = (int)((nl + BM * cg - 1) / (BM * cg));
    split = a.split;
    kb1 = (int)((a.vc + BK - 1) / BK);
    kb2 = (int)((a.live_n ? live_pad(nl, a.T) : a.T) + BK - 1) / BK;
    n1 = a.with_dh ? n_mu1 * n_nt * split : 0;
    n2 = a.with_dw ? (int)((a.vc + BM * cg - 1) / (BM * cg)) * n_nt : 0;
    r1 = n1 % P;
    c1 = n1 / P + (p < r1 ? 1 : 0);
    lead = r1 == 0 ? 0 : (kb1 / split + kb2 / 2) / kb2;
  }

  __device__ __forceinline__ bool get(int k, BwdUnit& u) const {
    u.run = 0;
    u.k0 = 0;
    if (k < c1) {
      const int id = p + k * P;
      u.dw = 0;
      u.nu = id % n_nt;
      u.mu = id / n_nt % n_mu1;
      u.run = id / (n_nt * n_mu1);
      u.k0 = (int)((int64_t)u.run * kb1 / split);
      u.k1 = (int)((int64_t)(u.run + 1) * kb1 / split);
      return true;
    }
    int j = k - c1, id;
    const int nb = P - r1;
    if (p >= r1 && j < lead) {
      id = p - r1 + j * nb;
    } else {
      if (p >= r1) j -= lead;
      id = lead * nb + p + j * P;
    }
    if (id >= n2) return false;
    u.dw = 1;
    u.nu = id % n_nt;
    u.mu = id / n_nt;
    u.k1 = kb2;
    return true;
  }
};

template <int CG>
__global__ void __launch_bounds__(Shape<CG, EPI_CE_STORE>::THREADS, 1)
bwd_kernel(const __grid_constant__ CUtensorMap dz_k, const __grid_constant__ CUtensorMap w_mn,
           const __grid_constant__ CUtensorMap part, const __grid_constant__ CUtensorMap dz_mn,
           const __grid_constant__ CUtensorMap h_mn, const __grid_constant__ CUtensorMap dw, BwdArgs g) {
  using S = Shape<CG, EPI_CE_STORE>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t sbase = (smem_u32(smem_raw) + 1023u) & ~1023u;
  uint8_t* sgen = smem_raw + (sbase - smem_u32(smem_raw));
  const uint32_t epi_base = sbase + S::STAGES * S::STAGE_BYTES;
  uint64_t* full = reinterpret_cast<uint64_t*>(sgen + S::STAGES * S::STAGE_BYTES + S::EPI_BYTES);
  uint64_t* empty = full + S::STAGES;
  uint64_t* tfull = empty + S::STAGES;  // [2]
  uint64_t* tempty = tfull + 2;         // [2]
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(tempty + 2);
  volatile int* s_abort = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = CG == 2 ? cluster_ctarank() : 0u;
  if (threadIdx.x == 0) {
    for (int s = 0; s < S::STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&tfull[b], 1);
      mbar_init(&tempty[b], S::WARPS * CG);
    }
    *s_abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) tmem_alloc<CG>(smem_u32(tmem_slot));
  fence_before();
  __syncthreads();
  if (CG == 2) cluster_sync_all();
  fence_after();
  pdl_launch();
  pdl_wait();
  const uint32_t tmem = *tmem_slot;
  const BwdPlan plan(g, CG, (int)gridDim.x / CG, (int)blockIdx.x / CG);

  if (warp == 0) {
    // ---- TMA producer ----
    if (lane == 0) {
      const uint32_t full0 = CG == 2 ? mapa_u32(smem_u32(full), 0) : smem_u32(full);
      uint32_t stage = 0, phase = 0;
      BwdUnit u;
      for (int k = 0; plan.get(k, u); ++k) {
        const int a_row = u.mu * BM * CG + (int)rank * BM, b_row = u.nu * BN + (int)rank * S::B_ROWS;
        for (int kb = u.k0; kb < u.k1; ++kb) {
          if (!mbar_wait_bounded(&empty[stage], phase ^ 1u, s_abort)) break;
          if (rank == 0)
            mbar_arrive_expect_tx(&full[stage], u.dw ? CG * S::STAGE_BYTES : CG * (g.a_rows * BK * 2 + S::B_BYTES));
          const uint32_t sa = sbase + stage * S::STAGE_BYTES, bar = full0 + stage * 8u;
          if (u.dw) {
            load_operand<CG, true, BM>(sa, &dz_mn, bar, kb * BK, a_row);
            load_operand<CG, true, S::B_ROWS>(sa + S::A_BYTES, &h_mn, bar, kb * BK, b_row);
          } else {
            load_operand<CG, false, BM>(sa, &dz_k, bar, kb * BK, a_row);
            load_operand<CG, true, S::B_ROWS>(sa + S::A_BYTES, &w_mn, bar, kb * BK, b_row);
          }
          if (++stage == S::STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (*s_abort) break;  // a wait gave up: issue nothing more
      }
      // every stage's last release has arrived before this CTA may leave (see gemm_kernel)
      for (int i = 0; i < S::STAGES; ++i) {
        if (*s_abort)
          drain_wait(&empty[stage], phase ^ 1u);
        else
          mbar_wait_bounded(&empty[stage], phase ^ 1u, s_abort);
        if (++stage == S::STAGES) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
  } else if (warp == 1) {
    // ---- MMA issuer (the cluster's even CTA) ----
    if (lane == 0 && rank == 0) {
      uint32_t stage = 0, phase = 0, ab = 0, aphase = 0;
      auto products = [&](auto a_mn, uint32_t d, int k0, int k1) {
        constexpr bool A_MN = decltype(a_mn)::value;
        constexpr uint32_t ID = idesc<CG, A_MN, true>();
        for (int kb = k0; kb < k1; ++kb) {
          mbar_wait_bounded(&full[stage], phase, s_abort);  // (not tested for a break, see gemm_kernel)
          fence_after();
          const uint32_t sa = sbase + stage * S::STAGE_BYTES;
          const uint64_t da = sdesc<A_MN>(sa), db = sdesc<true>(sa + S::A_BYTES);
#pragma unroll
          for (int j = 0; j < BK / 16; ++j)
            mma_bf16<CG>(d, da + kstep<A_MN>() * j, db + kstep<true>() * j, ID, kb > k0 || j > 0);
          const uint32_t eb = smem_u32(&empty[stage]);
          mma_commit<CG>(eb);
          if (CG == 2) mma_commit<CG>(mapa_u32(eb, 1));
          if (++stage == S::STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
      };
      BwdUnit u;
      for (int k = 0; plan.get(k, u); ++k) {
        const bool free_acc = CG == 2 ? mbar_wait_cluster_bounded(&tempty[ab], aphase ^ 1u, s_abort)
                                      : mbar_wait_bounded(&tempty[ab], aphase ^ 1u, s_abort);
        if (!free_acc) break;
        fence_after();
        if (u.dw)
          products(std::true_type{}, tmem + ab * BN, u.k0, u.k1);
        else
          products(std::false_type{}, tmem + ab * BN, u.k0, u.k1);
        if (*s_abort) break;
        const uint32_t fb = smem_u32(&tfull[ab]);
        mma_commit<CG>(fb);
        if (CG == 2) mma_commit<CG>(mapa_u32(fb, 1));
        if (++ab == 2) {
          ab = 0;
          aphase ^= 1u;
        }
      }
    }
  } else {
    // ---- epilogue: thread = accumulator row, two warps to a lane quarter, each half of the columns ----
    const int quarter = warp & 3, half = (warp - 2) >> 2;
    const uint32_t buf = epi_base + (uint32_t)(half * 4 + quarter) * 2u * EPI_BUF_BYTES;
    const int64_t nl = g.live_n ? (int64_t)*g.live_n : g.T;
    uint32_t ab = 0, aphase = 0, box = 0;
    BwdUnit u;
    for (int k = 0; plan.get(k, u); ++k) {
      mbar_wait_bounded(&tfull[ab], aphase, s_abort);
      fence_after();
      const int64_t row0 = (int64_t)u.mu * BM * CG + (int64_t)rank * BM + quarter * 32;
      const uint32_t taddr = tmem + ((uint32_t)(quarter * 32) << 16) + ab * BN;
      const AccRelease release{CG == 2 && rank != 0 ? mapa_u32(smem_u32(&tempty[ab]), 0) : 0u, &tempty[ab], lane};
      if (u.dw)
        epi_ce_store(&dw, taddr, row0, g.vc, g.H, u.nu * BN, 0, half, g.dw_scale, g.dw_bf16, g.dw_accumulate, buf, box,
                     lane, release);
      else
        epi_ce_store(&part, taddr, row0, nl, g.H, u.nu * BN, u.run, half, 1.f, false, g.dh_accumulate, buf, box, lane,
                     release);
      if (++ab == 2) {
        ab = 0;
        aphase ^= 1u;
      }
    }
    if (lane == 0) bulk_wait_all();  // this warp's stores are complete
  }

  fence_before();
  __syncthreads();
  if (CG == 2) cluster_sync_all();  // neither CTA leaves while the other may still signal it
  if (*s_abort && threadIdx.x == 0) atomicOr(&g.acc->flags, kFlagWaitTimeout);
  if (warp == 1) {
    fence_after();
    tmem_dealloc<CG>(tmem);
  }
}

}  // namespace lmhead
}  // namespace grpo
