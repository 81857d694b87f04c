#pragma once
// Host side shared by the LM-head entry points: the operands' tensor maps, the persistent launch of a
// GEMM instance, and the backward's second stream.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <cstdlib>
#include <mutex>

#include "grpo_lmhead_gemm.cuh"

namespace grpo {
namespace lmhead {

inline PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  });
  return fn;
}

// bf16 matrix [outer][ld] of which [outer][inner] is addressed, box {64, box_outer}, 128-byte
// swizzle; reads past either extent return zeros.
inline bool make_map(CUtensorMap* m, const void* base, uint64_t inner, uint64_t outer, uint64_t ld, uint32_t box_outer) {
  auto fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[2] = {inner, outer};
  cuuint64_t strides[1] = {ld * 2};
  cuuint32_t box[2] = {(cuuint32_t)BK, box_outer};
  cuuint32_t estr[2] = {1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The dlogits chunk buffer [T][ld] as a TMA store target: the chunk's vc columns, box 32 x 32,
// 64-byte swizzle (the epilogue's staging layout).
inline bool map_dz_store(CUtensorMap* m, const void* base, int64_t T, int64_t vc, int64_t ld) {
  auto fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[2] = {(cuuint64_t)vc, (cuuint64_t)T};
  cuuint64_t strides[1] = {(cuuint64_t)ld * 2};
  cuuint32_t box[2] = {(cuuint32_t)EPI_BOX, (cuuint32_t)EPI_BOX};
  cuuint32_t estr[2] = {1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Operand maps. K-major [rows][K]: box {64 K, box_rows rows}. MN-major [K][MN]: box {64 MN, 64 K}.
inline bool map_k(CUtensorMap* m, const void* base, int64_t rows, int64_t k, int64_t ld, int box_rows) {
  return make_map(m, base, (uint64_t)k, (uint64_t)rows, (uint64_t)ld, (uint32_t)box_rows);
}
inline bool map_mn(CUtensorMap* m, const void* base, int64_t k, int64_t mn, int64_t ld) {
  return make_map(m, base, (uint64_t)mn, (uint64_t)k, (uint64_t)ld, 64u);
}

// CTAs per tile: 2 (paired MMA, the default) or 1 (GRPO_LMHEAD_CTA_GROUP=1, kept for comparison).
inline int cta_group() {
  const char* e = getenv("GRPO_LMHEAD_CTA_GROUP");
  return (e && e[0] == '1') ? 1 : 2;
}

// One persistent launch of `units` work units on clusters of CG CTAs. The first launch of an instance on a
// device sets its shared-memory limit and caches how many CTAs (or CTA pairs) fit at once.
// pdl: launched while the kernel before it on the stream still runs; the kernel itself waits (pdl_wait).
template <int CG, typename S, auto* kern, typename... Args>
int launch_units(int64_t units, cudaStream_t st, bool pdl, const Args&... args) {
  int dev = 0;
  GRPO_CUDA_TRY(cudaGetDevice(&dev));
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  int n_attr = 0;
  if (CG == 2) {
    attr[n_attr].id = cudaLaunchAttributeClusterDimension;
    attr[n_attr].val.clusterDim.x = CG;
    attr[n_attr].val.clusterDim.y = 1;
    attr[n_attr++].val.clusterDim.z = 1;
  }
  cfg.blockDim = dim3(S::THREADS, 1, 1);
  cfg.dynamicSmemBytes = S::SMEM;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = n_attr;
  int max_units = 0;
  {
    static std::mutex mu;
    static int cached[64] = {};
    std::lock_guard<std::mutex> lock(mu);
    if (dev >= 0 && dev < 64) max_units = cached[dev];
    if (max_units == 0) {
      GRPO_CUDA_TRY(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)S::SMEM));
      if (CG == 2) {
        cfg.gridDim = dim3(2 * 1024, 1, 1);
        GRPO_CUDA_TRY(cudaOccupancyMaxActiveClusters(&max_units, kern, &cfg));
      } else {
        max_units = sm_count();
      }
      if (max_units < 1) return GRPO_ERR_UNSUPPORTED;
      if (dev >= 0 && dev < 64) cached[dev] = max_units;
    }
  }
  units = std::min<int64_t>(units, max_units);
  if (units <= 0) return GRPO_OK;
  cfg.gridDim = dim3((unsigned)(CG * units), 1, 1);
  if (pdl) {
    attr[n_attr].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[n_attr++].val.programmaticStreamSerializationAllowed = 1;
    cfg.numAttrs = n_attr;
  }
  GRPO_CUDA_TRY(cudaLaunchKernelEx(&cfg, kern, args...));
  return GRPO_OK;
}

// One persistent launch over g's units.
template <int CG, int EPI, bool AMN, bool BMN>
int launch_t(const CUtensorMap& ma, const CUtensorMap& mb, const CUtensorMap& mc, GemmArgs g, cudaStream_t st,
             bool pdl) {
  g.n_m = (int)((g.M + BM * CG - 1) / (BM * CG));
  return launch_units<CG, Shape<CG, EPI>, &gemm_kernel<CG, EPI, AMN, BMN>>((int64_t)g.n_m * g.n_n, st, pdl, ma, mb, mc, g);
}

// mc: the TMA store target of the dlogits epilogue (unused by the other epilogues)
template <int EPI, bool AMN, bool BMN>
int launch(int cg, const CUtensorMap& ma, const CUtensorMap& mb, const CUtensorMap& mc, const GemmArgs& g,
           cudaStream_t st, bool pdl = false) {
  return cg == 2 ? launch_t<2, EPI, AMN, BMN>(ma, mb, mc, g, st, pdl) : launch_t<1, EPI, AMN, BMN>(ma, mb, mc, g, st, pdl);
}

// Vocabulary tiles per backward chunk: at most 66 (16896 columns), the chunks of equal width
// (V = 151936 -> 594 tiles -> 9 chunks of 66).
constexpr int kMaxChunkTiles = 66;

// The backward's second stream and its events, one set per device, created by the first call
// that needs them (with the device current) and kept for the process lifetime. A call holds
// `lock` while it enqueues its backward, so calls from several host threads never interleave
// their records of these events; their work on the shared stream runs in enqueue order.
struct Overlap {
  cudaStream_t aux = nullptr;
  cudaEvent_t dz_ready = nullptr, joined = nullptr, buf_free[2] = {nullptr, nullptr};
};

// Whether the next chunk's recompute may run beside this chunk's d_h and dW
// (GRPO_LMHEAD_OVERLAP=0 keeps every launch on the caller's stream).
inline bool overlap_on() {
  const char* e = getenv("GRPO_LMHEAD_OVERLAP");
  return !(e && e[0] == '0');
}

// Whether launches for `st` may go to the second stream: not while a capture that is not st's own holds
// it (a call of another thread, between its end and its graph's end). Calls then keep to one stream.
inline bool overlap_free(cudaStream_t aux, cudaStream_t st) {
  cudaStreamCaptureStatus a, b;
  unsigned long long ia = 0, ib = 0;
  if (cudaStreamGetCaptureInfo(aux, &a, &ia) != cudaSuccess || cudaStreamGetCaptureInfo(st, &b, &ib) != cudaSuccess) {
    (void)cudaGetLastError();
    return false;
  }
  return a == cudaStreamCaptureStatusNone || (b == cudaStreamCaptureStatusActive && ia == ib);
}

inline Overlap* overlap_state(std::unique_lock<std::mutex>& lock, cudaStream_t st) {
  static Overlap per_dev[64];
  static std::mutex mu;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) {
    (void)cudaGetLastError();
    return nullptr;
  }
  lock = std::unique_lock<std::mutex>(mu);
  Overlap& o = per_dev[dev];
  if (!o.aux) {
    Overlap n;
    const unsigned ef = cudaEventDisableTiming;
    if (cudaStreamCreateWithFlags(&n.aux, cudaStreamNonBlocking) != cudaSuccess ||
        cudaEventCreateWithFlags(&n.dz_ready, ef) != cudaSuccess ||
        cudaEventCreateWithFlags(&n.joined, ef) != cudaSuccess ||
        cudaEventCreateWithFlags(&n.buf_free[0], ef) != cudaSuccess ||
        cudaEventCreateWithFlags(&n.buf_free[1], ef) != cudaSuccess) {
      (void)cudaGetLastError();
      return nullptr;  // (what was created is kept until exit; the call falls back to one stream)
    }
    o = n;
  }
  return overlap_free(o.aux, st) ? &o : nullptr;
}

}  // namespace lmhead
}  // namespace grpo
