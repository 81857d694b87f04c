// The global norm of many gradient tensors, each tensor's own, and the clip: what stands between a step's
// finish and the optimizer ("Sizing mini-batches and micro-batches", "The hard part: deferred
// normalization": scale by 1/max(sum, 1), then clip, then step).
//
//   S_i = sum_j g_ij^2,  S = sum_i S_i,  norm = s sqrt(S),  factor = s min(1, max_norm / norm)
//   out_ij = factor g_ij
//
// Bound by memory: every element is read once for the norm, and read and written once by the clip, which
// cannot begin before the norm is known. A tensor is cut into chunks, a block each; the tensors' addresses
// and sizes travel in the kernel's parameters (no table in device memory, nothing to keep alive, and a
// captured call replays by itself).
#include <algorithm>
#include <cmath>
#include <cstdlib>

#include "grpo_common.cuh"

namespace grpo {
namespace clip {

constexpr int kThreads = 256;
constexpr int kVec = 8;               // elements a thread takes at a time
constexpr int64_t kMinChunk = 8192;   // elements of a chunk, at least: 32 a thread
constexpr int64_t kMaxChunks = 16384; // chunks of a call, about, at most: one block sums their partials
constexpr int kFold = 16;             // vectors a thread sums in float before it folds them into a double
constexpr int kFinalThreads = 1024;
constexpr int kSeg = 256;  // partials that a warp of the last kernel sums at a time
constexpr int kFew = 8;    // a tensor of at most so many chunks is summed by one thread

// The tensors of one launch. chunk0[i]: the first chunk of tensor i among the launch's, chunk0[n] their count.
template <int N>
struct Table {
  int32_t n;
  int32_t chunk0[N + 1];
  int64_t numel[N];
  const void* src[N];
  void* dst[N];       // (clip)
  uint8_t kind[N];    // bit 0: src is bf16, bit 1: dst is bf16
};

constexpr int32_t kMaxTensors = 1 << 24;
constexpr int kSmall = 32, kLarge = 512;  // tensors per launch: 1 KB and 17 KB of parameters

template <int N>
__device__ __forceinline__ int tensor_of(const Table<N>& t, int chunk) {
  int lo = 0, hi = t.n - 1;  // the last i with chunk0[i] <= chunk (tensors without elements have no chunk)
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (t.chunk0[mid] <= chunk)
      lo = mid;
    else
      hi = mid - 1;
  }
  return lo;
}

// (plain loads: the clip may run in place)
__device__ __forceinline__ void load8(const float* p, bool aligned, float (&v)[kVec]) {
  if (aligned) {
    const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  } else {
#pragma unroll
    for (int i = 0; i < kVec; ++i) v[i] = p[i];
  }
}

__device__ __forceinline__ void load8(const __nv_bfloat16* p, bool aligned, float (&v)[kVec]) {
  if (aligned) {
    const uint4 a = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = bf16_lo(w[i]);
      v[2 * i + 1] = bf16_hi(w[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < kVec; ++i) v[i] = __bfloat162float(p[i]);
  }
}

__device__ __forceinline__ double block_sum(double s, double* red) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  __syncthreads();
  if (lane == 0) red[warp] = s;
  __syncthreads();
  s = 0.0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) s += red[w];
  return s;
}

// The sum of the squares of n elements at p, the same in every thread. Thread t takes vectors t, t + 256, ..
// of 8 elements, in float up to 16 of them, then in double (a chain of 16 and a tree: 20 roundings of
// 2^-24 at most); the order goes by the index alone, whatever the address. A sum that may have left float's
// range -- above 2^120, not a number, or below 2^-80 with an element that is not 0 -- is formed once more
// in double, where no square over- or underflows.
template <typename T>
__device__ __forceinline__ double chunk_sum(const T* p, int64_t n, double* red) {
  const bool aligned = (reinterpret_cast<uintptr_t>(p) & 15u) == 0;
  const int64_t nv = n / kVec;
  double s = 0.0;
  uint32_t any = 0;
  for (int64_t v0 = threadIdx.x; v0 < nv; v0 += (int64_t)kFold * kThreads) {
    float a[kVec] = {};
#pragma unroll 4
    for (int k = 0; k < kFold; ++k) {
      const int64_t v = v0 + (int64_t)k * kThreads;
      if (v >= nv) break;
      float x[kVec];
      load8(p + v * kVec, aligned, x);
#pragma unroll
      for (int i = 0; i < kVec; ++i) {
        a[i] = fmaf(x[i], x[i], a[i]);
        any |= __float_as_uint(x[i]);
      }
    }
    s += (double)tree_sum<kVec, false>(a);
  }
  if (threadIdx.x < n - nv * kVec) {
    const float x = (float)p[nv * kVec + threadIdx.x];
    s += (double)(x * x);
    any |= __float_as_uint(x);
  }
  s = block_sum(s, red);
  if (s >= 8.271806125530277e-25 && s <= 1.329227995784916e36) return s;  // 2^-80 .. 2^120
  if (!__syncthreads_or((any & 0x7fffffffu) != 0)) return 0.0;
  s = 0.0;
  for (int64_t i = threadIdx.x; i < n; i += kThreads) {
    const double x = (double)(float)p[i];
    s = fma(x, x, s);
  }
  return block_sum(s, red);
}

template <int N>
__global__ void __launch_bounds__(kThreads) norm_kernel(const __grid_constant__ Table<N> t, int64_t chunk, double* part) {
  __shared__ double red[kThreads / 32];
  const int i = tensor_of(t, (int)blockIdx.x);
  const int64_t at = (int64_t)((int)blockIdx.x - t.chunk0[i]) * chunk;
  const int64_t n = t.numel[i] - at < chunk ? t.numel[i] - at : chunk;
  const double s = (t.kind[i] & 1) ? chunk_sum(static_cast<const __nv_bfloat16*>(t.src[i]) + at, n, red)
                                   : chunk_sum(static_cast<const float*>(t.src[i]) + at, n, red);
  if (threadIdx.x == 0) part[blockIdx.x] = s;
}

struct FinalArgs {
  const double* part;      // the launch's chunks
  const double* before;    // sum of the launches before, or NULL
  double* sum;             // out: with this launch's
  float* tensor_norms;     // this launch's tensors, or NULL
  const grpo_step_acc* acc;
  int32_t deferred, last;
  float max_norm;
  grpo_grad_norm_result* result;
};

// The launch's partials summed per tensor, the tensors' sums, and with the last launch the result. Tensors
// of a few chunks take a thread each; of the others a warp takes 256 chunks at a time (8 loads a lane in
// flight), whose sums one thread adds in order.
template <int N>
__global__ void __launch_bounds__(kFinalThreads) final_kernel(const __grid_constant__ Table<N> t, FinalArgs a) {
  constexpr int kSegs = (int)(kMaxChunks / kSeg) + 2 * N;  // (a call has at most kMaxChunks + n chunks)
  __shared__ double seg[kSegs], of[N], red[kFinalThreads / 32];
  __shared__ int seg0[N + 1];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  double s = 1.0;
  if (a.deferred) s = 1.0 / (double)(a.acc->divisor > 1 ? a.acc->divisor : 1);
  if (tid == 0) {
    int k = 0;
    for (int i = 0; i < t.n; ++i) {
      seg0[i] = k;
      const int c = t.chunk0[i + 1] - t.chunk0[i];
      k += c <= kFew ? 0 : (c + kSeg - 1) / kSeg;
    }
    seg0[t.n] = k;
  }
  __syncthreads();
  for (int i = tid; i < t.n; i += kFinalThreads) {
    const int c0 = t.chunk0[i], c = t.chunk0[i + 1] - c0;
    if (c > kFew) continue;
    double x[kFew], v = 0.0;
#pragma unroll
    for (int k = 0; k < kFew; ++k) x[k] = k < c ? a.part[c0 + k] : 0.0;
#pragma unroll
    for (int k = 0; k < kFew; ++k) v += x[k];
    of[i] = v;
  }
  for (int g = warp; g < seg0[t.n]; g += kFinalThreads / 32) {
    int lo = 0, hi = t.n - 1;  // the last tensor with seg0 <= g
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (seg0[mid] <= g)
        lo = mid;
      else
        hi = mid - 1;
    }
    const int c0 = t.chunk0[lo] + (g - seg0[lo]) * kSeg, c1 = min(c0 + kSeg, t.chunk0[lo + 1]);
    double x[kSeg / 32], v = 0.0;
#pragma unroll
    for (int k = 0; k < kSeg / 32; ++k) x[k] = c0 + k * 32 + lane < c1 ? a.part[c0 + k * 32 + lane] : 0.0;
#pragma unroll
    for (int k = 0; k < kSeg / 32; ++k) v += x[k];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (lane == 0) seg[g] = v;
  }
  __syncthreads();
  double v = 0.0;
  for (int i = tid; i < t.n; i += kFinalThreads) {
    if (t.chunk0[i + 1] - t.chunk0[i] > kFew) {
      double u = 0.0;
      for (int g = seg0[i]; g < seg0[i + 1]; ++g) u += seg[g];
      of[i] = u;
    }
    v += of[i];
    if (a.tensor_norms) a.tensor_norms[i] = (float)(s * sqrt(of[i]));
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (lane == 0) red[warp] = v;
  __syncthreads();
  if (tid != 0) return;
  double total = a.before ? *a.before : 0.0;
#pragma unroll
  for (int w = 0; w < kFinalThreads / 32; ++w) total += red[w];
  *a.sum = total;
  if (!a.last) return;
  grpo_grad_norm_result r;
  const double norm = s * sqrt(total);
  r.sum_sq = total;
  r.norm = (float)norm;
  r.status = a.acc ? a.acc->result.status : GRPO_OK;
  if (r.status == GRPO_OK && !isfinite(total)) r.status = GRPO_STEP_SKIPPED_NONFINITE;
  r.coef = r.status != GRPO_OK ? 0.f : (float)(norm > (double)a.max_norm ? s * ((double)a.max_norm / norm) : s);
  r.reserved0 = 0;
  r.reserved1 = 0;
  *a.result = r;
}

__device__ __forceinline__ void store8(float* p, const float (&v)[kVec]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&v)[kVec]) {
  *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                                            pack_bf16x2(v[6], v[7]));
}
__device__ __forceinline__ void put(float* p, float v) { *p = v; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// out = f g, rounded once to out's type; zeros, with nothing read, where the step is skipped.
template <typename S, typename D>
__device__ __forceinline__ void clip_chunk(const S* src, D* dst, int64_t n, float f, bool skip) {
  const bool aligned = ((reinterpret_cast<uintptr_t>(src) | reinterpret_cast<uintptr_t>(dst)) & 15u) == 0;
  int64_t done = 0;
  if (aligned) {
    const int64_t nv = n / kVec;
    done = nv * kVec;
#pragma unroll 4
    for (int64_t v = threadIdx.x; v < nv; v += kThreads) {
      float x[kVec] = {};
      if (!skip) load8(src + v * kVec, true, x);
#pragma unroll
      for (int i = 0; i < kVec; ++i) x[i] = skip ? 0.f : x[i] * f;
      store8(dst + v * kVec, x);
    }
  }
#pragma unroll 4
  for (int64_t i = done + threadIdx.x; i < n; i += kThreads) put(dst + i, skip ? 0.f : (float)src[i] * f);
}

template <int N>
__global__ void __launch_bounds__(kThreads) clip_kernel(const __grid_constant__ Table<N> t, int64_t chunk,
                                                        const grpo_grad_norm_result* result) {
  const int b = (int)(gridDim.x - 1 - blockIdx.x);  // from the end: what the norm has read last is still in L2
  const float f = result->coef;
  const bool skip = result->status != GRPO_OK;
  const int i = tensor_of(t, b);
  const int64_t at = (int64_t)(b - t.chunk0[i]) * chunk;
  const int64_t n = t.numel[i] - at < chunk ? t.numel[i] - at : chunk;
  if (t.src[i] == t.dst[i] && !skip && f == 1.f) return;  // in place, and the factor changes nothing
  const float* sf = static_cast<const float*>(t.src[i]) + at;
  const __nv_bfloat16* sb = static_cast<const __nv_bfloat16*>(t.src[i]) + at;
  float* df = static_cast<float*>(t.dst[i]) + at;
  __nv_bfloat16* db = static_cast<__nv_bfloat16*>(t.dst[i]) + at;
  switch (t.kind[i]) {
    case 0: clip_chunk(sf, df, n, f, skip); break;
    case 1: clip_chunk(sb, df, n, f, skip); break;
    case 2: clip_chunk(sf, db, n, f, skip); break;
    default: clip_chunk(sb, db, n, f, skip); break;
  }
}

// ---- host -------------------------------------------------------------------------------------

// Elements of a chunk, by the call's sizes alone (the order of the sums follows from it): a power of two
// that cuts the call into about 16384 chunks at most.
int64_t chunk_of(int64_t total) {
  int64_t c = kMinChunk;
  while (c * kMaxChunks < total) c *= 2;
  return c;
}

int check_list(const void* const* p, const int64_t* numels, const int32_t* dtypes, int32_t n, int64_t* total) {
  if (n < 0 || n > kMaxTensors || (n > 0 && (!p || !numels || !dtypes))) return GRPO_ERR_INVALID;
  *total = 0;
  for (int32_t i = 0; i < n; ++i) {
    if (dtypes[i] != GRPO_DTYPE_F32 && dtypes[i] != GRPO_DTYPE_BF16) return GRPO_ERR_UNSUPPORTED;
    const uintptr_t size = dtypes[i] == GRPO_DTYPE_BF16 ? 2 : 4;
    if (numels[i] < 0 || numels[i] > ((int64_t)1 << 48) || (numels[i] > 0 && (!p[i] || (uintptr_t)p[i] % size)))
      return GRPO_ERR_INVALID;
    *total += numels[i];
    if (*total > ((int64_t)1 << 48)) return GRPO_ERR_INVALID;
  }
  return GRPO_OK;
}

struct Span {
  uintptr_t lo, hi;
  int write;
};

// Whether a tensor that is written overlaps another that is read or written. A tensor clipped in place is
// one span. n > 0; spans: room for 2 n.
bool overlaps(const void* const* src, const int32_t* sd, void* const* dst, const int32_t* dd, const int64_t* numels,
              int32_t n, Span* spans) {
  int32_t m = 0;
  for (int32_t i = 0; i < n; ++i) {
    if (numels[i] == 0) continue;
    const uintptr_t d = (uintptr_t)dst[i], s = (uintptr_t)src[i];
    spans[m++] = {d, d + (uintptr_t)numels[i] * (dd[i] == GRPO_DTYPE_BF16 ? 2 : 4), 1};
    if (s != d || sd[i] != dd[i]) spans[m++] = {s, s + (uintptr_t)numels[i] * (sd[i] == GRPO_DTYPE_BF16 ? 2 : 4), 0};
  }
  std::sort(spans, spans + m, [](const Span& a, const Span& b) { return a.lo < b.lo; });
  uintptr_t read = 0, written = 0;  // the furthest ends so far
  for (int32_t i = 0; i < m; ++i) {
    if (spans[i].lo < written || (spans[i].write && spans[i].lo < read)) return true;
    (spans[i].write ? written : read) = std::max(spans[i].write ? written : read, spans[i].hi);
  }
  return false;
}

// The tables of a list, one launch each: go(table, first tensor, last launch).
template <int N, typename Go>
int each_table(const void* const* src, const int32_t* sd, void* const* dst, const int32_t* dd, const int64_t* numels,
               int32_t n, int64_t chunk, Go go) {
  for (int32_t i0 = 0; i0 == 0 || i0 < n; i0 += N) {
    Table<N> t;
    t.n = std::min(n - i0, N);
    int64_t c = 0;
    for (int32_t k = 0; k < t.n; ++k) {
      const int32_t i = i0 + k;
      t.chunk0[k] = (int32_t)c;
      c += (numels[i] + chunk - 1) / chunk;
      t.numel[k] = numels[i];
      t.src[k] = src[i];
      t.dst[k] = dst ? dst[i] : nullptr;
      t.kind[k] = (uint8_t)((sd[i] == GRPO_DTYPE_BF16) | (dd && dd[i] == GRPO_DTYPE_BF16) << 1);
    }
    t.chunk0[t.n] = (int32_t)c;
    const int rc = go(t, i0, i0 + N >= n);
    if (rc != GRPO_OK) return rc;
  }
  return GRPO_OK;
}

template <int N>
int norm_launches(const void* const* grads, const int64_t* numels, const int32_t* dtypes, int32_t n, int64_t chunk,
                  FinalArgs f, double* part, double* sum, cudaStream_t st) {
  float* norms = f.tensor_norms;
  return each_table<N>(grads, dtypes, nullptr, nullptr, numels, n, chunk, [&](const Table<N>& t, int32_t i0, bool last) -> int {
    if (t.chunk0[t.n] > 0) {
      norm_kernel<N><<<(unsigned)t.chunk0[t.n], kThreads, 0, st>>>(t, chunk, part);
      GRPO_CUDA_TRY(cudaGetLastError());
    }
    f.part = part;
    f.before = i0 ? sum : nullptr;
    f.sum = sum;
    f.tensor_norms = norms ? norms + i0 : nullptr;
    f.last = last;
    final_kernel<N><<<1, kFinalThreads, 0, st>>>(t, f);
    GRPO_CUDA_TRY(cudaGetLastError());
    return GRPO_OK;
  });
}

}  // namespace clip
}  // namespace grpo

using namespace grpo;
using namespace grpo::clip;

extern "C" GRPO_API size_t grpo_grad_norm_workspace_size(int64_t total_numel, int32_t n) {
  if (total_numel < 0 || n < 0 || n > kMaxTensors || total_numel > ((int64_t)1 << 48)) return 0;
  // the running sum, then the partials of a launch's chunks
  return 256 + 8 * (size_t)(total_numel / chunk_of(total_numel) + n);
}

extern "C" GRPO_API int grpo_grad_norm(const void* const* grads, const int64_t* numels, const int32_t* dtypes, int32_t n,
                                       float max_norm, const grpo_step_acc* acc, int32_t deferred, float* tensor_norms,
                                       grpo_grad_norm_result* result, void* workspace, size_t workspace_bytes,
                                       void* stream) {
  int64_t total = 0;
  const int rc = check_list(grads, numels, dtypes, n, &total);
  if (rc != GRPO_OK) return rc;
  if (!result || (uintptr_t)result % alignof(grpo_grad_norm_result) || !(max_norm >= 0.f) || (deferred && !acc) ||
      (uintptr_t)acc % alignof(grpo_step_acc) || !workspace || (uintptr_t)workspace % 8)
    return GRPO_ERR_INVALID;
  if (workspace_bytes < grpo_grad_norm_workspace_size(total, n)) return GRPO_ERR_CAPACITY;
  FinalArgs f{};
  f.tensor_norms = tensor_norms;
  f.acc = acc;
  f.deferred = deferred != 0;
  f.max_norm = max_norm;
  f.result = result;
  double* sum = static_cast<double*>(workspace);
  double* part = sum + 32;
  return n <= kSmall ? norm_launches<kSmall>(grads, numels, dtypes, n, chunk_of(total), f, part, sum, as_stream(stream))
                     : norm_launches<kLarge>(grads, numels, dtypes, n, chunk_of(total), f, part, sum, as_stream(stream));
}

extern "C" GRPO_API int grpo_grad_clip(const void* const* src, const int32_t* src_dtypes, void* const* dst,
                                       const int32_t* dst_dtypes, const int64_t* numels, int32_t n,
                                       const grpo_grad_norm_result* result, void* stream) {
  int64_t total = 0;
  int rc = check_list(src, numels, src_dtypes, n, &total);
  if (rc == GRPO_OK) rc = check_list(dst, numels, dst_dtypes, n, &total);
  if (rc != GRPO_OK) return rc;
  if (!result || (uintptr_t)result % alignof(grpo_grad_norm_result)) return GRPO_ERR_INVALID;
  if (total == 0) return GRPO_OK;
  Span few[2 * kSmall], *spans = few;
  if (n > kSmall) {
    spans = static_cast<Span*>(std::malloc(2 * (size_t)n * sizeof(Span)));
    if (!spans) return GRPO_ERR_CAPACITY;
  }
  const bool clash = overlaps(src, src_dtypes, dst, dst_dtypes, numels, n, spans);
  if (spans != few) std::free(spans);
  if (clash) return GRPO_ERR_INVALID;
  const cudaStream_t st = as_stream(stream);
  const int64_t chunk = chunk_of(total);
  auto go = [&](const auto& t, int32_t, bool) -> int {
    if (t.chunk0[t.n] == 0) return GRPO_OK;
    clip_kernel<<<(unsigned)t.chunk0[t.n], kThreads, 0, st>>>(t, chunk, result);
    GRPO_CUDA_TRY(cudaGetLastError());
    return GRPO_OK;
  };
  return n <= kSmall ? each_table<kSmall>(src, src_dtypes, dst, dst_dtypes, numels, n, chunk, go)
                     : each_table<kLarge>(src, src_dtypes, dst, dst_dtypes, numels, n, chunk, go);
}

static_assert(sizeof(grpo_grad_norm_result) == 32, "grpo_grad_norm_result is 32 bytes");
