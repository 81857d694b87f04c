// The global norm of many gradient tensors, each tensor's own, and the clip: what stands between a step's
// finish and the optimizer ("Sizing mini-batches and micro-batches", "The hard part: deferred
// normalization": scale by 1/max(sum, 1), then clip, then step).
//
//   S_i = sum_j g_ij^2,  S = sum_i S_i,  norm = s sqrt(S),  factor = s min(1, max_norm / norm)
//   out_ij = factor g_ij
//
// Bound by memory: every element is read once for the norm, and read and written once by the clip, which
// cannot begin before the norm is known. 1.24e9 bf16 in 219 tensors: the norm 343 us, 7.2 TB/s of reads, and 8
// to 12 for the last kernel; 311M float into bf16: 172 us, and the clip 258, 7.2 TB/s. The elements of all tensors
// are cut into equal shares, one to a block; a block leaves a partial sum for each tensor of its share. (A chunk
// of each tensor to a block, with a search and a joining of its own, took 133 us for the norm of 213M bf16; the
// shares take 67.) The tensors' addresses and sizes travel in the kernel's parameters: no table in device memory,
// nothing to keep alive, and a captured call replays by itself.
#include <algorithm>
#include <cmath>
#include <cstdlib>
#include <type_traits>

#include "grpo_common.cuh"

namespace grpo {
namespace clip {

constexpr int kThreads = 256;
constexpr int kVec = 8;        // elements a thread takes at a time
constexpr int kSlot = 256;     // shares and tensors begin at multiples of so many elements (a tensor is padded)
constexpr int kWave = 912;     // 152 SMs x 6 blocks: a constant, the order of the sums follows from it
constexpr int kMaxShares = 6 * kWave;
constexpr int kShare = 32768;  // elements of a share, at least, where there are several waves
constexpr int kFold = 8;       // vectors a thread sums before it folds them into its compensated sum
constexpr int kFinalThreads = 1024;
constexpr int kSeg = 16;  // partials of a tensor that a thread of the last kernel sums
constexpr int kFew = 16;  // a tensor of at most so many such sums is finished by one thread, others by a warp

// The tensors of one launch. slot0[i]: the first slot of tensor i among the launch's, slot0[n] their count. Share w
// is the slots [w share, (w + 1) share); its partial sum of tensor i is number w + i.
template <int N>
struct Table {
  static constexpr int kSize = N;
  int32_t n;
  int32_t slot0[N + 1];
  int64_t numel[N];
  const void* src[N];
  void* dst[N];     // (clip)
  uint8_t kind[N];  // bit 0: src is bf16, bit 1: dst is bf16
};

constexpr int32_t kMaxTensors = 1 << 24;
constexpr int64_t kMaxNumel = (int64_t)1 << 38;  // (slots are counted in 32 bits)
constexpr int kSmall = 32, kLarge = 512;  // tensors per launch: 1 KB and 17 KB of parameters

template <int N>
__device__ __forceinline__ int tensor_of(const Table<N>& t, int slot) {
  int lo = 0, hi = t.n - 1;  // the last i with slot0[i] <= slot (a tensor without elements has no slot)
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (t.slot0[mid] <= slot)
      lo = mid;
    else
      hi = mid - 1;
  }
  return lo;
}

// The slots [from, to) of the launch that lie in tensor i, as elements of it.
template <int N>
__device__ __forceinline__ void piece(const Table<N>& t, int i, int from, int to, int64_t& at, int64_t& n) {
  const int s0 = t.slot0[i], s1 = t.slot0[i + 1];
  at = (int64_t)((from > s0 ? from : s0) - s0) * kSlot;
  const int64_t end = (int64_t)((to < s1 ? to : s1) - s0) * kSlot;
  n = (end < t.numel[i] ? end : t.numel[i]) - at;
}

// A thread's 8 elements as they lie in memory: 16 bytes of bf16, 32 of float. (Plain loads: the clip may
// run in place.)
template <typename T>
struct Raw {
  uint4 q[sizeof(T) / 2];
};

template <bool ALIGNED, typename T>
__device__ __forceinline__ Raw<T> load8(const T* p) {
  Raw<T> r;
  if constexpr (ALIGNED) {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) r.q[i] = reinterpret_cast<const uint4*>(p)[i];
  } else if constexpr (sizeof(T) == 4) {
    const uint32_t* w = reinterpret_cast<const uint32_t*>(p);
    r.q[0] = make_uint4(w[0], w[1], w[2], w[3]);
    r.q[1] = make_uint4(w[4], w[5], w[6], w[7]);
  } else {
    const uint16_t* w = reinterpret_cast<const uint16_t*>(p);
    uint32_t v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = (uint32_t)w[2 * i] | (uint32_t)w[2 * i + 1] << 16;
    r.q[0] = make_uint4(v[0], v[1], v[2], v[3]);
  }
  return r;
}

template <typename T>
__device__ __forceinline__ void unpack(const Raw<T>& r, float (&v)[kVec]) {
#pragma unroll
  for (int i = 0; i < (int)sizeof(T) / 2; ++i) {
    const uint32_t w[4] = {r.q[i].x, r.q[i].y, r.q[i].z, r.q[i].w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if constexpr (sizeof(T) == 4) {
        v[4 * i + k] = __uint_as_float(w[k]);
      } else {
        v[2 * k] = bf16_lo(w[k]);
        v[2 * k + 1] = bf16_hi(w[k]);
      }
    }
  }
}

// The bits that tell whether an element is not 0: all but the signs.
template <typename T>
__device__ __forceinline__ uint32_t magnitudes(const Raw<T>& r) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < (int)sizeof(T) / 2; ++i) m |= r.q[i].x | r.q[i].y | r.q[i].z | r.q[i].w;
  return m & (sizeof(T) == 4 ? 0x7fffffffu : 0x7fff7fffu);
}

// The threads' values summed: in the warps as T (float: 5 roundings), over the warps in double. An SM adds two
// doubles a clock: a tree of them over 256 threads takes longer than reading 16 KB.
template <typename T>
__device__ __forceinline__ double block_sum(T v, double* red) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  __syncthreads();
  if (lane == 0) red[warp] = (double)v;
  __syncthreads();
  if (threadIdx.x == 0) {
    double s = red[0];
#pragma unroll
    for (int w = 1; w < kThreads / 32; ++w) s += red[w];
    red[0] = s;
  }
  __syncthreads();
  return red[0];
}

template <typename T>
__device__ __noinline__ double wide_sum(const T* p, int64_t n, double* red) {
  double s = 0.0;
  for (int64_t i = threadIdx.x; i < n; i += kThreads) {
    const double x = (double)(float)p[i];
    s = fma(x, x, s);
  }
  return block_sum(s, red);
}

// The sum of the squares of the n elements at p, the same in every thread. Thread t takes vectors t, t + 256, ..
// of 8 elements: 8 of them in four float chains, those folded into a float sum with its rounding errors
// beside it, the threads' sums joined by block_sum (a chain of 16, a tree of 4, the joining: 26 roundings of
// 2^-24 at most). The order goes by the index alone, whatever the address. A sum that may have left float's
// range -- above 2^120, not a number, or below 2^-80 with an element that is not 0 -- is formed once more
// in double, where no square over- or underflows.
template <bool ALIGNED, typename T>
__device__ __forceinline__ double chunk_sum(const T* p, int64_t n, double* red) {
  constexpr int kLoads = ALIGNED ? 8 / (int)sizeof(T) : 1;  // vectors in flight: 64 bytes a thread, 96 KB an SM
  const int nv = (int)(n / kVec);  // (a share has 2^28 elements at most)
  float s = 0.f, err = 0.f;
  uint32_t any = 0;
  float a[4] = {};
  auto add = [&](const Raw<T>& r) {
    float x[kVec];
    unpack(r, x);
#pragma unroll
    for (int i = 0; i < kVec; ++i) a[i & 3] = fmaf(x[i], x[i], a[i & 3]);
    any |= magnitudes(r);
  };
  auto fold = [&]() {  // s + err += the chains, s rounded, err what that leaves out (Knuth's two-sum)
    const float x = __fadd_rn(__fadd_rn(a[0], a[2]), __fadd_rn(a[1], a[3])), t = __fadd_rn(s, x), b = __fsub_rn(t, s);
    err = __fadd_rn(err, __fadd_rn(__fsub_rn(s, __fsub_rn(t, b)), __fsub_rn(x, b)));
    s = t;
    a[0] = a[1] = a[2] = a[3] = 0.f;
  };
  int v = threadIdx.x;
  for (; v + (kFold - 1) * kThreads < nv; v += kFold * kThreads) {
#pragma unroll 1
    for (int k = 0; k < kFold; k += kLoads) {
      Raw<T> r[kLoads];
#pragma unroll
      for (int l = 0; l < kLoads; ++l) r[l] = load8<ALIGNED>(p + (int64_t)(v + (k + l) * kThreads) * kVec);
#pragma unroll
      for (int l = 0; l < kLoads; ++l) add(r[l]);
    }
    fold();
  }
#pragma unroll 1
  for (; v < nv; v += kThreads) add(load8<ALIGNED>(p + (int64_t)v * kVec));
  if (threadIdx.x < n - (int64_t)nv * kVec) {
    const float x = (float)p[(int64_t)nv * kVec + threadIdx.x];
    a[0] = fmaf(x, x, a[0]);
    any |= __float_as_uint(x) & 0x7fffffffu;
  }
  fold();
  const double sum = block_sum(s + err, red);
  if (sum >= 8.271806125530277e-25 && sum <= 1.329227995784916e36) return sum;  // 2^-80 .. 2^120
  return __syncthreads_or(any != 0) ? wide_sum(p, n, red) : 0.0;
}

template <int N>
__global__ void __launch_bounds__(kThreads, 6) norm_kernel(const __grid_constant__ Table<N> t, int share, double* part) {
  __shared__ double red[kThreads / 32];
  pdl_launch();
  const int from = (int)blockIdx.x * share, to = min(from + share, t.slot0[t.n]);
  for (int i = tensor_of(t, from); i < t.n && t.slot0[i] < to; ++i) {
    int64_t at, n;
    piece(t, i, from, to, at, n);
    if (n <= 0) continue;  // a tensor without elements
    auto sum = [&](auto* p) {
      return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 ? chunk_sum<true>(p, n, red) : chunk_sum<false>(p, n, red);
    };
    const double s = (t.kind[i] & 1) ? sum(static_cast<const __nv_bfloat16*>(t.src[i]) + at)
                                     : sum(static_cast<const float*>(t.src[i]) + at);
    if (threadIdx.x == 0) part[(int)blockIdx.x + i] = s;
  }
}

// What the last kernel has to know of a launch's tensors: part0[i], the first of tensor i's partial sums,
// count[i], and seg0[i], the first of its segments of kSeg partials.
template <int N>
struct Partials {
  int32_t n, total;  // (total: the partials' places)
  int32_t part0[N], count[N], seg0[N + 1];
};

struct FinalArgs {
  const double* part;      // the launch's partials
  const double* before;    // sum of the launches before, or NULL
  double* sum;             // out: with this launch's
  float* tensor_norms;     // this launch's tensors, or NULL
  const grpo_step_acc* acc;
  int32_t deferred, last;
  float max_norm;
  grpo_grad_norm_result* result;
};

// sqrt(u) s, rounded to float: in float where u's range allows.
__device__ __forceinline__ float scaled_root(double u, double s) {
  const float f = (float)u;
  return f > 1e-30f && f < 1e30f ? sqrtf(f) * (float)s : (float)(sqrt(u) * s);
}

// The launch's partials summed per tensor, the tensors' sums, and with the last launch the result: a thread
// for each segment of a tensor, a thread or a warp for each tensor, a warp for all. The partials and the table are
// brought into shared memory first, and few warps add doubles (see block_sum).
template <int N>
__global__ void __launch_bounds__(kFinalThreads) final_kernel(const __grid_constant__ Partials<N> t, FinalArgs a) {
  extern __shared__ double part[];  // [t.total]
  __shared__ double seg[kMaxShares / kSeg + N], of[N];
  __shared__ int part0[N], count[N], seg0[N + 1];  // (a parameter indexed by the thread would be read lane by lane)
  const int tid = threadIdx.x, lane = tid & 31;
  {
    const int32_t *p = t.part0, *c = t.count, *g = t.seg0;
    asm("" : "+l"(p), "+l"(c), "+l"(g));  // by address
    for (int i = tid; i <= t.n; i += kFinalThreads) {
      if (i < t.n) {
        part0[i] = p[i];
        count[i] = c[i];
      }
      seg0[i] = g[i];
    }
  }
  pdl_launch();
  pdl_wait();
  double s = 1.0;
  if (a.deferred) s = 1.0 / (double)(a.acc->divisor > 1 ? a.acc->divisor : 1);
#pragma unroll 4
  for (int i = tid; i < t.total; i += kFinalThreads) part[i] = a.part[i];  // (places without a sum are not read below)
  __syncthreads();
  for (int g = tid; g < seg0[t.n]; g += kFinalThreads) {
    int lo = 0, hi = t.n - 1;  // the last tensor with seg0 <= g
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (seg0[mid] <= g)
        lo = mid;
      else
        hi = mid - 1;
    }
    const int k0 = (g - seg0[lo]) * kSeg, k1 = min(k0 + kSeg, count[lo]);
    double u = 0.0;
    for (int k = k0; k < k1; ++k) u += part[part0[lo] + k];
    seg[g] = u;
  }
  __syncthreads();
  for (int i = tid; i < t.n; i += kFinalThreads) {
    if (seg0[i + 1] - seg0[i] > kFew) continue;
    double u = 0.0;
    for (int g = seg0[i]; g < seg0[i + 1]; ++g) u += seg[g];
    of[i] = u;
    if (a.tensor_norms) a.tensor_norms[i] = scaled_root(u, s);
  }
  for (int i = tid >> 5; i < t.n; i += kFinalThreads / 32) {
    if (seg0[i + 1] - seg0[i] <= kFew) continue;  // warp-uniform
    double u = 0.0;
    for (int g = seg0[i] + lane; g < seg0[i + 1]; g += 32) u += seg[g];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) u += __shfl_xor_sync(0xffffffffu, u, o);
    if (lane == 0) {
      of[i] = u;
      if (a.tensor_norms) a.tensor_norms[i] = scaled_root(u, s);
    }
  }
  __syncthreads();
  if (tid >= 32) return;
  double v = 0.0;
  for (int i = lane; i < t.n; i += 32) v += of[i];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (tid != 0) return;
  const double total = a.before ? *a.before + v : v;
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

// out = f g, rounded once to out's type; zeros, with nothing read, where the step is skipped. From the end, as
// the shares are taken: what the norm has read last is still in L2.
template <typename S, typename D>
__device__ __forceinline__ void clip_piece(const S* src, D* dst, int64_t n, float f, bool skip) {
  const bool aligned = ((reinterpret_cast<uintptr_t>(src) | reinterpret_cast<uintptr_t>(dst)) & 15u) == 0;
  if (skip) {
    for (int64_t i = threadIdx.x; i < n; i += kThreads) put(dst + i, 0.f);
    return;
  }
  const int64_t nv = aligned ? n / kVec : 0;
  // past the last whole vector, or all of it: by element
  int64_t i = n - 1 - threadIdx.x;
  for (; i - 3 * kThreads >= nv * kVec; i -= 4 * kThreads) {
    S x[4];
#pragma unroll
    for (int l = 0; l < 4; ++l) x[l] = src[i - l * kThreads];
#pragma unroll
    for (int l = 0; l < 4; ++l) put(dst + i - l * kThreads, (float)x[l] * f);
  }
  for (; i >= nv * kVec; i -= kThreads) put(dst + i, (float)src[i] * f);
  constexpr int kLoads = 8 / (int)sizeof(S);
  auto put8 = [&](int64_t at, const Raw<S>& r) {
    float x[kVec];
    unpack(r, x);
#pragma unroll
    for (int k = 0; k < kVec; ++k) x[k] *= f;
    store8(dst + at * kVec, x);
  };
  int64_t v = nv - 1 - threadIdx.x;
  for (; v - (kLoads - 1) * kThreads >= 0; v -= kLoads * kThreads) {  // (all loads of a group before its stores)
    Raw<S> r[kLoads];
#pragma unroll
    for (int l = 0; l < kLoads; ++l) r[l] = load8<true>(src + (v - l * kThreads) * kVec);
#pragma unroll
    for (int l = 0; l < kLoads; ++l) put8(v - l * kThreads, r[l]);
  }
  for (; v >= 0; v -= kThreads) put8(v, load8<true>(src + v * kVec));
}

template <int N>
__global__ void __launch_bounds__(kThreads, 6) clip_kernel(const __grid_constant__ Table<N> t, int share,
                                                           const grpo_grad_norm_result* result) {
  const int from = (int)(gridDim.x - 1 - blockIdx.x) * share, to = min(from + share, t.slot0[t.n]);
  int i = tensor_of(t, to - 1);
  pdl_launch();
  pdl_wait();
  const float f = result->coef;
  const bool skip = result->status != GRPO_OK;
  for (; i >= 0 && t.slot0[i + 1] > from; --i) {
    int64_t at, n;
    piece(t, i, from, to, at, n);
    if (n <= 0 || (t.src[i] == t.dst[i] && !skip && f == 1.f)) continue;  // (in place, a factor of 1 changes nothing)
    const float* sf = static_cast<const float*>(t.src[i]) + at;
    const __nv_bfloat16* sb = static_cast<const __nv_bfloat16*>(t.src[i]) + at;
    float* df = static_cast<float*>(t.dst[i]) + at;
    __nv_bfloat16* db = static_cast<__nv_bfloat16*>(t.dst[i]) + at;
    switch (t.kind[i]) {
      case 0: clip_piece(sf, df, n, f, skip); break;
      case 1: clip_piece(sb, df, n, f, skip); break;
      case 2: clip_piece(sf, db, n, f, skip); break;
      default: clip_piece(sb, db, n, f, skip); break;
    }
  }
}

// ---- host -------------------------------------------------------------------------------------

// A launch that may begin while the kernel before it on the stream still runs (each waits for it itself).
template <typename... P, typename... A>
int launch_dep(void (*kern)(P...), int64_t blocks, unsigned threads, size_t smem, cudaStream_t st, const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3((unsigned)blocks, 1, 1);
  cfg.blockDim = dim3(threads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  GRPO_CUDA_TRY(cudaLaunchKernelEx(&cfg, kern, args...));
  return GRPO_OK;
}

int check_list(const void* const* p, const int64_t* numels, const int32_t* dtypes, int32_t n, int64_t* total) {
  if (n < 0 || n > kMaxTensors || (n > 0 && (!p || !numels || !dtypes))) return GRPO_ERR_INVALID;
  *total = 0;
  for (int32_t i = 0; i < n; ++i) {
    if (dtypes[i] != GRPO_DTYPE_F32 && dtypes[i] != GRPO_DTYPE_BF16) return GRPO_ERR_UNSUPPORTED;
    const uintptr_t size = dtypes[i] == GRPO_DTYPE_BF16 ? 2 : 4;
    if (numels[i] < 0 || numels[i] > kMaxNumel || (numels[i] > 0 && (!p[i] || (uintptr_t)p[i] % size)))
      return GRPO_ERR_INVALID;
    *total += numels[i];
    if (*total > kMaxNumel) return GRPO_ERR_INVALID;
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

// Slots of a share of the norm: one wave of blocks up to 32768 elements each (8 slots at least: a vector a
// thread); above, as many full waves of shares no smaller, up to 6: blocks that end early then make room for
// others (2^31 elements of bf16: one wave 627 us, six 588), what is read last lies together at the tensors' end
// (where the clip begins), and the last kernel's partials stay few.
int norm_share(int32_t slots) {
  const int waves = std::min(std::max(1, (int)((int64_t)slots * kSlot / ((int64_t)kWave * kShare))), kMaxShares / kWave);
  return std::max(8, (slots + waves * kWave - 1) / (waves * kWave));
}

// The clip leaves nothing to sum: a wave of shares, or of 32768 elements each as many as there are (311M
// float to bf16: 270 us with the norm's shares, 257 with these).
int clip_share(int32_t slots) { return std::max(8, std::min((slots + kWave - 1) / kWave, 32768 / kSlot)); }

// The tables of a list, one launch each: go(table, slots of a share, shares, first tensor, last launch).
template <int N, typename Go>
int each_table(const void* const* src, const int32_t* sd, void* const* dst, const int32_t* dd, const int64_t* numels,
               int32_t n, int (*share_of)(int32_t), Go go) {
  for (int32_t i0 = 0; i0 == 0 || i0 < n; i0 += N) {
    Table<N> t;
    t.n = std::min(n - i0, N);
    int32_t slots = 0;
    for (int32_t k = 0; k < t.n; ++k) {
      const int32_t i = i0 + k;
      t.slot0[k] = slots;
      slots += (int32_t)((numels[i] + kSlot - 1) / kSlot);
      t.numel[k] = numels[i];
      t.src[k] = src[i];
      t.dst[k] = dst ? dst[i] : nullptr;
      t.kind[k] = (uint8_t)((sd[i] == GRPO_DTYPE_BF16) | (dd && dd[i] == GRPO_DTYPE_BF16) << 1);
    }
    t.slot0[t.n] = slots;
    const int share = share_of(slots);
    const int rc = go(t, share, (slots + share - 1) / share, i0, i0 + N >= n);
    if (rc != GRPO_OK) return rc;
  }
  return GRPO_OK;
}

template <int N>
int norm_launches(const void* const* grads, const int64_t* numels, const int32_t* dtypes, int32_t n, FinalArgs f,
                  double* part, double* sum, cudaStream_t st) {
  float* norms = f.tensor_norms;
  return each_table<N>(grads, dtypes, nullptr, nullptr, numels, n, norm_share, [&](const Table<N>& t, int share, int shares, int32_t i0, bool last) -> int {
    if (shares > 0) {
      norm_kernel<N><<<(unsigned)shares, kThreads, 0, st>>>(t, share, part);
      GRPO_CUDA_TRY(cudaGetLastError());
    }
    f.part = part;
    f.before = i0 ? sum : nullptr;
    f.sum = sum;
    f.tensor_norms = norms ? norms + i0 : nullptr;
    f.last = last;
    Partials<N> p;
    p.n = t.n;
    p.total = shares > 0 ? shares + t.n - 1 : 0;
    int32_t segs = 0;
    for (int32_t i = 0; i < t.n; ++i) {
      const int32_t s0 = t.slot0[i], s1 = t.slot0[i + 1];
      p.part0[i] = s0 / share + i;
      p.count[i] = s1 > s0 ? (s1 - 1) / share - s0 / share + 1 : 0;
      p.seg0[i] = segs;
      segs += (p.count[i] + kSeg - 1) / kSeg;
    }
    p.seg0[t.n] = segs;
    const size_t smem = sizeof(double) * (size_t)p.total;
    if (smem > 16384)  // (with the static part past 48 KB)
      GRPO_CUDA_TRY(cudaFuncSetAttribute(final_kernel<N>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)(sizeof(double) * (kMaxShares + N))));
    return launch_dep(final_kernel<N>, 1, kFinalThreads, smem, st, p, f);
  });
}

}  // namespace clip
}  // namespace grpo

using namespace grpo;
using namespace grpo::clip;

extern "C" GRPO_API size_t grpo_grad_norm_workspace_size(int64_t total_numel, int32_t n) {
  if (total_numel < 0 || n < 0 || n > kMaxTensors || total_numel > kMaxNumel) return 0;
  // the running sum, then the partials of a launch
  return 256 + 8 * (size_t)(std::min<int64_t>(kMaxShares, total_numel / kSlot + n) + std::min(n, kLarge));
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
  return n <= kSmall ? norm_launches<kSmall>(grads, numels, dtypes, n, f, part, sum, as_stream(stream))
                     : norm_launches<kLarge>(grads, numels, dtypes, n, f, part, sum, as_stream(stream));
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
  auto go = [&](const auto& t, int share, int shares, int32_t, bool) -> int {
    if (shares == 0) return GRPO_OK;
    return launch_dep(clip_kernel<std::decay_t<decltype(t)>::kSize>, shares, kThreads, 0, st, t, share, result);
  };
  return n <= kSmall ? each_table<kSmall>(src, src_dtypes, dst, dst_dtypes, numels, n, clip_share, go)
                     : each_table<kLarge>(src, src_dtypes, dst, dst_dtypes, numels, n, clip_share, go);
}

static_assert(sizeof(grpo_grad_norm_result) == 32, "grpo_grad_norm_result is 32 bytes");
