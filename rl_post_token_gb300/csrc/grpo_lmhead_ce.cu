// Softmax cross entropy from hidden states: z = h W^T is formed tile by tile on the tensor cores and
// consumed in the GEMM's epilogue (formulas in grpo_lmhead_ce.cuh); no more of the [T, V] dlogits is stored
// than two pieces of the vocabulary, and of the logits no more than 256 MB.
//
//  compact    the unmasked tokens first, in token order, and their hidden states gathered: every GEMM
//             below runs over them only (a fine-tuning batch masks its prompts). Not with mask NULL
//  pass A     per (token, 256 vocabulary entries) the softmax's (shift, sum), the target logit and, with
//             label smoothing, the sum of the logits
//  reduce     per token the tiles joined in a fixed order: loss, log-prob, lse and the gradient's factors
//  backward   per vocabulary piece the bf16 dlogits, in one of two buffers: of the logits formed once more, or
//             where the vocabulary is one piece of moderate size of those that pass A kept (ce_keep); then
//             d_h (+)= dz W_c and dW_c = dz^T h in one launch (grpo_lmhead_ce_bwd.cuh), on a second stream
//             beside the next piece's
//
// Bound by the tensor cores with many tokens: 2 T V H flops of pass A and 6 T V H of the backward, of which
// the 2 T V H of the logits' second forming stand for a store and two readings of the [T, V] logits. 4096
// unmasked tokens of 8192, V = 151936, H = 2048 (1.02e13 flops): 5.4 ms serialised, 1.9 PFLOP/s; 5.8 to 6.35 ms
// among others under the power cap, 1.6 to 1.77, where plain bf16 products of the same length reach 1.73. With
// few tokens by the readings of W (two) and the writing of dW: 16 tokens, V = 32000, H = 768 (98 MB without the
// second reading): 44 us of five dependent launches.
#include <algorithm>
#include <cmath>
#include <cstdlib>
#include <mutex>

#include "grpo_lmhead_ce_bwd.cuh"
#include "grpo_lmhead_host.cuh"

namespace grpo {
namespace lmhead {

constexpr int kCompactThreads = 256;
constexpr int64_t kCeMaxH = (int64_t)1 << 24;  // (256 rows' vectors are counted in 32 bits)

// The count of bytes that are not 0.
__device__ __forceinline__ int32_t nonzero_bytes(uint32_t w) { return __popc(__vsetne4(w, 0u)); }

// The unmasked tokens' indices first, in token order, then the masked ones', and the unmasked count; their
// hidden states gathered in that order, zeros behind them up to the padded count (dW reduces over those rows);
// the masked tokens' d_h rows zeroed (dh_vec 16-byte vectors; no GEMM writes them). Every block counts the whole
// mask for itself, which is less than a launch of its own for that: block b then takes the tokens
// [b per, (b + 1) per), per a multiple of 16, 256 at a time; its rows' vectors are dealt to all its threads.
__global__ void __launch_bounds__(kCompactThreads) ce_compact_kernel(int64_t T, int64_t per, int H, const uint8_t* mask,
                                                                     const __nv_bfloat16* h, int32_t* idx,
                                                                     int32_t* live_n, __nv_bfloat16* h_live, void* d_h,
                                                                     int dh_vec) {
  pdl_launch();
  constexpr int kWarps = kCompactThreads / 32;
  __shared__ int32_t sums[2][kWarps], live_of[kWarps], on_row[kCompactThreads], off_row[kCompactThreads];
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5, nvec = H >> 3;
  const uint4 z4 = make_uint4(0u, 0u, 0u, 0u);
  const int64_t t0 = (int64_t)blockIdx.x * per, t1 = t0 + per < T ? t0 + per : T;
  int32_t before = 0, total = 0;
  int64_t done = 0;
  if ((reinterpret_cast<uintptr_t>(mask) & 15u) == 0) {
    done = T / 16 * 16;
#pragma unroll 4
    for (int64_t t = (int64_t)tid * 16; t < done; t += kCompactThreads * 16) {
      const uint4 v = *reinterpret_cast<const uint4*>(mask + t);
      const int32_t n = nonzero_bytes(v.x) + nonzero_bytes(v.y) + nonzero_bytes(v.z) + nonzero_bytes(v.w);
      total += n;
      before += t < t0 ? n : 0;
    }
  }
#pragma unroll 8
  for (int64_t t = done + tid; t < T; t += kCompactThreads) {
    const int32_t n = mask[t] != 0;
    total += n;
    before += t < t0 ? n : 0;
  }
  total = __reduce_add_sync(0xffffffffu, total);
  before = __reduce_add_sync(0xffffffffu, before);
  if (lane == 0) {
    sums[0][w] = total;
    sums[1][w] = before;
  }
  __syncthreads();
  total = before = 0;
#pragma unroll
  for (int k = 0; k < kWarps; ++k) {
    total += sums[0][k];
    before += sums[1][k];
  }
  if (blockIdx.x == gridDim.x - 1) {
    if (tid == 0) *live_n = total;
    const int64_t pad = live_pad(total, T) < T ? live_pad(total, T) : T;
    uint4* rest = reinterpret_cast<uint4*>(h_live) + (int64_t)total * nvec;
    for (int64_t k = tid; k < (pad - total) * nvec; k += kCompactThreads) rest[k] = z4;
  }
  for (int64_t b = t0; b < t1; b += kCompactThreads) {
    const int64_t t = b + tid;
    const bool in = t < t1, on = in && mask[t] != 0;
    const unsigned m = __ballot_sync(0xffffffffu, on);
    if (lane == 0) live_of[w] = __popc(m);
    __syncthreads();
    int32_t rank = __popc(m & ((1u << lane) - 1u)), all = 0;  // unmasked tokens of [b, t)
#pragma unroll
    for (int k = 0; k < kWarps; ++k) {
      rank += k < w ? live_of[k] : 0;
      all += live_of[k];
    }
    if (in) {
      const int64_t masked = t - (before + rank);  // masked tokens before t
      idx[on ? before + rank : total + masked] = (int32_t)t;
      (on ? on_row[rank] : off_row[tid - rank]) = tid;
    }
    __syncthreads();
    // the block's unmasked rows lie side by side in the compact order
    uint4* dst = reinterpret_cast<uint4*>(h_live) + (int64_t)before * nvec;
    const uint4* src = reinterpret_cast<const uint4*>(h) + b * nvec;
#pragma unroll 4
    for (int k = tid; k < all * nvec; k += kCompactThreads) {
      const int r = k / nvec;
      dst[k] = src[(int64_t)on_row[r] * nvec + (k - r * nvec)];
    }
    if (d_h) {
      const int off = (int)(t1 - b < kCompactThreads ? t1 - b : kCompactThreads) - all;
      uint4* rows = reinterpret_cast<uint4*>(d_h) + b * dh_vec;
      for (int k = tid; k < off * dh_vec; k += kCompactThreads) {
        const int r = k / dh_vec;
        rows[(int64_t)off_row[r] * dh_vec + (k - r * dh_vec)] = z4;
      }
    }
    before += all;
    __syncthreads();  // (live_of and the rows are written again)
  }
}

struct CeReduceArgs {
  int64_t T, V;
  int n_col_tiles;
  const float *part_m, *part_s, *part_z, *zy;  // part_z: with label smoothing
  const int32_t* target;
  const float* w_tok;
  float smoothing, z_loss;
  float *lse2, *coef, *ea;  // [T] out, by token: what the dlogits epilogue takes
  float *loss_tok, *logp_tok, *lse_tok;
  grpo_step_acc* acc;
  const int32_t *idx, *live_n;  // the compact order, or NULL
};

// What a token's joined partials (t: shift and sum, z: sum of the logits) give; all 0 for a masked one.
struct CeToken {
  float loss, logp, lse, l2, sw, cp;
  bool bad;
};

// A token's target logit (NaN for a bad target) and weight: loaded before the partials are joined, which hides
// the loads' latency.
struct CeInputs {
  float zy, w;
};

__device__ __forceinline__ CeInputs ce_inputs(const CeReduceArgs& a, int64_t tok) {
  const float zy = a.zy[tok];  // (whatever it holds where no column is the target)
  const int32_t y = a.target[tok];
  return {y >= 0 && (int64_t)y < a.V ? zy : __int_as_float(0x7fc00000), a.w_tok ? a.w_tok[tok] : 1.f};
}

__device__ __forceinline__ CeToken ce_token(const CeReduceArgs& a, const CeInputs& in, MS t, float z) {
  CeToken o;
  const float nan = __int_as_float(0x7fc00000);
  const float zy = in.zy;
  const float l2s = log2f(t.s);
  o.l2 = t.m + l2s;
  // rows past the vouched range of logits count as non-finite, as in the policy loss
  const bool ok = fabsf(o.l2) <= kLseMax * kLog2e;
  o.lse = ok ? o.l2 * kLn2 : nan;
  o.logp = ok ? (fmaf(zy, kLog2e, -t.m) - l2s) * kLn2 : nan;  // without cancellation
  o.loss = -(1.f - a.smoothing) * o.logp + a.z_loss * o.lse * o.lse;
  // lse - mean z, from the shift too
  if (a.part_z) o.loss += a.smoothing * ((t.m - z / (float)a.V * kLog2e) + l2s) * kLn2;
  o.sw = in.w;
  o.cp = o.sw * fmaf(2.f * a.z_loss, o.lse, 1.f);
  if (!isfinite(o.loss)) o.cp = o.sw = nan;  // (also with a weight of 0: the gradient is NaN)
  o.bad = !isfinite(o.cp);
  return o;
}

__device__ __forceinline__ void ce_store_token(const CeReduceArgs& a, int64_t tok, const CeToken& o) {
  a.loss_tok[tok] = o.loss;
  if (a.logp_tok) a.logp_tok[tok] = o.logp;
  if (a.lse_tok) a.lse_tok[tok] = o.lse;
}

constexpr int kCeReduceWarps = 32;

// Every 32nd tile's partials of row i from `first` on, folded in order; four tiles' loads at a time.
__device__ __forceinline__ void ce_fold(const CeReduceArgs& a, int64_t i, int first, MS& t, float& z) {
  for (int c0 = first; c0 < a.n_col_tiles; c0 += 4 * kCeReduceWarps) {
    MS u[4];
    float v[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int c = c0 + k * kCeReduceWarps;
      const int64_t at = (int64_t)c * a.T + i;
      const bool in = c < a.n_col_tiles;
      u[k] = in ? MS{a.part_m[at], a.part_s[at]} : MS{-INFINITY, 0.f};
      v[k] = in && a.part_z ? a.part_z[at] : 0.f;
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      t = ms2_combine(t, u[k]);
      z += v[k];
    }
  }
}

// A block takes 32 tokens (lane = token: a partial's load is one 128-byte line), its warps every 32nd
// vocabulary tile in order; four warps join eight warps' each, warp 0 the four, in order.
__global__ void __launch_bounds__(kCeReduceWarps * 32) ce_reduce_kernel(CeReduceArgs a) {
  pdl_launch();
  pdl_wait();
  __shared__ float wm[kCeReduceWarps][32], ws[kCeReduceWarps][32], wz[kCeReduceWarps][32];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int64_t i = (int64_t)blockIdx.x * 32 + lane;
  const bool in = i < a.T, live = in && (!a.idx || i < (int64_t)*a.live_n);
  const int64_t tok = in && a.idx ? (int64_t)a.idx[i] : i;
  CeInputs given{};
  if (w == 0 && live) given = ce_inputs(a, tok);
  MS t{-INFINITY, 0.f};
  float z = 0.f;
  if (live) ce_fold(a, i, w, t, z);
  wm[w][lane] = t.m;
  ws[w][lane] = t.s;
  wz[w][lane] = z;
  __syncthreads();
  auto join = [&](int first, int step, int n) {
    MS r{wm[first][lane], ws[first][lane]};
    float s = wz[first][lane];
#pragma unroll
    for (int k = 1; k < n; ++k) {
      r = ms2_combine(r, MS{wm[first + k * step][lane], ws[first + k * step][lane]});
      s += wz[first + k * step][lane];
    }
    t = r;
    z = s;
  };
  if (w < 4) {
    join(w * 8, 1, 8);
    wm[w * 8][lane] = t.m;
    ws[w * 8][lane] = t.s;
    wz[w * 8][lane] = z;
  }
  __syncthreads();
  if (w != 0) return;
  bool bad = false;
  if (in) {
    CeToken o{};
    if (live) {
      join(0, 8, 4);
      o = ce_token(a, given, t, z);
      bad = o.bad;
    }
    ce_store_token(a, tok, o);
    a.lse2[tok] = o.l2;
    a.coef[tok] = o.sw;
    a.ea[tok] = o.cp;
  }
  const unsigned n_tok = __popc(__ballot_sync(0xffffffffu, in)), n_live = __popc(__ballot_sync(0xffffffffu, live)),
                 n_bad = __popc(__ballot_sync(0xffffffffu, bad));
  if (lane == 0) {
    atomicAdd(reinterpret_cast<unsigned long long*>(&a.acc->n_tokens), (unsigned long long)n_tok);
    if (n_live) atomicAdd(reinterpret_cast<unsigned long long*>(&a.acc->n_valid), (unsigned long long)n_live);
    if (n_bad) atomicAdd(reinterpret_cast<unsigned long long*>(&a.acc->n_nonfinite), (unsigned long long)n_bad);
  }
}

struct CeDzArgs {
  int64_t T, V, ld;  // ld: columns of x and dz
  const float* x;    // [T][ld] the kept products, by compact row
  __nv_bfloat16* dz;
  const int32_t *target, *idx, *live_n;
  const float *lse2, *coef, *ea;
  float cap, inv_cap, ce_hot, ce_smooth;
};

// 8 columns of a row's dlogits from its kept logits (the formula of epi_ce_dlogits; k: the target's place).
template <bool CAP>
__device__ __forceinline__ uint4 ce_dz8(const CeDzArgs& a, const float* x, float sw, float l2, float cp, int64_t k) {
  const float4 x0 = reinterpret_cast<const float4*>(x)[0], x1 = reinterpret_cast<const float4*>(x)[1];
  const float ce = sw * a.ce_smooth, cy = sw * a.ce_hot;
  float v[8] = {x0.x, x0.y, x0.z, x0.w, x1.x, x1.y, x1.z, x1.w};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float t = 0.f, d = 1.f;
    if constexpr (CAP) {
      tanh_pair(__fmul_rn(v[i], a.inv_cap), t, d);
      v[i] = a.cap * t;
    }
    v[i] = (fmaf(cp, ex2(fmaf(v[i], kLog2e, -l2)), -ce) - (i == k ? cy : 0.f)) * d;
  }
  return make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
}

// The dlogits of the kept logits: a block takes 2048 columns of every gridDim.y-th row. The rows up to the
// padded count are zeros (dW reduces over them).
template <bool CAP>
__global__ void __launch_bounds__(256) ce_dz_kernel(CeDzArgs a) {
  pdl_launch();
  pdl_wait();
  const int64_t nl = a.live_n ? (int64_t)*a.live_n : a.T, pad = a.live_n ? live_pad(nl, a.T) : a.T;
  const int64_t rows = pad < a.T ? pad : a.T, col = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 8;
  if (col >= a.V) return;
#pragma unroll 2
  for (int64_t r = blockIdx.y; r < rows; r += gridDim.y) {
    uint4 w = make_uint4(0u, 0u, 0u, 0u);
    const int64_t tok = r < nl ? (a.idx ? (int64_t)a.idx[r] : r) : -1;
    const float sw = tok >= 0 ? a.coef[tok] : 0.f;
    if (sw != 0.f) w = ce_dz8<CAP>(a, a.x + r * a.ld + col, sw, a.lse2[tok], a.ea[tok], a.target[tok] - col);
    *reinterpret_cast<uint4*>(a.dz + r * a.ld + col) = w;
  }
}

// ce_reduce_kernel and ce_dz_kernel in one, for few tokens: a block takes 2048 columns of one row, and joins
// that row's partials for itself; the first column block writes the token's outputs.
template <bool CAP>
__global__ void __launch_bounds__(256) ce_reduce_dz_kernel(CeReduceArgs r, CeDzArgs a) {
  const int lane = threadIdx.x & 31;
  pdl_launch();
  pdl_wait();
  const int64_t i = blockIdx.y, nl = a.live_n ? (int64_t)*a.live_n : a.T, pad = a.live_n ? live_pad(nl, a.T) : a.T;
  const int64_t tok = a.idx ? (int64_t)a.idx[i] : i;
  CeToken o{};
  if (i < nl) {  // (uniform)
    const CeInputs given = ce_inputs(r, tok);
    // ce_reduce_kernel's order, its warps the lanes here: every 32nd tile, eight joined, then the four
    MS t{-INFINITY, 0.f};
    float z = 0.f;
    ce_fold(r, i, lane, t, z);
    auto join = [&](int first, int step, int n) {
      MS u{__shfl_sync(0xffffffffu, t.m, first), __shfl_sync(0xffffffffu, t.s, first)};
      float s = __shfl_sync(0xffffffffu, z, first);
#pragma unroll
      for (int k = 1; k < n; ++k) {
        u = ms2_combine(u, MS{__shfl_sync(0xffffffffu, t.m, first + k * step), __shfl_sync(0xffffffffu, t.s, first + k * step)});
        s += __shfl_sync(0xffffffffu, z, first + k * step);
      }
      t = u;
      z = s;
    };
    join(lane & 24, 1, 8);
    join(0, 8, 4);
    o = ce_token(r, given, t, z);
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    ce_store_token(r, tok, o);
    atomicAdd(reinterpret_cast<unsigned long long*>(&r.acc->n_tokens), 1ull);
    if (i < nl) atomicAdd(reinterpret_cast<unsigned long long*>(&r.acc->n_valid), 1ull);
    if (o.bad) atomicAdd(reinterpret_cast<unsigned long long*>(&r.acc->n_nonfinite), 1ull);
  }
  const int64_t col = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 8;
  if (i >= pad || col >= a.V) return;
  uint4 w = make_uint4(0u, 0u, 0u, 0u);
  if (o.sw != 0.f) w = ce_dz8<CAP>(a, a.x + i * a.ld + col, o.sw, o.l2, o.cp, a.target[tok] - col);
  *reinterpret_cast<uint4*>(a.dz + i * a.ld + col) = w;
}

// d_h = scale (the runs' float sums, joined in an order that goes by `split`), rounded once; compact row r to
// its token's row. A block takes 256 / G vectors of 4, G groups of its threads every G-th run.
template <int G>
__global__ void __launch_bounds__(256) ce_dh_kernel(const int32_t* live_n, const int32_t* row_idx, int64_t T, int H4,
                                                    const float* part, int split, float scale, void* d_h, int out_bf16) {
  pdl_launch();
  pdl_wait();
  constexpr int W = 256 / G;
  __shared__ float4 sh[G > 1 ? G : 1][W];
  const int64_t n = (live_n ? (int64_t)*live_n : T) * H4, stride = T * H4;
  const float4* p = reinterpret_cast<const float4*>(part);
  const int x = threadIdx.x % W, y = threadIdx.x / W;
  for (int64_t i0 = (int64_t)blockIdx.x * W; i0 < n; i0 += (int64_t)gridDim.x * W) {
    const int64_t i = i0 + x;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    if (i < n) {
#pragma unroll(G > 1 ? 2 : 8)
      for (int s = y; s < split; s += G) {
        const float4 o = p[s * stride + i];
        v = make_float4(v.x + o.x, v.y + o.y, v.z + o.z, v.w + o.w);
      }
    }
    if constexpr (G > 1) {
      __syncthreads();
      sh[y][x] = v;
      __syncthreads();
      if (y == 0)
#pragma unroll
        for (int k = 1; k < G; ++k) {
          const float4 o = sh[k][x];
          v = make_float4(v.x + o.x, v.y + o.y, v.z + o.z, v.w + o.w);
        }
    }
    if (y != 0 || i >= n) continue;
    v = make_float4(v.x * scale, v.y * scale, v.z * scale, v.w * scale);
    const int64_t r = i / H4, to = (row_idx ? (int64_t)row_idx[r] : r) * H4 + (i - r * H4);
    if (out_bf16)
      reinterpret_cast<uint2*>(d_h)[to] = make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
    else
      reinterpret_cast<float4*>(d_h)[to] = v;
  }
}

}  // namespace lmhead
}  // namespace grpo

using namespace grpo;
using namespace grpo::lmhead;

namespace {

struct CeLayout {
  size_t part_m, part_s, part_z, zy, lse2, coef, ea, idx, live_n, h_live, dz[2], part, x, total;
  int n_col_tiles, chunk_tiles, n_chunks, split, keep;
  int64_t vchunk;  // columns of a dlogits buffer
};

// Vocabulary tiles per piece: pieces of up to 256 MB of dlogits, 66 tiles at least (16896 columns: 277 MB
// at 8192 tokens). Larger pieces mean fewer launches and fuller last rounds; the dlogits' way through memory
// hides behind the products.
int ce_chunk_tiles(int64_t T) {
  return (int)std::max<int64_t>(kMaxChunkTiles, std::min<int64_t>(((int64_t)256 << 20) / (T * BN * 2), INT32_MAX / BN));
}

// Runs that d_h's reduction over a piece is cut into: so many that a unit of d_h is at most a third of what
// one of 76 pairs of SMs has to do for d_h and dW together (the rest then evens out), each of 8 K blocks or
// more. The sizes alone decide: the workspace's size and the order of the sums follow from it.
int ce_split(int64_t T, int64_t H, int chunk_tiles) {
  const int64_t n_nt = (H + BN - 1) / BN, kb1 = (int64_t)chunk_tiles * (BN / BK), kb2 = (T + BK - 1) / BK;
  const int64_t load = ((T + 2 * BM - 1) / (2 * BM) * n_nt * kb1 + (int64_t)chunk_tiles * n_nt * kb2) / 76;
  return (int)std::max<int64_t>(1, std::min<int64_t>((3 * kb1 + load - 1) / std::max<int64_t>(load, 1), kb1 / 8));
}

// Whether pass A keeps its logits, as float, for the dlogits: where the vocabulary is one piece and they take
// 256 MB at most, and 8 bytes an entry (a store, a reading) cost less than 2 H flops. That goes by H: from 1088 on,
// or from 768 where rows that are no multiple of 128 bytes slow the products; with few tokens (T <= H / 4)
// forming them again is a reading of W; and a few MB stay in L2. Kept and formed again, us of a call:
// 800 x 50257 with H = 768, 1024, 1280, 2048: 225 and 217, 266 and 272, 310 and 335, 442 and 509; 250 x 50257 x
// 512 82 and 76, 100 x 151936 x 512 142 and 148, 16 x 32000 x 768 50 and 56, 500 x 9000 x 512 40 and 41,
// 999 x 50257 x 1000 325 and 339 (the only size measured off 64 rows).
bool ce_keep(int64_t T, int64_t H, int64_t vchunk, int n_chunks) {
  const int64_t bytes = T * vchunk * 4;
  return n_chunks == 1 && (bytes <= ((int64_t)20 << 20) ||
                           (bytes <= ((int64_t)256 << 20) && (4 * T <= H || H >= (H % BK ? 768 : 1088))));
}

// CTAs per tile: 1 where tiles of 128 tokens come to less than 3/4 of the rounds over the SMs in pass A that the
// pairs' of 256 take. (A CTA by itself loads half as much again for a tile: 800 x 50257 x 1000, 10 rounds and 11,
// 390 us of a call against 318; 600 x 1024, 7 and 8, 222 and 204; 300 x 512, 4 and 6, 90 and 95; 64 x 151936 x 2048,
// 4 and 8, 354 and 407.) GRPO_LMHEAD_CTA_GROUP decides where it is set.
int ce_cta_group(int64_t T, int n_col_tiles) {
  if (getenv("GRPO_LMHEAD_CTA_GROUP")) return cta_group();
  auto rounds = [&](int64_t rows, int64_t slots) { return ((T + rows - 1) / rows * n_col_tiles + slots - 1) / slots; };
  const int64_t sms = sm_count();
  return 4 * rounds(BM, sms) < 3 * rounds(2 * BM, std::max<int64_t>(sms / 2, 1)) ? 1 : 2;
}

CeLayout ce_layout(int64_t T, int64_t V, int64_t H) {
  CeLayout w{};
  w.n_col_tiles = (int)((V + BN - 1) / BN);
  const int most = ce_chunk_tiles(T);
  w.n_chunks = (w.n_col_tiles + most - 1) / most;
  w.chunk_tiles = (w.n_col_tiles + w.n_chunks - 1) / w.n_chunks;
  w.n_chunks = (w.n_col_tiles + w.chunk_tiles - 1) / w.chunk_tiles;
  w.vchunk = (int64_t)w.chunk_tiles * BN;
  w.split = ce_split(T, H, w.chunk_tiles);
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off += (bytes + 255) / 256 * 256;
    return at;
  };
  const size_t t4 = (size_t)T * 4, parts = (size_t)w.n_col_tiles * t4;
  w.part_m = take(parts);
  w.part_s = take(parts);
  w.part_z = take(parts);
  w.zy = take(t4);
  w.lse2 = take(t4);
  w.coef = take(t4);
  w.ea = take(t4);
  w.idx = take(t4);
  w.live_n = take(4);
  w.h_live = take((size_t)T * H * 2);
  w.dz[0] = take((size_t)T * w.vchunk * 2);
  w.dz[1] = w.n_chunks > 1 ? take((size_t)T * w.vchunk * 2) : w.dz[0];
  w.part = take((size_t)w.split * T * H * 4);  // d_h's float sums, of each run
  w.keep = ce_keep(T, H, w.vchunk, w.n_chunks);
  w.x = w.keep ? take((size_t)T * w.vchunk * 4) : 0;
  w.total = off;
  return w;
}

// Whether the reduce and the kept logits' dlogits are one launch: every column block of a row then joins the
// row's partials again, which is worth a launch while that is little to read (64 x 9000 x 128: 27.7 us of a call and
// 31.6 by two launches; above the limit, 16 x 32000 x 768: 48.2 and 47.2, 64 x 32000 x 768: 56 and 51).
bool ce_joint(int64_t T, int64_t col_blocks, int n_col_tiles) { return T * col_blocks * n_col_tiles <= (1 << 14); }

struct CeCall {
  const void* W;
  int64_t T, V, H;
  const int32_t* target;
  float smoothing, cap, scale;
  void *d_h, *dW;
  int dh_bf16, dw_bf16, dw_accumulate, cg;
  grpo_step_acc* acc;
  CeLayout ws;
  uint8_t* base;
  const void* h_src;      // h, or the compact hidden states
  const int32_t *idx, *live_n;
  cudaStream_t st;
  // Rows of A that a CTA loads of the tokens' operands: all 128 of the tile, or with fewer tokens theirs (the
  // others' accumulator rows are then whatever the stage held, and nothing reads them).
  int a_rows() const { return cg == 1 && T < BM ? (int)((T + 7) / 8 * 8) : BM; }
  float* f(size_t off) const { return reinterpret_cast<float*>(base + off); }
};

// A launch that may begin while the kernel before it on the stream still runs (see pdl_wait).
template <typename... P, typename... A>
int launch_dep(void (*kern)(P...), dim3 grid, unsigned threads, cudaStream_t st, const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads, 1, 1);
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  GRPO_CUDA_TRY(cudaLaunchKernelEx(&cfg, kern, P(args)...));
  return GRPO_OK;
}

// The target of EPI_CE_STORE: [runs][rows][cols], boxes of 32 rows x 64 bytes in the 64-byte swizzle.
bool map_out(CUtensorMap* m, const void* base, int64_t cols, int64_t rows, int64_t runs, int64_t ld, bool bf16) {
  auto fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t size = bf16 ? 2 : 4;
  cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)rows, (cuuint64_t)runs};
  cuuint64_t strides[2] = {(cuuint64_t)ld * size, (cuuint64_t)ld * rows * size};
  cuuint32_t box[3] = {(cuuint32_t)(64 / size), 32, 1}, estr[3] = {1, 1, 1};
  return fn(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3, const_cast<void*>(base), dims,
            strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int PLAIN, int CAP>
int ce_logits(const CeCall& c, GemmArgs g, cudaStream_t st, int64_t vc, bool pdl) {
  CUtensorMap ma, mb, mc = {};
  if (!map_k(&ma, c.h_src, c.T, c.H, c.H, c.a_rows()) || !map_k(&mb, c.W, c.V, c.H, c.H, BN / c.cg)) return GRPO_ERR_UNSUPPORTED;
  if (epi_is_dlogits(PLAIN) && !map_dz_store(&mc, g.dz, c.T, vc, g.ldz)) return GRPO_ERR_UNSUPPORTED;
  if (g.keep && !map_out(&mc, c.f(c.ws.x), c.V, c.T, 1, c.ws.vchunk, false)) return GRPO_ERR_UNSUPPORTED;
  g.M = c.T;
  g.K = c.H;
  g.V = c.V;
  g.m_fast = 1;  // consecutive units share the W tile
  g.target = c.target;
  g.row_idx = c.idx;
  g.live_n = c.live_n;
  g.acc = c.acc;
  g.zy = c.f(c.ws.zy);
  g.a_rows = c.a_rows();
  g.cap = c.cap;
  g.gain = (float)std::min<int64_t>(c.H, kGainMaxH) * 0x1p-30f;
  g.inv_cap = 1.f / c.cap;
  return c.cap > 0.f ? launch<CAP, false, false>(c.cg, ma, mb, mc, g, st, pdl)
                     : launch<PLAIN, false, false>(c.cg, ma, mb, mc, g, st, pdl);
}

// Both products of piece `chunk`, the vocabulary columns [v0, v0 + vc).
template <int CG>
int ce_products(const CeCall& c, const __nv_bfloat16* dz, int chunk, int64_t v0, int64_t vc, cudaStream_t st, bool pdl) {
  CUtensorMap dz_k = {}, w = {}, part = {}, dz_mn = {}, h = {}, dw = {};
  if (c.d_h && (!map_k(&dz_k, dz, c.T, vc, c.ws.vchunk, c.a_rows()) ||
                !map_mn(&w, static_cast<const __nv_bfloat16*>(c.W) + v0 * c.H, vc, c.H, c.H) ||
                !map_out(&part, c.f(c.ws.part), c.H, c.T, c.ws.split, c.H, false)))
    return GRPO_ERR_UNSUPPORTED;
  if (c.dW && (!map_mn(&dz_mn, dz, c.T, vc, c.ws.vchunk) || !map_mn(&h, c.h_src, c.T, c.H, c.H) ||
               !map_out(&dw, static_cast<uint8_t*>(c.dW) + v0 * c.H * (c.dw_bf16 ? 2 : 4), c.H, vc, 1, c.H, c.dw_bf16)))
    return GRPO_ERR_UNSUPPORTED;
  BwdArgs g{};
  g.T = c.T;
  g.a_rows = c.a_rows();
  g.H = c.H;
  g.vc = vc;
  g.with_dh = c.d_h != nullptr;
  g.with_dw = c.dW != nullptr;
  g.split = (int)std::min<int64_t>(c.ws.split, (vc + BK - 1) / BK);  // (the last piece may have few K blocks)
  g.dh_accumulate = chunk > 0;
  g.dw_accumulate = c.dw_accumulate;
  g.dw_bf16 = c.dw_bf16;
  g.dw_scale = c.scale;
  g.live_n = c.live_n;
  g.acc = c.acc;
  const int64_t n_nt = (c.H + BN - 1) / BN, rows = BM * CG;
  const int64_t units = n_nt * ((c.d_h ? (c.T + rows - 1) / rows * g.split : 0) + (c.dW ? (vc + rows - 1) / rows : 0));
  return launch_units<CG, Shape<CG, EPI_CE_STORE>, &bwd_kernel<CG>>(units, st, pdl, dz_k, w, part, dz_mn, h, dw, g);
}

int ce_backward(const CeCall& c, const CeDzArgs& kept, bool kept_done) {
  std::unique_lock<std::mutex> lock;
  Overlap* ov = overlap_on() && c.ws.n_chunks > 1 ? overlap_state(lock, c.st) : nullptr;
  const cudaStream_t bst = ov ? ov->aux : c.st;
  auto pieces = [&]() -> int {
    for (int i = 0; i < c.ws.n_chunks; ++i) {
      const int ct0 = i * c.ws.chunk_tiles, nct = std::min(c.ws.chunk_tiles, c.ws.n_col_tiles - ct0);
      const int64_t v0 = (int64_t)ct0 * BN, vc = std::min<int64_t>((int64_t)nct * BN, c.V - v0);
      __nv_bfloat16* dz = reinterpret_cast<__nv_bfloat16*>(c.base + c.ws.dz[ov ? i & 1 : 0]);
      if (ov && i >= 2) GRPO_CUDA_TRY(cudaStreamWaitEvent(c.st, ov->buf_free[i & 1], 0));
      int rc;
      if (c.ws.keep) {
        const int64_t gx = (c.V + 2047) / 2048, gy = std::min<int64_t>(c.T, std::max<int64_t>(1, (int64_t)sm_count() * 16 / gx));
        rc = kept_done ? GRPO_OK
                       : launch_dep(c.cap > 0.f ? ce_dz_kernel<true> : ce_dz_kernel<false>,
                                    dim3((unsigned)gx, (unsigned)gy), 256, c.st, kept);
      } else {
        GemmArgs g{};
        g.lse2 = c.f(c.ws.lse2);
        g.coef = c.f(c.ws.coef);
        g.ea = c.f(c.ws.ea);
        g.ce_hot = 1.f - c.smoothing;
        g.ce_smooth = c.smoothing / (float)c.V;
        g.dz = dz;
        g.ldz = c.ws.vchunk;
        g.v0 = v0;
        g.col_tile0 = ct0;
        g.n_n = nct;
        g.live_mode = c.live_n ? LIVE_ROWS_PADDED : LIVE_NONE;
        rc = ce_logits<EPI_CE_DLOGITS, EPI_CE_DLOGITS_CAP>(c, g, c.st, vc, !(ov && i >= 2));
      }
      if (rc != GRPO_OK) return rc;
      if (ov) {
        GRPO_CUDA_TRY(cudaEventRecord(ov->dz_ready, c.st));
        GRPO_CUDA_TRY(cudaStreamWaitEvent(bst, ov->dz_ready, 0));
      }
      rc = c.cg == 2 ? ce_products<2>(c, dz, i, v0, vc, bst, !ov) : ce_products<1>(c, dz, i, v0, vc, bst, !ov);
      if (rc != GRPO_OK) return rc;
      if (ov) GRPO_CUDA_TRY(cudaEventRecord(ov->buf_free[i & 1], bst));
    }
    if (c.d_h) {
      const int H4 = (int)(c.H / 4);
      // Eight threads to a vector where the vectors alone are too few to fill the SMs; one where they do (999 x
      // 1000: 9 us against 12 with eight). A constant, not the device's SMs: the order of the sums follows from it.
      const bool wide = c.ws.split > 4 && c.T * H4 < 152 * 1024;
      auto kern = wide ? ce_dh_kernel<8> : ce_dh_kernel<1>;
      const int64_t per = wide ? 32 : 256, blocks = std::min<int64_t>((c.T * H4 + per - 1) / per, (int64_t)sm_count() * 16);
      const int rc = launch_dep(kern, dim3((unsigned)blocks), 256, bst, c.live_n, c.idx, c.T, H4, c.f(c.ws.part), c.ws.split,
                                c.scale, c.d_h, c.dh_bf16);
      if (rc != GRPO_OK) return rc;
    }
    return GRPO_OK;
  };
  int rc = pieces();
  // the caller's stream continues after every launch of the call (also after an error)
  if (ov && (cudaEventRecord(ov->joined, bst) != cudaSuccess || cudaStreamWaitEvent(c.st, ov->joined, 0) != cudaSuccess)) {
    (void)cudaGetLastError();
    if (rc == GRPO_OK) rc = GRPO_ERR_CUDA;
  }
  return rc;
}

// Whether [a, a + n) and [b, b + m) meet (NULL meets nothing).
bool meet(const void* a, size_t n, const void* b, size_t m) {
  const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
  return a && b && x < y + m && y < x + n;
}

bool known_dtype(int32_t d) { return d == GRPO_DTYPE_F32 || d == GRPO_DTYPE_BF16; }

}  // namespace

extern "C" GRPO_API size_t grpo_lmhead_ce_workspace_size(int64_t T, int64_t V, int64_t H) {
  if (T <= 0 || V <= 0 || H <= 0 || T > INT32_MAX / 2 || V > INT32_MAX / 2 || H > kCeMaxH) return 0;
  return ce_layout(T, V, H).total;
}

extern "C" GRPO_API int grpo_lmhead_ce_fwd_bwd(const void* h, const void* W, int64_t T, int64_t V, int64_t H,
                                               const int32_t* target, const uint8_t* mask, const grpo_ce_terms* terms,
                                               float grad_scale, void* d_h, int32_t d_h_dtype, void* dW,
                                               int32_t dW_dtype, uint32_t flags, float* loss_tok, float* logp_tok,
                                               float* lse_tok, grpo_step_acc* acc, void* workspace,
                                               size_t workspace_bytes, void* stream) {
  const grpo_ce_terms none = {0.f, 0.f, 0.f, nullptr};
  const grpo_ce_terms& tm = terms ? *terms : none;
  if (!(tm.label_smoothing >= 0.f && tm.label_smoothing <= 1.f) || !(tm.z_loss >= 0.f && std::isfinite(tm.z_loss)))
    return GRPO_ERR_INVALID;
  if (tm.soft_cap != 0.f && !(tm.soft_cap >= 1e-6f && tm.soft_cap <= 1e6f)) return GRPO_ERR_INVALID;
  if (!std::isfinite(grad_scale)) return GRPO_ERR_INVALID;
  if (T < 0 || V < 1 || H < 8 || H % 8 != 0 || !acc || (uintptr_t)acc % alignof(grpo_step_acc)) return GRPO_ERR_INVALID;
  if (T > INT32_MAX / 2 || V > INT32_MAX / 2 || H > kCeMaxH) return GRPO_ERR_INVALID;
  if (flags & ~(uint32_t)GRPO_LMHEAD_DW_ACCUMULATE) return GRPO_ERR_INVALID;
  if ((d_h && !known_dtype(d_h_dtype)) || (dW && !known_dtype(dW_dtype))) return GRPO_ERR_UNSUPPORTED;
  // (a bf16 sum would be rounded at every call)
  if (dW && (flags & GRPO_LMHEAD_DW_ACCUMULATE) && dW_dtype != GRPO_DTYPE_F32) return GRPO_ERR_INVALID;
  if (T == 0) {
    if (dW && !(flags & GRPO_LMHEAD_DW_ACCUMULATE))
      GRPO_CUDA_TRY(cudaMemsetAsync(dW, 0, (size_t)V * H * (dW_dtype == GRPO_DTYPE_BF16 ? 2 : 4), as_stream(stream)));
    return GRPO_OK;
  }
  if (!h || !W || !target || !loss_tok || !workspace) return GRPO_ERR_INVALID;
  if (((uintptr_t)h | (uintptr_t)W | (uintptr_t)d_h | (uintptr_t)dW) & 15u || ((uintptr_t)workspace & 255u))
    return GRPO_ERR_INVALID;
  const size_t nh = (size_t)T * H, nw = (size_t)V * H;
  const size_t bh = nh * (d_h_dtype == GRPO_DTYPE_BF16 ? 2 : 4), bw = nw * (dW_dtype == GRPO_DTYPE_BF16 ? 2 : 4);
  if (meet(d_h, bh, h, nh * 2) || meet(d_h, bh, W, nw * 2) || meet(d_h, bh, dW, bw) || meet(dW, bw, h, nh * 2) ||
      meet(dW, bw, W, nw * 2))
    return GRPO_ERR_INVALID;
  CeCall c{};
  c.ws = ce_layout(T, V, H);
  if (workspace_bytes < c.ws.total) return GRPO_ERR_CAPACITY;
  c.h_src = h;
  c.W = W;
  c.T = T;
  c.V = V;
  c.H = H;
  c.target = target;
  c.smoothing = tm.label_smoothing;
  c.cap = tm.soft_cap;
  c.scale = grad_scale;
  c.d_h = d_h;
  c.dW = dW;
  c.dh_bf16 = d_h_dtype == GRPO_DTYPE_BF16;
  c.dw_bf16 = dW_dtype == GRPO_DTYPE_BF16;
  c.dw_accumulate = (flags & GRPO_LMHEAD_DW_ACCUMULATE) != 0;
  c.cg = ce_cta_group(T, c.ws.n_col_tiles);
  c.acc = acc;
  c.base = static_cast<uint8_t*>(workspace);
  c.st = as_stream(stream);
  bool pdl = false;  // whether a kernel of this call comes before
  if (mask) {
    int32_t* idx = reinterpret_cast<int32_t*>(c.base + c.ws.idx);
    int32_t* live_n = reinterpret_cast<int32_t*>(c.base + c.ws.live_n);
    __nv_bfloat16* h_live = reinterpret_cast<__nv_bfloat16*>(c.base + c.ws.h_live);
    // 16 tokens a block or more, no more blocks than 8 to an SM
    const int64_t per = ((T + (int64_t)sm_count() * 8 - 1) / ((int64_t)sm_count() * 8) + 15) / 16 * 16;
    ce_compact_kernel<<<(unsigned)((T + per - 1) / per), kCompactThreads, 0, c.st>>>(
        T, per, (int)H, mask, static_cast<const __nv_bfloat16*>(h), idx, live_n, h_live, d_h, (int)(H / (c.dh_bf16 ? 8 : 4)));
    GRPO_CUDA_TRY(cudaGetLastError());
    c.h_src = h_live;
    c.idx = idx;
    c.live_n = live_n;
    pdl = true;
  }
  GemmArgs g{};
  g.part_m = c.f(c.ws.part_m);
  g.part_s = c.f(c.ws.part_s);
  g.part_s2 = c.smoothing > 0.f ? c.f(c.ws.part_z) : nullptr;
  g.n_n = c.ws.n_col_tiles;
  g.live_mode = c.live_n ? LIVE_ROWS : LIVE_NONE;
  g.keep = c.ws.keep && (d_h || dW);
  int rc = ce_logits<EPI_CE_PARTIALS, EPI_CE_PARTIALS_CAP>(c, g, c.st, 0, pdl);
  if (rc != GRPO_OK) return rc;
  CeReduceArgs r{};
  r.T = T;
  r.V = V;
  r.n_col_tiles = c.ws.n_col_tiles;
  r.part_m = g.part_m;
  r.part_s = g.part_s;
  r.part_z = g.part_s2;
  r.zy = c.f(c.ws.zy);
  r.target = target;
  r.w_tok = tm.w_tok;
  r.smoothing = c.smoothing;
  r.z_loss = tm.z_loss;
  r.lse2 = c.f(c.ws.lse2);
  r.coef = c.f(c.ws.coef);
  r.ea = c.f(c.ws.ea);
  r.loss_tok = loss_tok;
  r.logp_tok = logp_tok;
  r.lse_tok = lse_tok;
  r.acc = acc;
  r.idx = c.idx;
  r.live_n = c.live_n;
  const bool grads = d_h || dW;
  const CeDzArgs kept{T, V, c.ws.vchunk, c.f(c.ws.x), reinterpret_cast<__nv_bfloat16*>(c.base + c.ws.dz[0]), target, c.idx,
                      c.live_n, r.lse2, r.coef, r.ea, c.cap, 1.f / c.cap, 1.f - c.smoothing, c.smoothing / (float)V};
  const int64_t gx = (V + 2047) / 2048;
  const bool joint = grads && c.ws.keep && ce_joint(T, gx, c.ws.n_col_tiles);
  rc = joint ? launch_dep(c.cap > 0.f ? ce_reduce_dz_kernel<true> : ce_reduce_dz_kernel<false>,
                          dim3((unsigned)gx, (unsigned)T), 256, c.st, r, kept)
             : launch_dep(ce_reduce_kernel, dim3((unsigned)((T + 31) / 32)), kCeReduceWarps * 32, c.st, r);
  if (rc != GRPO_OK || !grads) return rc;
  return ce_backward(c, kept, joint);
}
