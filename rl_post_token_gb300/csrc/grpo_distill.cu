// Distillation of a student's logits rows from a teacher's top tokens, loss and dlogits in one
// call (formulas in grpo_distill.cuh). Per row: the softmax sums over its tiles (grpo_vocab.cuh; the
// tail kinds leave the listed tokens out of them and add them singly), the list's arithmetic by one
// warp, and dlogits over the tiles again.
//
// Two kernels with the same bits, chosen at the end of the file:
//  * cluster_kernel  the row stays in the shared memory of a cluster of 1 to 8 CTAs between its two
//                    readings, so HBM sees one read and one write of it
//  * row_kernel      one CTA per row, the second reading from L2 (or HBM, where the rows at work are
//                    larger): short and very long rows, and the loss alone of many rows
#include <algorithm>
#include <cmath>
#include <mutex>

#include "grpo_distill.cuh"

namespace grpo {

size_t max_smem_optin();

namespace distill {

struct Args {
  const void* logits;
  int64_t T, V, ld;
  const int64_t* tok_src;
  const int32_t* top_idx;
  const float* top_logp;
  int64_t ld_top;
  int32_t K;
  const uint8_t* mask;
  const float* w_tok;
  float c;      // log2(e) / temperature
  float scale;  // grad_scale / temperature
  void* dlogits;
  int64_t ld_out;
  float* loss_tok;
  grpo_step_acc* acc;
  int32_t n_tiles;
  int32_t slots;           // cluster_kernel: tile slots per CTA
  int32_t n_blocks, fold;  // row_kernel: `fold` consecutive tiles per kept partial
};

// What the list's warp leaves for the others.
struct Stats {
  float shift, mult;  // dlogits = mult 2^(z c - shift) outside the list, c = scale_at(shift)
};

__device__ __forceinline__ float grad_scale_of(const Args& a, int64_t src) {
  return a.w_tok ? a.scale * a.w_tok[src] : a.scale;
}

__device__ __forceinline__ void count(grpo_step_acc* acc, unsigned long long tokens, unsigned long long valid,
                                      unsigned long long nonfinite) {
  if (tokens) atomicAdd(reinterpret_cast<unsigned long long*>(&acc->n_tokens), tokens);
  if (valid) atomicAdd(reinterpret_cast<unsigned long long*>(&acc->n_valid), valid);
  if (nonfinite) atomicAdd(reinterpret_cast<unsigned long long*>(&acc->n_nonfinite), nonfinite);
}

// Calls f(d, k) in every lane for each listed token of the tile, d its element of the tile and k its
// place in the list: the warp looks at 32 entries at a time.
template <typename T, typename F>
__device__ __forceinline__ void for_listed(const int32_t* sh_tok, int K, int64_t e0, int64_t n, F f) {
  const int lane = (int)(threadIdx.x & 31);
#pragma unroll 1
  for (int k0 = 0; k0 < K; k0 += 32) {
    const int64_t tok = sh_tok[k0 + lane], d = tok - e0;
    unsigned hits = __ballot_sync(0xffffffffu, tok >= 0 && d >= 0 && d < n);
    for (; hits; hits &= hits - 1) {
      const int l = __ffs(hits) - 1;
      f(__shfl_sync(0xffffffffu, (int)d, l), k0 + l);
    }
  }
}

// The listed elements of this lane's vectors set to -inf (vectors as tile_vec has them).
template <typename T>
__device__ __forceinline__ void drop_listed(uint4 (&x)[kTileVecs], const int32_t* sh_tok, int K, int tile, int lane) {
  constexpr int E = 16 / (int)sizeof(T);
  for_listed<T>(sh_tok, K, (int64_t)tile * tile_elems<T>(), tile_elems<T>(), [&](int d, int) {
    const int j = d / E, l = (j >> 2) & 31, u = (j >> 7) * 4 + ((j - (l >> 1)) & 3);
    if (l == lane) {
      // word of the lane's 32, and what of it stays
      const int at = u * 4 + (sizeof(T) == 2 ? (d % E) >> 1 : d % E);
      const uint32_t keep = sizeof(T) == 2 ? (d & 1 ? 0x0000FFFFu : 0xFFFF0000u) : 0u;
      const uint32_t ninf = (sizeof(T) == 2 ? 0xFF80FF80u : 0xFF800000u) & ~keep;
#pragma unroll
      for (int v = 0; v < kTileVecs; ++v) {
        if (at == 4 * v) x[v].x = (x[v].x & keep) | ninf;
        if (at == 4 * v + 1) x[v].y = (x[v].y & keep) | ninf;
        if (at == 4 * v + 2) x[v].z = (x[v].z & keep) | ninf;
        if (at == 4 * v + 3) x[v].w = (x[v].w & keep) | ninf;
      }
    }
  });
}

// The same for a tile in shared memory, before it is read: `tile0` is its first element's address.
template <typename T>
__device__ __forceinline__ void drop_listed_smem(uint32_t tile0, const int32_t* sh_tok, int K, int tile, int lane) {
  const int64_t e0 = (int64_t)tile * tile_elems<T>();
#pragma unroll 1
  for (int k0 = 0; k0 < K; k0 += 32) {
    const int64_t tok = sh_tok[k0 + lane], d = tok - e0;
    if (tok >= 0 && d >= 0 && d < tile_elems<T>()) {
      const uint32_t at = tile0 + (uint32_t)d * (uint32_t)sizeof(T);
      if constexpr (sizeof(T) == 2)
        asm volatile("st.shared.u16 [%0], %1;" ::"r"(at), "h"((uint16_t)0xFF80u) : "memory");
      else
        asm volatile("st.shared.u32 [%0], %1;" ::"r"(at), "r"(0xFF800000u) : "memory");
    }
  }
  __syncwarp();
}

template <typename T>
__device__ __forceinline__ void put_elem(T* p, float v) {
  if constexpr (sizeof(T) == 2)
    *p = __float2bfloat16_rn(v);
  else
    *p = v;
}

// The dlogits of a vector.
template <typename T>
__device__ __forceinline__ uint4 grad_vec(const uint4& v, float c, const Stats& s) {
  constexpr int E = 16 / (int)sizeof(T);
  float f[E];
  vec_floats<T>(v, f);
  const float2 c2 = make_float2(c, c), m2 = make_float2(-s.shift, -s.shift), g2 = make_float2(s.mult, s.mult);
#pragma unroll
  for (int i = 0; i < E; i += 2) {
    const float2 t = __ffma2_rn(make_float2(f[i], f[i + 1]), c2, m2);
    const float2 e = __fmul2_rn(make_float2(ex2(t.x), ex2(t.y)), g2);
    f[i] = e.x;
    f[i + 1] = e.y;
  }
  if constexpr (sizeof(T) == 2)
    return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
  else
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
}

// Elements [i0, i1) of a vector to p[i0].., one by one.
template <typename T>
__device__ __noinline__ void store_elems(T* p, uint4 v, int i0, int i1) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 16 / (int)sizeof(T); ++i)
    if (i >= i0 && i < i1) {
      if constexpr (sizeof(T) == 2)
        reinterpret_cast<uint16_t*>(p)[i] = (uint16_t)(w[i / 2] >> (16 * (i & 1)));
      else
        reinterpret_cast<uint32_t*>(p)[i] = w[i];
    }
}

// A vector stored to a row from element e0 on (cut at the row's end), a row of any alignment. Only rows
// of dlogits that lie otherwise in their 16 bytes than their logits come here.
template <typename T>
__device__ __forceinline__ void store_vec(T* row, int64_t e0, int64_t V, const uint4& v) {
  if (e0 < V) store_elems(row + e0, v, 0, (int)min((int64_t)(16 / (int)sizeof(T)), V - e0));
}

// Aligned vector j of those that hold a row, `off` the row's bytes past a 16-byte boundary; what the
// vector holds outside the row stays as it is.
template <typename T>
__device__ __forceinline__ void store_cover(T* row, int64_t j, int off, int64_t V, const uint4& v) {
  constexpr int E = 16 / (int)sizeof(T);
  T* p = reinterpret_cast<T*>(reinterpret_cast<uint8_t*>(row) + j * 16 - off);
  const int64_t e0 = (j * 16 - off) / (int64_t)sizeof(T);  // (a multiple of the element, also below 0)
  if (e0 >= 0 && e0 + E <= V)
    *reinterpret_cast<uint4*>(p) = v;
  else if (e0 < V)
    store_elems(p, v, e0 < 0 ? (int)-e0 : 0, (int)min((int64_t)E, V - e0));
}

// ------------------------------------------------------------------------------------------
// One CTA per row.
// ------------------------------------------------------------------------------------------
constexpr int kMaxBlocks = 384;  // softmax partials kept per row: the tiles of the cluster kernel's longest

template <typename T, int KIND, bool ALIGNED, int NT>
__global__ void __launch_bounds__(NT, NT == 128 ? 8 : 1) row_kernel(Args a) {
  __shared__ alignas(16) float sh_list[Entries::kWords * GRPO_TOPK_MAX];
  __shared__ float sh_corr[GRPO_TOPK_MAX], pm[kMaxBlocks], ps[kMaxBlocks];
  __shared__ Stats stats;
  constexpr int E = 16 / (int)sizeof(T), NW = NT / 32;
  constexpr bool TAIL = KIND != GRPO_DISTILL_FORWARD_TOPK;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const Entries entries(sh_list, padded_list(a.K));
  const int64_t V = a.V, nvec = (V + E - 1) / E;
  unsigned long long c_tok = 0, c_val = 0, c_bad = 0;
  for (int64_t row_i = blockIdx.x; row_i < a.T; row_i += gridDim.x) {
    const int64_t src = a.tok_src ? a.tok_src[row_i] : row_i;
    const T* row = static_cast<const T*>(a.logits) + row_i * a.ld;
    T* dz = a.dlogits ? static_cast<T*>(a.dlogits) + row_i * a.ld_out : nullptr;
    const int off = dz ? row_off(dz) : 0;
    const bool valid = src >= 0 && a.mask[src] != 0;
    ++c_tok;
    if (!valid) {
      if (tid == 0 && src >= 0) a.loss_tok[src] = 0.f;
      if (dz)
        for (int64_t j = tid; j <= nvec; j += NT) store_cover(dz, j, off, V, make_uint4(0, 0, 0, 0));
      continue;
    }
    ++c_val;
    List<T, KIND> list(entries, a.K, V, lane);
    if (warp == 0) list.load(a.top_idx + src * a.ld_top, a.top_logp + src * a.ld_top, row);
    if (TAIL) __syncthreads();
    for (int b = warp; b < a.n_blocks; b += NW) {
      Part p{-INFINITY, 0.f, 0.f};
      for (int f = 0; f < a.fold; ++f) {
        const int tile = b * a.fold + f;
        if (tile >= a.n_tiles) break;
        uint4 x[kTileVecs];
#pragma unroll
        for (int u = 0; u < kTileVecs; ++u)
          x[u] = load_vec<T, ALIGNED>(row, (int64_t)tile * (32 * kTileVecs) + tile_vec(lane, u), V);
        if (TAIL) drop_listed<T>(x, entries.tok, a.K, tile, lane);
        const Part tp = tile_part<T, false>(x, warp_max_nan(tile_lane_max<T>(x)), a.c);
        p = f == 0 ? tp : part_join(p, tp);
      }
      if (lane == 0) {
        pm[b] = p.m;
        ps[b] = p.s;
      }
    }
    __syncthreads();
    if (warp == 0) {
      Stats st;
      bool finite;
      const float g = grad_scale_of(a, src);
      list.stats(join_blocks(a.n_blocks, lane, [&](int i) { return make_float2(pm[i], ps[i]); }), a.c, g, st.shift, st.mult);
      const float loss = list.token_loss(g, finite);
      for (int k = lane; k < list.padded; k += 32) sh_corr[k] = list.entry_grad(k, g);
      if (lane == 0) {
        a.loss_tok[src] = loss;
        stats = st;
        if (!finite) ++c_bad;
      }
    }
    __syncthreads();
    if (dz) {
      const Stats st = stats;
      const float c = scale_at(st.shift, a.c);
      if (ALIGNED || off == row_off(row)) {
        for (int64_t j = tid; j <= nvec; j += NT) {
          uint4 v = make_uint4(0, 0, 0, 0);
          if (st.mult != 0.f) v = grad_vec<T>(load_cover<T, ALIGNED>(row, j, off, V), c, st);
          store_cover(dz, j, off, V, v);
        }
      } else {
        for (int64_t j = tid; j < nvec; j += NT) {
          uint4 v = make_uint4(0, 0, 0, 0);
          if (st.mult != 0.f) v = grad_vec<T>(load_vec<T, ALIGNED>(row, j, V), c, st);
          store_vec(dz, j * E, V, v);
        }
      }
      __syncthreads();
      for (int k = tid; k < a.K; k += NT)
        if (entries.tok[k] >= 0) put_elem(dz + entries.tok[k], sh_corr[k]);
    }
    __syncthreads();  // the shared arrays are rewritten by the next row
  }
  if (tid == 0) count(a.acc, c_tok, c_val, c_bad);
}

template <typename T, int KIND, bool ALIGNED, int NT>
int launch_row_nt(const Args& a, int per_sm, cudaStream_t st) {
  const int64_t grid = std::min<int64_t>(a.T, (int64_t)sm_count() * per_sm);
  row_kernel<T, KIND, ALIGNED, NT><<<(unsigned)grid, NT, 0, st>>>(a);
  GRPO_CUDA_TRY(cudaGetLastError());
  return GRPO_OK;
}

// ------------------------------------------------------------------------------------------
// The cluster kernel: persistent clusters of C CTAs, one CTA per SM; the tiles of a row are split
// evenly over the CTAs. Read row k (masked and padding rows are not read) is owned by CTA k % C, which
// does its list's arithmetic. Warps of a CTA:
//   0, 1    producers: fetch the CTA's tiles, row after row, into a ring of slots, as far ahead as there
//           are free ones; warp 0 puts every row's listed tokens into shared memory
//   2, 3    lists of the rows this CTA owns, in turn: loads a list and the listed logits ahead of time,
//           joins the row's partials once all have arrived, and sends what pass 2 needs (stats, the
//           listed tokens' dlogits) to every CTA
//   4..19   the tiles, dealt to the 16 warps in turn, from row to row on where a row has one for every
//           warp (each row from warp 4 on: 818 us at 8192 x 151936 bf16, so 811). Pass 1: the tile's
//           partial, sent to the row's owner. Pass 2: dlogits from the same slot, the listed tokens'
//           over them; then the slot is free.
// Everything sent goes by asynchronous stores that an mbarrier of the receiver counts, so nobody waits
// for a cluster barrier. The list's arithmetic by every CTA of the cluster (no owner) took 1.9x at C = 4:
// a list is thousands of cycles of latency. Pass 1 of a row before pass 2 of the row before it hides the
// exchange, but leaves no free slots (8192 x 50257 bf16: 499 against 398 us) or takes more CTAs a row,
// each with its own waits (8192 x 151936 on 4: 892 against 785, one producer).
//
// 8192 x 151936 bf16, K = 64: 752 us, 6.63 TB/s, bound by HBM (reads and writes mixed; 735 us at the copy
// rate); FORWARD_TAIL 824, REVERSE_TAIL 856. On rows of 25 tiles the exchange and the two rounds of tiles are
// longer than the row's share of the bandwidth, 243 us: 50264 columns, K = 37, 290 us (330 and 342); 50257,
// whose tiles are shifted as they are read and whose rows' ends are filled in, 391 (406 and 419).
//
// Barriers: full/empty of the slots; listed[k & 1] (the tokens are in shared memory; the tail kinds,
// which need them in pass 1); parts (owner, per list warp: the row's partials are in); ready[k & 1] (the
// stats are in, and the tokens); grads[k & 1] (the list's dlogits are in). Why no buffer is rewritten too
// early: the partials of row k are complete only when every tile warp of the cluster is through pass 1 of
// row k, hence through pass 2 of row k - 1. So what is sent to ready[k & 1] and grads[k & 1] then finds row
// k - 2 done with in every CTA, and no phase of ready, grads, listed or parts is overtaken by a round. The
// tokens of row k are written when the stats of row k - 2 have come, with which row k - 3 is done with:
// they have four buffers. Warps without a tile in the CTA's rows wait for nothing; where rows have fewer
// tiles than warps, the same warps work on all of them, so that "every tile warp" holds.
// ------------------------------------------------------------------------------------------
constexpr int kTileWarps = 16;
constexpr int kListWarps = 2;  // (3: 4% slower at 152K and 10% at 50K, issue slots)
constexpr int kIssueWarps = 2;  // producers: the even slots and the odd ones
constexpr int kIssueLanes = 4;  // tiles that one of them issues together
constexpr int kFirstListWarp = kIssueWarps;
constexpr int kFirstTileWarp = kFirstListWarp + kListWarps;
constexpr int kClusterThreads = (kFirstTileWarp + kTileWarps) * 32;
constexpr int kMaxTiles = kMaxBlocks;
constexpr int kMaxSlots = 56;
constexpr int kMinTiles = 16;

struct ClusterShared {
  Stats stats[2];
  uint64_t full[kMaxSlots], empty[kMaxSlots];
  uint64_t parts[kListWarps], listed[2], ready[2], grads[2];
  int abort;
};

// Behind it, sized by the call: entries[kListWarps] (Entries), tok[4] and corr[2] (lists), part[kListWarps]
// ((m, s) of every tile of an owned row), and on the next 128 bytes the ring.
struct ClusterLayout {
  int padded;
  uint32_t entries, tok, corr, part, ring;  // byte offsets
  __host__ __device__ ClusterLayout(int K, int n_tiles) : padded(padded_list(K)) {
    entries = (uint32_t)(sizeof(ClusterShared) + 15) / 16 * 16;
    tok = entries + 4u * kListWarps * Entries::kWords * padded;
    corr = tok + 4u * 4 * padded;
    part = corr + 4u * 2 * padded;
    ring = (part + 8u * kListWarps * n_tiles + 127) / 128 * 128;
  }
};

template <typename T, int KIND, bool ALIGNED>
__global__ void __launch_bounds__(kClusterThreads, 1) cluster_kernel(Args a, int C) {
  extern __shared__ __align__(128) uint8_t smem_raw[];
  ClusterShared& sh = *reinterpret_cast<ClusterShared*>(smem_raw);
  const ClusterLayout at(a.K, a.n_tiles);
  uint8_t* ring = smem_raw + at.ring;
  int32_t* sh_tok = reinterpret_cast<int32_t*>(smem_raw + at.tok);
  float* sh_corr = reinterpret_cast<float*>(smem_raw + at.corr);
  float2* sh_part = reinterpret_cast<float2*>(smem_raw + at.part);
  const int padded = at.padded;
  constexpr int E = 16 / (int)sizeof(T);
  constexpr bool TAIL = KIND != GRPO_DISTILL_FORWARD_TOPK;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = (int)cluster_ctarank();
  const int64_t first = blockIdx.x / C, stride = gridDim.x / C;
  const int64_t V = a.V;
  const int S = a.slots;
  const int t0 = rank * a.n_tiles / C, mine = (rank + 1) * a.n_tiles / C - t0;  // tiles of this CTA
  volatile int* s_abort = &sh.abort;
  if (tid == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(&sh.full[s], 1);
      mbar_init(&sh.empty[s], 1);
    }
    for (int b = 0; b < kListWarps; ++b) mbar_init(&sh.parts[b], 1);
    for (int b = 0; b < 2; ++b) {
      mbar_init(&sh.listed[b], 1);
      mbar_init(&sh.ready[b], 1);
      mbar_init(&sh.grads[b], 1);
    }
    sh.abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  __syncthreads();
  cluster_sync_all();  // every CTA's barriers exist

  const T* base = static_cast<const T*>(a.logits);
  auto src_of = [&](int64_t r) -> int64_t { return a.tok_src ? a.tok_src[r] : r; };
  auto is_read = [&](int64_t src) { return src >= 0 && a.mask[src] != 0; };

  if (warp < kIssueWarps) {
    // ---- producers ----
    // A wait on a slot and a copy's issue take 150 to 250 cycles each, together longer than a row's share of
    // the bandwidth for one warp: two take turns, a few lanes issue together, and a batch waits for its own
    // slots alone, so that what is free is filled while the tiles' warps wait for the list (8192 x 151936
    // bf16: one warp, 32 lanes 812 us; two, 16 lanes 806; two, 4 lanes 757). Tiles at a row's ends, which the
    // whole warp fills up, come after the others. A slot belongs to one producer: were it another's turn, a
    // wait for the slot's last use could take the use before it for it (their parity is the same).
    int slot0 = 0;         // slot of the row's first tile
    uint32_t round0 = 0;   // times the ring had gone round there
    bool ok = true;
    int64_t nsrc = first < a.T ? src_of(first) : -1;
    bool nread = first < a.T && is_read(nsrc);
    uint32_t k = 0;
    int32_t tok[GRPO_TOPK_MAX / 32];
    auto load_tokens = [&](int64_t src) {
#pragma unroll
      for (int j = 0; j < GRPO_TOPK_MAX / 32; ++j) {
        tok[j] = -1;
        if (32 * j + lane < a.K) tok[j] = a.top_idx[src * a.ld_top + 32 * j + lane];
        if (tok[j] < 0 || (int64_t)tok[j] >= V) tok[j] = -1;
      }
    };
    if (warp == 0 && nread) load_tokens(nsrc);
    for (int64_t r = first; r < a.T && ok; r += stride) {
      const bool read = nread;
      if (r + stride < a.T) {  // the next row's index and mask while this row's tiles are issued
        nsrc = src_of(r + stride);
        nread = is_read(nsrc);
      } else {
        nread = false;
      }
      if (!read) {
        if (warp == 0 && nread) load_tokens(nsrc);
        continue;
      }
      if (warp == 0) {  // the tokens first: the tail kinds' pass 1 waits for them
        const int buf = (int)(k & 1u);
        if (k >= 2) {
          mbar_wait_bounded(&sh.ready[buf], ((k >> 1) - 1u) & 1u, s_abort);
          if (a.dlogits) mbar_wait_bounded(&sh.grads[buf], ((k >> 1) - 1u) & 1u, s_abort);
        }
#pragma unroll
        for (int j = 0; j < GRPO_TOPK_MAX / 32; ++j)
          if (32 * j < a.K) sh_tok[(int)(k & 3u) * padded + 32 * j + lane] = tok[j];
        __syncwarp();
        if (lane == 0) {
          if (TAIL) mbar_arrive(&sh.listed[buf]);
          // the row's stats and its list's dlogits will be counted (and the tokens are published)
          mbar_arrive_expect_tx(&sh.ready[buf], 8u);
          if (a.dlogits) mbar_arrive_expect_tx(&sh.grads[buf], 4u * (uint32_t)padded);
        }
        ++k;
        if (nread) load_tokens(nsrc);
      }
      const T* row = base + r * a.ld;
      const int off = ALIGNED ? 0 : row_off(row);
      const uint32_t bytes = kTileBytes + (off ? 16u : 0u);
      auto edge = [&](int i) { return (t0 + i == 0 && off) || t0 + i >= a.n_tiles - 2; };
      // the row's tiles up to the ring's end, then those from its start on
      const int n1 = min(mine, S - slot0);
#pragma unroll 1
      for (int part = 0; part < 2 && ok; ++part) {
        const int lo = part ? n1 : 0, hi = part ? mine : n1;  // tile i is in slot base_slot + i
        const int base_slot = part ? -n1 : slot0;
        const uint32_t round = round0 + (part ? 1u : 0u);
        for (int i0 = lo + ((base_slot + lo + warp) & 1); i0 < hi && ok; i0 += kIssueWarps * kIssueLanes) {
          if (round > 0)
            for (int i = i0; i < min(hi, i0 + kIssueWarps * kIssueLanes) && ok; i += kIssueWarps)
              ok = mbar_wait_bounded(&sh.empty[base_slot + i], (round - 1) & 1u, s_abort);
          ok = __all_sync(0xffffffffu, ok);
          const int i = i0 + lane * kIssueWarps;
          if (ok && lane < kIssueLanes && i < hi && !edge(i)) {
            const int slot = base_slot + i;
            // (the tail kinds' warps have written to the slot)
            if (TAIL) fence_proxy_async_smem();
            mbar_arrive_expect_tx(&sh.full[slot], bytes);
            bulk_g2s(ring + (size_t)slot * kSlotBytes,
                     reinterpret_cast<const uint8_t*>(row) + (int64_t)(t0 + i) * kTileBytes - off, bytes, &sh.full[slot]);
          }
          __syncwarp();
        }
      }
      // (their slots are free: the waits above took in every tile)
      for (int i = 0; i < mine && ok; ++i) {
        if (!edge(i)) {
          if (t0 + i < a.n_tiles - 3) i = max(i, min(mine, a.n_tiles - 2 - t0) - 1);  // on to the last tiles
          continue;
        }
        const int slot = i < n1 ? slot0 + i : i - n1;
        if (slot % kIssueWarps != warp) continue;
        if (TAIL) fence_proxy_async_smem();
        fetch_tile<T>(ring + (size_t)slot * kSlotBytes, row, off, t0 + i, a.n_tiles, V, lane, &sh.full[slot]);
      }
      ok = !__any_sync(0xffffffffu, *s_abort);
      slot0 += mine;
      if (slot0 >= S) {
        slot0 -= S;
        ++round0;
      }
    }
    // a wait gave up: let the copies in flight land before the CTA's memory goes away (bounded; a slot
    // whose copy was not issued runs into the limit)
    if (!ok || *s_abort) {
      const uint64_t begin = global_timer_ns();
      for (int s = lane; s < S; s += 32) {
        const uint32_t filled = round0 + (s < slot0 ? 1u : 0u);  // fills of the slot so far
        while (filled > 0 && !mbar_try_wait(&sh.full[s], (filled - 1) & 1u) && global_timer_ns() - begin < 1000000000ull) {}
      }
    }
  } else if (warp < kFirstTileWarp) {
    // ---- the lists of the rows this CTA owns ----
    const int me = warp - kFirstListWarp;
    const Entries entries(smem_raw + at.entries + (uint32_t)me * 4u * Entries::kWords * padded, padded);
    const float2* part = sh_part + me * a.n_tiles;
    unsigned long long c_val = 0, c_bad = 0;
    uint32_t k = 0, own = 0;  // read rows, owned rows so far
    for (int64_t r = first; r < a.T; r += stride) {
      const int64_t src = src_of(r);
      if (!is_read(src)) continue;
      const uint32_t row_k = k++;
      if ((int)(row_k % (uint32_t)C) != rank) continue;
      const uint32_t j_own = own++;
      if ((int)(j_own % kListWarps) != me) continue;
      const uint32_t use = j_own / kListWarps;
      // the partials of all tiles will be counted: 8 bytes each
      if (lane == 0) mbar_arrive_expect_tx_relaxed(&sh.parts[me], 8u * (uint32_t)a.n_tiles);
      List<T, KIND> list(entries, a.K, V, lane);
      list.load(a.top_idx + src * a.ld_top, a.top_logp + src * a.ld_top, base + r * a.ld);
      const float g = grad_scale_of(a, src);
      mbar_wait_bounded(&sh.parts[me], use & 1u, s_abort);
      const Part p = join_blocks(a.n_tiles, lane, [&](int i) { return part[i]; });
      Stats st;
      bool finite;
      list.stats(p, a.c, g, st.shift, st.mult);
      const int buf = (int)(row_k & 1u);
      if (lane < C)
        st_async_v2f32(mapa_u32(smem_u32(&sh.stats[buf]), (uint32_t)lane), st.shift, st.mult,
                       mapa_u32(smem_u32(&sh.ready[buf]), (uint32_t)lane));
      const float loss = list.token_loss(g, finite);
      if (a.dlogits)
        for (int k = lane; k < list.padded; k += 32) {
          const float d = list.entry_grad(k, g);
          const uint32_t dst = smem_u32(sh_corr + buf * padded + k), bar = smem_u32(&sh.grads[buf]);
          for (int c = 0; c < C; ++c) st_async_f32(mapa_u32(dst, (uint32_t)c), d, mapa_u32(bar, (uint32_t)c));
        }
      __syncwarp();  // the entries are rewritten by the next list
      if (lane == 0) a.loss_tok[src] = loss;
      ++c_val;
      if (!finite) ++c_bad;
    }
    if (lane == 0) count(a.acc, 0, c_val, c_bad);
  } else {
    // ---- tiles ----
    const int w = warp - kFirstTileWarp;
    const LaneOffsets lo4(lane);
    const uint32_t ring32 = smem_u32(ring);
    // a read row on its way: where its tiles are (slot of the first, rounds of the ring there), its number
    struct Row {
      T* dz;
      int off, off_out, slot0;  // bytes past a 16-byte boundary of the logits and the dlogits
      uint32_t round0, k;
      int i0;  // this warp's first tile
    };
    auto pass1 = [&](const Row& q) {
      if (w >= mine) return;
      if (TAIL) mbar_wait_bounded(&sh.listed[q.k & 1u], (q.k >> 1) & 1u, s_abort);
      // the row's owner and the list warp there that takes its partials
      const uint32_t owner = q.k % (uint32_t)C, box = (q.k / (uint32_t)C) % kListWarps;
      const uint32_t part = mapa_u32(smem_u32(sh_part + box * a.n_tiles + t0), owner), bar = mapa_u32(smem_u32(&sh.parts[box]), owner);
      for (int i = q.i0; i < mine; i += kTileWarps) {
        int slot = q.slot0 + i;
        uint32_t round = q.round0;
        if (slot >= S) {
          slot -= S;
          ++round;
        }
        mbar_wait_bounded(&sh.full[slot], round & 1u, s_abort);
        const uint32_t tile0 = ring32 + (uint32_t)slot * kSlotBytes;
        if (TAIL) drop_listed_smem<T>(tile0 + (uint32_t)q.off, sh_tok + (int)(q.k & 3u) * padded, a.K, t0 + i, lane);
        uint4 x[kTileVecs];
        read_tile<T, ALIGNED>(tile0, q.off, lo4, x);
        const Part p = tile_part<T, false>(x, warp_max_nan(tile_lane_max<T>(x)), a.c);
        if (lane == 0) st_async_v2f32(part + 8u * (uint32_t)i, p.m, p.s, bar);
      }
    };
    auto pass2 = [&](const Row& q) {
      if (w >= mine) return;
      const int buf = (int)(q.k & 1u);
      mbar_wait_bounded(&sh.ready[buf], (q.k >> 1) & 1u, s_abort);
      const Stats st = sh.stats[buf];
      const float c = scale_at(st.shift, a.c);
      for (int i = q.i0; i < mine; i += kTileWarps) {
        int slot = q.slot0 + i;
        if (slot >= S) slot -= S;
        if (q.dz) {
          const int tile = t0 + i;
          const uint32_t src = ring32 + (uint32_t)slot * kSlotBytes + (uint32_t)lane * 16u;
          const int64_t j0 = (int64_t)tile * (32 * kTileVecs) + lane;
          auto vec = [&](int u, bool shifted) -> uint4 {
            uint4 v = lds128(src + (uint32_t)u * 512u);
            if (shifted) v = shift_vec<T>(v, lds128(src + (uint32_t)u * 512u + 16u), q.off);
            v = grad_vec<T>(v, c, st);
            return st.mult != 0.f ? v : make_uint4(0, 0, 0, 0);
          };
          if (ALIGNED || q.off == q.off_out) {
            // the slot's vectors are aligned vectors of the row of dlogits, too
            uint8_t* out = reinterpret_cast<uint8_t*>(q.dz) - q.off;
            if ((tile > 0 || q.off == 0) && (int64_t)(tile + 1) * kTileBytes - q.off <= V * (int64_t)sizeof(T)) {
#pragma unroll
              for (int u = 0; u < kTileVecs; ++u) reinterpret_cast<uint4*>(out)[j0 + u * 32] = vec(u, false);
            } else {
#pragma unroll 1
              for (int u = 0; u < kTileVecs; ++u) store_cover(q.dz, j0 + u * 32, q.off, V, vec(u, false));
            }
            // and the vector that the last tile reaches into
            if (!ALIGNED && tile == a.n_tiles - 1 && q.off && lane == 0)
              store_cover(q.dz, j0 + kTileVecs * 32, q.off, V, vec(kTileVecs, false));
          } else {
#pragma unroll 1
            for (int u = 0; u < kTileVecs; ++u) store_vec(q.dz, (j0 + u * 32) * E, V, vec(u, q.off != 0));
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.empty[slot]);
      }
      if (!q.dz) return;
      // the listed tokens' over what other lanes have stored (the barriers of the warp above order them)
      mbar_wait_bounded(&sh.grads[buf], (q.k >> 1) & 1u, s_abort);
      const int lead = ALIGNED || q.off == q.off_out ? q.off / (int)sizeof(T) : 0;
      for (int i = q.i0; i < mine; i += kTileWarps) {
        // the elements that this warp has stored
        const int64_t e0 = (int64_t)(t0 + i) * tile_elems<T>() - lead;
        for_listed<T>(sh_tok + (int)(q.k & 3u) * padded, a.K, e0, t0 + i == a.n_tiles - 1 ? V : tile_elems<T>(), [&](int d, int e) {
          if (lane == 0) put_elem(q.dz + e0 + d, sh_corr[buf * padded + e]);
        });
      }
    };
    int slot0 = 0;        // slot of the next row's first tile
    uint32_t round0 = 0;  // times the ring had gone round there
    unsigned long long c_tok = 0;
    uint32_t k = 0;  // read rows so far
    int i0 = w;
    int64_t nsrc = first < a.T ? src_of(first) : -1;
    bool nread = first < a.T && is_read(nsrc);
    for (int64_t r = first; r < a.T; r += stride) {
      const int64_t src = nsrc;
      const bool read = nread;
      if (r + stride < a.T) {
        nsrc = src_of(r + stride);
        nread = is_read(nsrc);
      }
      ++c_tok;
      T* dz = a.dlogits ? static_cast<T*>(a.dlogits) + r * a.ld_out : nullptr;
      const int off_out = !ALIGNED && dz ? row_off(dz) : 0;
      if (!read) {
        if (rank == 0 && w == 0 && lane == 0 && src >= 0) a.loss_tok[src] = 0.f;
        if (dz)
          for (int i = w; i < mine; i += kTileWarps) {
            const int64_t j0 = (int64_t)(t0 + i) * (32 * kTileVecs) + lane;
            for (int u = 0; u < kTileVecs; ++u) store_cover(dz, j0 + u * 32, off_out, V, make_uint4(0, 0, 0, 0));
            if (!ALIGNED && t0 + i == a.n_tiles - 1 && lane == 0)
              store_cover(dz, j0 + kTileVecs * 32, off_out, V, make_uint4(0, 0, 0, 0));
          }
        continue;
      }
      const Row cur{dz, ALIGNED ? 0 : row_off(base + r * a.ld), off_out, slot0, round0, k++, i0};
      if (mine >= kTileWarps) i0 = (i0 + kTileWarps - mine % kTileWarps) % kTileWarps;
      slot0 += mine;
      if (slot0 >= S) {
        slot0 -= S;
        ++round0;
      }
      pass1(cur);
      pass2(cur);
    }
    if (rank == 0 && w == 0 && lane == 0) count(a.acc, c_tok, 0, 0);
  }
  __syncthreads();
  if (*s_abort && tid == 0) atomicOr(&a.acc->flags, kFlagWaitTimeout);
  cluster_sync_all();  // no CTA leaves while a peer may still store into or arrive on its memory
}

// CTAs per row: as few as hold its tiles, and up to 8 where the call has too few rows for the SMs.
int cluster_size(int64_t T, int n_tiles, int slots, int sms) {
  int C = 1;
  while (C * slots < n_tiles) C *= 2;
  while (C < 8 && 2 * C * T <= sms && 2 * C * 2 <= n_tiles) C *= 2;
  return C;
}

int cluster_slots(int K, int n_tiles) {
  const size_t optin = max_smem_optin(), head = ClusterLayout(K, n_tiles).ring;
  return optin > head ? (int)std::min<size_t>(kMaxSlots, (optin - head) / kSlotBytes) : 0;
}

template <typename T, int KIND, bool ALIGNED>
int launch_cluster(Args a, int C, cudaStream_t st) {
  auto kern = cluster_kernel<T, KIND, ALIGNED>;
  const size_t smem = ClusterLayout(a.K, a.n_tiles).ring + (size_t)a.slots * kSlotBytes;
  int dev = 0, n_clusters = 0;
  GRPO_CUDA_TRY(cudaGetDevice(&dev));
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = C;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.blockDim = dim3(kClusterThreads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  {
    static std::mutex mu;
    static bool ready[64] = {};
    static int fit[64][4] = {};  // clusters that run at once, by log2 C
    const int lc = C == 1 ? 0 : C == 2 ? 1 : C == 4 ? 2 : 3;
    std::lock_guard<std::mutex> lock(mu);
    const bool known = dev >= 0 && dev < 64;
    if (!known || !ready[dev]) {
      GRPO_CUDA_TRY(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)max_smem_optin()));
      if (known) ready[dev] = true;
    }
    if (known) n_clusters = fit[dev][lc];
    if (n_clusters == 0) {
      cfg.gridDim = dim3((unsigned)(C * 1024), 1, 1);  // (any smem above half an SM's: one CTA each)
      GRPO_CUDA_TRY(cudaOccupancyMaxActiveClusters(&n_clusters, kern, &cfg));
      if (n_clusters < 1) return GRPO_ERR_UNSUPPORTED;
      if (known) fit[dev][lc] = n_clusters;
    }
  }
  cfg.gridDim = dim3((unsigned)(std::min<int64_t>(a.T, n_clusters) * C), 1, 1);
  GRPO_CUDA_TRY(cudaLaunchKernelEx(&cfg, kern, a, C));
  return GRPO_OK;
}

template <typename T, int KIND, bool ALIGNED>
int launch(Args a, cudaStream_t st) {
  // The cluster kernel where a row has 16 tiles or more and fits, and dlogits are wanted or the rows are
  // fewer than the SMs. 8192 rows of bf16, FORWARD_TOPK, K = 64: 13 tiles, cluster 226 us, row_kernel 247
  // (K = 37: 220 and 224); 17 tiles 278 and 327; 25 tiles 291 and 483. Their loss alone needs no second
  // reading: 17 tiles 180 and 119, 25 tiles 210 and 154; 64 rows of 17 tiles 10 to 12 either way.
  const int sms = sm_count();
  a.slots = cluster_slots(a.K, a.n_tiles);
  if (a.n_tiles >= kMinTiles && a.n_tiles <= kMaxTiles && 8 * a.slots >= a.n_tiles && (a.dlogits || 2 * a.T <= sms))
    return launch_cluster<T, KIND, ALIGNED>(a, cluster_size(a.T, a.n_tiles, a.slots, sms), st);
  a.fold = (a.n_tiles + kMaxBlocks - 1) / kMaxBlocks;
  a.n_blocks = (a.n_tiles + a.fold - 1) / a.fold;
  // many rows: small blocks, eight rows in flight on an SM (2048 x 400008 fp32: 1912 us, one large block each
  // 2589); few: large ones
  if (a.T > 2 * sms) return launch_row_nt<T, KIND, ALIGNED, 128>(a, 8, st);
  return launch_row_nt<T, KIND, ALIGNED, 512>(a, 1, st);
}

template <typename T>
int dispatch(const Args& a, int32_t kind, bool aligned, cudaStream_t st) {
  if (kind == GRPO_DISTILL_FORWARD_TOPK)
    return aligned ? launch<T, GRPO_DISTILL_FORWARD_TOPK, true>(a, st) : launch<T, GRPO_DISTILL_FORWARD_TOPK, false>(a, st);
  if (kind == GRPO_DISTILL_FORWARD_TAIL)
    return aligned ? launch<T, GRPO_DISTILL_FORWARD_TAIL, true>(a, st) : launch<T, GRPO_DISTILL_FORWARD_TAIL, false>(a, st);
  return aligned ? launch<T, GRPO_DISTILL_REVERSE_TAIL, true>(a, st) : launch<T, GRPO_DISTILL_REVERSE_TAIL, false>(a, st);
}

}  // namespace distill
}  // namespace grpo

using namespace grpo;

extern "C" GRPO_API int grpo_distill_topk_fwd_bwd(const void* logits, int32_t dtype, int64_t T, int64_t V, int64_t ld,
                                                  const int64_t* tok_src, const int32_t* top_idx,
                                                  const float* top_logp, int64_t ld_top, int32_t K,
                                                  const uint8_t* mask, int32_t kind, float temperature,
                                                  const float* w_tok, float grad_scale, void* dlogits, int64_t ld_out,
                                                  float* loss_tok, grpo_step_acc* acc, void* stream) {
  if (dtype != GRPO_DTYPE_F32 && dtype != GRPO_DTYPE_BF16) return GRPO_ERR_UNSUPPORTED;
  if (kind != GRPO_DISTILL_FORWARD_TOPK && kind != GRPO_DISTILL_FORWARD_TAIL && kind != GRPO_DISTILL_REVERSE_TAIL)
    return GRPO_ERR_INVALID;
  if (T < 0 || V < 1 || ld < V || V > (int64_t)INT32_MAX || T > (int64_t)INT32_MAX || !acc) return GRPO_ERR_INVALID;
  if (K < 1 || K > GRPO_TOPK_MAX || ld_top < K) return GRPO_ERR_INVALID;
  if (dlogits && ld_out < V) return GRPO_ERR_INVALID;
  if (!(temperature > 0.f) || !std::isfinite(temperature) || !std::isfinite(grad_scale)) return GRPO_ERR_INVALID;
  const float c = (float)(1.4426950408889634 / (double)temperature);
  if (!(c < 0x1p126f) || c < 1.1754944e-38f) return GRPO_ERR_INVALID;  // (its powers of two are float32 numbers)
  if (T == 0) return GRPO_OK;
  if (!logits || !top_idx || !top_logp || !mask || !loss_tok) return GRPO_ERR_INVALID;
  const size_t es = dtype == GRPO_DTYPE_F32 ? 4 : 2;
  const uintptr_t in = reinterpret_cast<uintptr_t>(logits), out = reinterpret_cast<uintptr_t>(dlogits);
  if (in % es || out % es || reinterpret_cast<uintptr_t>(acc) % alignof(grpo_step_acc)) return GRPO_ERR_INVALID;
  // dlogits is written while other rows of the logits are still to be read; the logits' own buffer would not be
  // (each row is read before it is written), but row_kernel reads by the non-coherent path what it writes
  if (dlogits && in < out + ((T - 1) * ld_out + V) * es && out < in + ((T - 1) * ld + V) * es) return GRPO_ERR_INVALID;

  distill::Args a{};
  a.logits = logits;
  a.T = T;
  a.V = V;
  a.ld = ld;
  a.tok_src = tok_src;
  a.top_idx = top_idx;
  a.top_logp = top_logp;
  a.ld_top = ld_top;
  a.K = K;
  a.mask = mask;
  a.w_tok = w_tok;
  a.c = c;
  a.scale = (float)((double)grad_scale / (double)temperature);
  a.dlogits = dlogits;
  a.ld_out = ld_out;
  a.loss_tok = loss_tok;
  a.acc = acc;
  a.n_tiles = (int32_t)((V * (int64_t)es + kTileBytes - 1) / kTileBytes);
  const bool aligned = ((in | out) & 15u) == 0 && (ld * es) % 16 == 0 && (!dlogits || (ld_out * es) % 16 == 0);
  const cudaStream_t st = as_stream(stream);
  return dtype == GRPO_DTYPE_BF16 ? distill::dispatch<__nv_bfloat16>(a, kind, aligned, st)
                                  : distill::dispatch<float>(a, kind, aligned, st);
}
