#pragma once
// Vocabulary rows read in warp tiles, for the scoring and distillation kernels.
//
// A row of V logits is cut into tiles of 4 KB (2048 bf16 or 1024 float32 logits), one warp's work: 8
// vectors of 16 bytes a lane. A tile's softmax partial is taken against its own maximum,
//     m = max z log2(e)/tau,   s = sum 2^t,   q = sum 2^t t,   t = z log2(e)/tau - m
//     (another scale where |m| is past 2^31: shift_of),
// and the row's from its tiles'. Element -> lane -> tile depends on V alone, so a row's sums are the
// same bits however many CTAs, and whichever of them, read its tiles and however the row is aligned
// in memory.
//
// Tiles go through shared memory (bulk copies, one mbarrier per slot): the loads in flight cost no
// registers, and a row that does not start on a 16-byte boundary is fetched by the aligned vectors it
// touches and shifted into place when it is read from its slot.
#include "grpo_common.cuh"

namespace grpo {

constexpr int kTileVecs = 8;                       // vectors per lane
constexpr int kTileBytes = 32 * kTileVecs * 16;    // 4 KB
constexpr int kSlotBytes = kTileBytes + 128;       // and the vector an unaligned tile reaches into

template <typename T>
__host__ __device__ constexpr int tile_elems() { return kTileBytes / (int)sizeof(T); }

__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

__device__ __forceinline__ uint32_t max_nan_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// Warp maximum; NaN if any lane's value is.
__device__ __forceinline__ float warp_max_nan(float x) {
  float r;
  asm("redux.sync.max.NaN.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
  return r;
}

template <typename T>
__device__ __forceinline__ float elem_f32(const T* p) {
  if constexpr (sizeof(T) == 2)
    return __bfloat162float(*p);
  else
    return *p;
}

// 16 bytes of a row from element e0 (which may lie before it), -inf outside [0, V); read element by
// element.
template <typename T>
__device__ __forceinline__ uint4 edge_vec(const T* row, int64_t e0, int64_t V) {
  constexpr int E = 16 / (int)sizeof(T);
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = sizeof(T) == 2 ? 0xFF80FF80u : 0xFF800000u;
#pragma unroll
  for (int i = 0; i < E; ++i)
    if (e0 + i >= 0 && e0 + i < V) {
      if constexpr (sizeof(T) == 2) {
        const uint32_t h = reinterpret_cast<const uint16_t*>(row)[e0 + i];
        w[i / 2] = i & 1 ? (w[i / 2] & 0x0000FFFFu) | (h << 16) : (w[i / 2] & 0xFFFF0000u) | h;
      } else {
        w[i] = reinterpret_cast<const uint32_t*>(row)[e0 + i];
      }
    }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Bytes by which a row's start (and with it every tile's) lies past a 16-byte boundary.
__device__ __forceinline__ int row_off(const void* row) { return (int)(reinterpret_cast<uintptr_t>(row) & 15u); }

// The part of fetch_tile at a row's ends: the slot's vectors [v0, v1) are wholly inside the row, the
// others up to `all` are filled in here. (Out of line: few tiles come here, and the streaming loops
// are short of instruction cache.)
template <typename T>
__device__ __noinline__ int2 fetch_edges(uint8_t* slot, const T* row, int off, int tile, int64_t V, int lane, int all) {
  constexpr int E = 16 / (int)sizeof(T);
  int v0 = 0, v1 = all;
  const int64_t to_end = V * (int64_t)sizeof(T) - (int64_t)tile * kTileBytes + off;  // from the slot's start
  if (to_end < (int64_t)v1 * 16) v1 = (int)(to_end / 16);
  if (tile == 0 && off) v0 = 1;
  const int64_t e0 = ((int64_t)tile * kTileBytes - off) / (int64_t)sizeof(T);
  // at most one vector at either end holds elements of the row and others: read element by element
  if (v0 && lane == 0) reinterpret_cast<uint4*>(slot)[0] = edge_vec(row, e0, V);
  const int cut = v1 > v0 ? v1 : v0;
  if (lane == 0 && cut < all) reinterpret_cast<uint4*>(slot)[cut] = edge_vec(row, e0 + (int64_t)cut * E, V);
  const uint32_t ninf = sizeof(T) == 2 ? 0xFF80FF80u : 0xFF800000u;
  for (int v = cut + 1 + lane; v < all; v += 32) reinterpret_cast<uint4*>(slot)[v] = make_uint4(ninf, ninf, ninf, ninf);
  fence_proxy_async_smem();  // before the copy that refills the slot
  __syncwarp();              // before lane 0's arrive on the slot's barrier
  return make_int2(v0, v1);
}

// Starts the fetch of a tile into a slot; every lane of the warp calls it. The slot receives the
// aligned vectors that hold the tile, so the tile starts `off` bytes into it. Those wholly inside the
// row come by one bulk copy, which completes on `bar`; what the row's ends cut is filled in by the
// lanes (no byte outside the row is read), -inf where there is no element, before lane 0 arrives on
// `bar`. (A lane that waits on `bar` sees both.)
template <typename T>
__device__ __forceinline__ void fetch_tile(uint8_t* slot, const T* row, int off, int tile, int n_tiles, int64_t V,
                                           int lane, uint64_t* bar) {
  int2 v = make_int2(0, kTileVecs * 32 + (off ? 1 : 0));
  // (the last vector of the last tile but one may be cut, too)
  if ((tile == 0 && off) || tile + 1 >= n_tiles - 1) v = fetch_edges(slot, row, off, tile, V, lane, v.y);
  if (lane == 0) {
    const uint32_t bytes = v.y > v.x ? (uint32_t)(v.y - v.x) * 16u : 0u;
    mbar_arrive_expect_tx(bar, bytes);
    if (bytes)
      bulk_g2s(slot + v.x * 16, reinterpret_cast<const uint8_t*>(row) + (int64_t)tile * kTileBytes - off + v.x * 16, bytes,
               bar);
  }
}

// Vector of a tile held by (lane, u): a lane's 8 vectors are two runs of 64 bytes. u rotates within a
// run so that the 8 lanes of a shared-memory phase touch different banks.
__device__ __forceinline__ int tile_vec(int lane, int u) {
  return (u >> 2) * 128 + lane * 4 + ((u + (lane >> 1)) & 3);
}

// 16 bytes from `off` bytes (uniform over the warp) into the pair of vectors a, b.
template <typename T>
__device__ __forceinline__ uint4 shift_vec(const uint4& a, const uint4& b, int off) {
  uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  if (off & 8) {
#pragma unroll
    for (int i = 0; i < 6; ++i) w[i] = w[i + 2];
  }
  if (off & 4) {
#pragma unroll
    for (int i = 0; i < 5; ++i) w[i] = w[i + 1];
  }
  if (sizeof(T) == 2 && (off & 2)) {
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], 16);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
  return v;
}

// Byte offsets of this lane's vectors 0..3 in a tile (4..7 follow 2048 bytes on).
struct LaneOffsets {
  uint32_t o[4];
  __device__ explicit LaneOffsets(int lane) {
#pragma unroll
    for (int u = 0; u < 4; ++u) o[u] = (uint32_t)tile_vec(lane, u) * 16u;
  }
};

// This lane's vectors of the tile in the slot at a shared-memory address.
template <typename T, bool ALIGNED>
__device__ __forceinline__ void read_tile(uint32_t slot, int off, const LaneOffsets& lo, uint4 (&x)[kTileVecs]) {
#pragma unroll
  for (int u = 0; u < kTileVecs; ++u) {
    const uint32_t at = slot + lo.o[u & 3] + (u >> 2) * 2048u;
    x[u] = lds128(at);
    if (!ALIGNED && off != 0) x[u] = shift_vec<T>(x[u], lds128(at + 16), off);
  }
}

// Vector j of a row straight from global memory, -inf past its end. ALIGNED: the row starts on a
// 16-byte boundary. Of other rows the two aligned vectors that hold it, where both are inside the row.
template <typename T, bool ALIGNED>
__device__ __forceinline__ uint4 load_vec(const T* row, int64_t j, int64_t V) {
  constexpr int E = 16 / (int)sizeof(T);
  if (ALIGNED) {
    if ((j + 1) * E <= V) return __ldg(reinterpret_cast<const uint4*>(row) + j);
  } else if (j > 0 && (j + 2) * E <= V) {
    const int off = row_off(row);
    const uint4* p = reinterpret_cast<const uint4*>(reinterpret_cast<const uint8_t*>(row) - off) + j;
    return off ? shift_vec<T>(__ldg(p), __ldg(p + 1), off) : __ldg(p);
  }
  return edge_vec(row, j * E, V);
}

// Aligned vector j of those that hold a row (vector 0 holds its first element), -inf outside the row.
template <typename T, bool ALIGNED>
__device__ __forceinline__ uint4 load_cover(const T* row, int64_t j, int off, int64_t V) {
  const int64_t b = j * 16 - (ALIGNED ? 0 : off);
  if (b >= 0 && b + 16 <= V * (int64_t)sizeof(T))
    return __ldg(reinterpret_cast<const uint4*>(reinterpret_cast<const uint8_t*>(row) + b));
  return edge_vec(row, b / (int64_t)sizeof(T), V);
}

// Element i of a vector (a run-time index).
template <typename T>
__device__ __forceinline__ float vec_elem(const uint4& v, int i) {
  const int k = sizeof(T) == 2 ? i >> 1 : i;
  const uint32_t w = k & 2 ? (k & 1 ? v.w : v.z) : (k & 1 ? v.y : v.x);
  if constexpr (sizeof(T) == 2) return i & 1 ? bf16_hi(w) : bf16_lo(w);
  return __uint_as_float(w);
}

// Maximum of a vector's elements; NaN if one is.
template <typename T>
__device__ __forceinline__ float vec_max(const uint4& v) {
  if constexpr (sizeof(T) == 2) {
    const uint32_t a = max_nan_bf16x2(max_nan_bf16x2(v.x, v.y), max_nan_bf16x2(v.z, v.w));
    return max_nan(bf16_lo(a), bf16_hi(a));
  } else {
    return max_nan(max_nan(__uint_as_float(v.x), __uint_as_float(v.y)),
                   max_nan(__uint_as_float(v.z), __uint_as_float(v.w)));
  }
}

template <typename T>
__device__ __forceinline__ float tile_lane_max(const uint4 (&x)[kTileVecs]) {
  if constexpr (sizeof(T) == 2) {
    uint32_t a = max_nan_bf16x2(x[0].x, x[0].y), b = max_nan_bf16x2(x[0].z, x[0].w);
#pragma unroll
    for (int u = 1; u < kTileVecs; ++u) {
      a = max_nan_bf16x2(a, max_nan_bf16x2(x[u].x, x[u].y));
      b = max_nan_bf16x2(b, max_nan_bf16x2(x[u].z, x[u].w));
    }
    a = max_nan_bf16x2(a, b);
    return max_nan(bf16_lo(a), bf16_hi(a));
  } else {
    float m = vec_max<T>(x[0]);
#pragma unroll
    for (int u = 1; u < kTileVecs; ++u) m = max_nan(m, vec_max<T>(x[u]));
    return m;
  }
}

template <typename T>
__device__ __forceinline__ void vec_floats(const uint4& v, float (&f)[16 / sizeof(T)]) {
  if constexpr (sizeof(T) == 2) {
    f[0] = bf16_lo(v.x); f[1] = bf16_hi(v.x); f[2] = bf16_lo(v.y); f[3] = bf16_hi(v.y);
    f[4] = bf16_lo(v.z); f[5] = bf16_hi(v.z); f[6] = bf16_lo(v.w); f[7] = bf16_hi(v.w);
  } else {
    f[0] = __uint_as_float(v.x); f[1] = __uint_as_float(v.y);
    f[2] = __uint_as_float(v.z); f[3] = __uint_as_float(v.w);
  }
}

// The shift of a tile (or row) whose largest logit is z, and the scale that goes with it. z c rounded is
// off by half its last place, which fma(z, c, -m) leaves in the exponent. That costs only range below
// |z c| = 2^31: every t of the tile has the same term, of 64 at most. Above it 2^t would overflow or vanish
// for z itself (tiles of nothing but a mask of -1e30 made their row NaN). There the scale is the power of two
// above c, under which nothing is rounded and shifts keep the order of their logits; all other float32
// logits are 2^7 or more below z under either scale, so that their 2^t are 0 alike.
constexpr float kFarShift = 2147483648.f;

__device__ __forceinline__ float far_scale(float c) {
  return __uint_as_float((__float_as_uint(c) + 0x00800000u) & 0x7F800000u);
}
__device__ __forceinline__ bool is_far(float m) { return fabsf(m) >= kFarShift; }
__device__ __forceinline__ float scale_at(float m, float c) { return is_far(m) ? far_scale(c) : c; }
__device__ __forceinline__ float shift_of(float z, float c) {
  const float m = z * c;
  return is_far(m) ? z * far_scale(c) : m;
}
// From t or a difference of shifts under scale_at(m, c) to log2 units: 1, or c over its far scale (c's
// mantissa in [1/2, 1)).
__device__ __forceinline__ float unit_at(float m, float c) {
  return is_far(m) ? __uint_as_float((__float_as_uint(c) & 0x007FFFFFu) | 0x3F000000u) : 1.f;
}

// A softmax partial: (m, s, q) as above. m = -inf where nothing has mass.
struct Part {
  float m, s, q;
};

// Partials joined; the shift of q is moved with that of s: sum e (t + m - M) = q + (m - M) s.
__device__ __forceinline__ Part part_join(Part a, Part b) {
  const float M = fmaxf(a.m, b.m);
  if (M == -INFINITY) return {M, a.s + b.s, 0.f};
  const float da = a.m - M, db = b.m - M;
  const float fa = ex2(da), fb = ex2(db);
  const float qa = fa != 0.f ? fa * fmaf(da, a.s, a.q) : 0.f, qb = fb != 0.f ? fb * fmaf(db, b.s, b.q) : 0.f;
  return {M, fmaf(fa, a.s, fb * b.s), qa + qb};
}

// The warp's partials joined (every lane gets the result): all rescaled to the largest shift, the sums
// by a fixed tree.
template <bool Q>
__device__ __forceinline__ Part warp_part(Part v) {
  const float M = warp_max_nan(v.m);
  if (M == -INFINITY) return {M, 0.f, 0.f};
  const float d = v.m - M, f = ex2(d);
  float q = Q && f != 0.f ? f * fmaf(d, v.s, v.q) : 0.f, s = f * v.s;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    s += __shfl_xor_sync(0xffffffffu, s, o);
    if (Q) q += __shfl_xor_sync(0xffffffffu, q, o);
  }
  return {M, s, q};
}

// A tile's vectors by value.
struct Tile {
  uint4 x[kTileVecs];
};

// A lane's q where elements without mass made it 0 * -inf: their t is taken as the lowest finite value.
// (Out of line: the streaming loops are short of instruction cache.)
template <typename T>
__device__ __noinline__ float masked_q(Tile tile, float shift, float c) {
  constexpr int E = 16 / (int)sizeof(T);
  float2 q[2] = {{0.f, 0.f}, {0.f, 0.f}};
#pragma unroll
  for (int u = 0; u < kTileVecs; ++u) {
    float f[E];
    vec_floats<T>(tile.x[u], f);
#pragma unroll
    for (int i = 0; i < E; i += 2) {
      float2 t = __ffma2_rn(make_float2(f[i], f[i + 1]), make_float2(c, c), make_float2(-shift, -shift));
      const float2 e = make_float2(ex2(t.x), ex2(t.y));
      t = make_float2(fmaxf(t.x, -3.4028235e38f), fmaxf(t.y, -3.4028235e38f));
      q[(i / 2) & 1] = __ffma2_rn(e, t, q[(i / 2) & 1]);
    }
  }
  return (q[0].x + q[1].x) + (q[0].y + q[1].y);
}

// A tile's partial from its vectors, z_max its largest logit, c = log2(e)/tau. The sums run in packed
// pairs over the lane's vectors, then by a fixed tree over the lanes; every lane gets them. A NaN or +inf
// in the tile makes s NaN or inf. Logits that the scale takes below the float32 range (the type's lowest
// value as a mask) have no mass, like -inf.
template <typename T, bool Q>
__device__ __forceinline__ Part tile_part(const uint4 (&x)[kTileVecs], float z_max, float tau_c) {
  constexpr int E = 16 / (int)sizeof(T);
  float m = z_max * tau_c, c = tau_c, shift = m;
  if (is_far(m)) {  // (or -inf)
    c = far_scale(tau_c);
    m = z_max * c;
    shift = m == -INFINITY ? 0.f : m;
  }
  const float2 c2 = make_float2(c, c), m2 = make_float2(-shift, -shift);
  float2 s[2] = {{0.f, 0.f}, {0.f, 0.f}}, q[2] = {{0.f, 0.f}, {0.f, 0.f}};
#pragma unroll
  for (int u = 0; u < kTileVecs; ++u) {
    float f[E];
    vec_floats<T>(x[u], f);
#pragma unroll
    for (int i = 0; i < E; i += 2) {
      const float2 t = __ffma2_rn(make_float2(f[i], f[i + 1]), c2, m2);
      const float2 e = make_float2(ex2(t.x), ex2(t.y));
      const int k = (i / 2) & 1;
      s[k] = __fadd2_rn(s[k], e);
      if (Q) q[k] = __ffma2_rn(e, t, q[k]);
    }
  }
  float ss = (s[0].x + s[1].x) + (s[0].y + s[1].y), qq = 0.f;
  if (Q) {
    qq = (q[0].x + q[1].x) + (q[0].y + q[1].y);
    if (qq != qq) {  // (or a NaN row)
      Tile tile;
#pragma unroll
      for (int u = 0; u < kTileVecs; ++u) tile.x[u] = x[u];
      qq = masked_q<T>(tile, shift, c);
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    ss += __shfl_xor_sync(0xffffffffu, ss, o);
    if (Q) qq += __shfl_xor_sync(0xffffffffu, qq, o);
  }
  return {m, ss, qq};
}

}  // namespace grpo
