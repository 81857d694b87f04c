#pragma once
// Vocabulary rows read in warp tiles, for the scoring and distillation kernels.
//
// A row of V logits is cut into tiles of kTileVecs 16-byte vectors per lane (a warp reads a tile
// of 4 KB: 2048 bf16 or 1024 float32 logits, lane l holding vectors l, l + 32, ...). A tile's
// softmax partial is taken against the tile's own maximum,
//     m = max z log2(e)/tau,   s = sum 2^t,   q = sum 2^t t,   t = z log2(e)/tau - m,
// and the row's from its tiles' in tile order. Element -> lane -> tile depends on V alone, so a
// row's sums are the same bits however many CTAs, and whichever of them, read its tiles and
// however the row is aligned in memory.
#include <type_traits>

#include "grpo_common.cuh"

namespace grpo {

constexpr int kTileVecs = 8;

template <typename T>
__host__ __device__ constexpr int tile_elems() { return 32 * kTileVecs * (16 / (int)sizeof(T)); }

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

// -inf in every element of a 32-bit word of T.
template <typename T>
__host__ __device__ constexpr uint32_t neg_inf_word() { return sizeof(T) == 2 ? 0xFF80FF80u : 0xFF800000u; }

template <typename T>
__device__ __forceinline__ float elem_f32(const T* p) {
  if constexpr (sizeof(T) == 2)
    return __bfloat162float(*p);
  else
    return *p;
}

// Vector j (E elements from E j) of a row of V elements, -inf past its end. ALIGNED: the row
// starts on a 16-byte boundary; else its elements are read one by one.
template <typename T, bool ALIGNED>
__device__ __forceinline__ uint4 load_vec(const T* row, int64_t j, int64_t V) {
  constexpr int E = 16 / (int)sizeof(T);
  const int64_t e0 = j * E;
  if (ALIGNED && e0 + E <= V) return __ldg(reinterpret_cast<const uint4*>(row) + j);
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = neg_inf_word<T>();
  if (e0 < V) {
    if constexpr (sizeof(T) == 2) {
      const uint16_t* p = reinterpret_cast<const uint16_t*>(row) + e0;
#pragma unroll
      for (int i = 0; i < E; ++i)
        if (e0 + i < V) w[i / 2] = i & 1 ? (w[i / 2] & 0x0000FFFFu) | ((uint32_t)p[i] << 16) : (w[i / 2] & 0xFFFF0000u) | p[i];
    } else {
      const uint32_t* p = reinterpret_cast<const uint32_t*>(row) + e0;
#pragma unroll
      for (int i = 0; i < E; ++i)
        if (e0 + i < V) w[i] = p[i];
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// This lane's vectors of a tile.
template <typename T, bool ALIGNED>
__device__ __forceinline__ void load_tile(const T* row, int64_t tile, int64_t V, int lane, uint4 (&x)[kTileVecs]) {
  const int64_t j0 = tile * (32 * kTileVecs) + lane;
#pragma unroll
  for (int u = 0; u < kTileVecs; ++u) x[u] = load_vec<T, ALIGNED>(row, j0 + 32 * u, V);
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

// A softmax partial: (m, s, q) as above. s = 0 where nothing has mass (m is then -inf).
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

// The warp's partials joined by a fixed tree (every lane gets the result).
__device__ __forceinline__ Part warp_part(Part v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const Part w{__shfl_xor_sync(0xffffffffu, v.m, o), __shfl_xor_sync(0xffffffffu, v.s, o),
                 __shfl_xor_sync(0xffffffffu, v.q, o)};
    v = part_join(v, w);
  }
  return v;
}

// A tile's partial from its vectors and the lanes' maxima, c = log2(e)/tau. The sums run in
// packed pairs over the lane's vectors, then by a fixed tree over the lanes; every lane gets
// them. A NaN or +inf in the tile makes s NaN. Logits that c z takes below the float32 range
// (the type's lowest value as a mask) have no mass, like -inf.
template <typename T, bool Q>
__device__ __forceinline__ Part tile_part(const uint4 (&x)[kTileVecs], float lane_max, float c) {
  constexpr int E = 16 / (int)sizeof(T);
  const float m = warp_max_nan(lane_max) * c;
  if (m == -INFINITY) return {m, 0.f, 0.f};
  const float2 c2 = make_float2(c, c), m2 = make_float2(-m, -m);
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
    if (qq != qq) {  // 0 * -inf of an element without mass (or a NaN row): once more without them
      qq = 0.f;
#pragma unroll
      for (int u = 0; u < kTileVecs; ++u) {
        float f[E];
        vec_floats<T>(x[u], f);
#pragma unroll
        for (int i = 0; i < E; ++i) {
          const float t = fmaf(f[i], c, -m), e = ex2(t);
          if (e != 0.f) qq = fmaf(e, t, qq);
        }
      }
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
