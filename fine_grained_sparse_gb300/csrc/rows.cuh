// What the kernels over rows and tensors share: pieces of a row in registers,
// pairs of fp32 values, sums over a block, and the 8-bit form of 128 values
// (E4M3 codes with one fp32 scale).
#pragma once

#include "common.cuh"

namespace fgs {

constexpr int kRowGroup = 128;  // columns of a row with one scale

// N values of a row as fp32, 16 bytes or one value at a time: load and store take
// no other N.
template <typename T, int N>
struct Piece {
  static_assert(N == 1 || N * sizeof(T) == 16, "one value or 16 bytes");
  float v[N];
};

template <int N>
__device__ __forceinline__ Piece<__nv_bfloat16, N> load(const __nv_bfloat16* p) {
  Piece<__nv_bfloat16, N> o;
  if constexpr (N == 1) {
    o.v[0] = __bfloat162float(*p);
  } else {
    const uint4 u = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      o.v[2 * i] = __uint_as_float(w[i] << 16);
      o.v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  return o;
}
template <int N>
__device__ __forceinline__ Piece<float, N> load(const float* p) {
  Piece<float, N> o;
  if constexpr (N == 1) {
    o.v[0] = *p;
  } else {
    const float4 u = *reinterpret_cast<const float4*>(p);
    o.v[0] = u.x, o.v[1] = u.y, o.v[2] = u.z, o.v[3] = u.w;
  }
  return o;
}
template <int N>
__device__ __forceinline__ void store(__nv_bfloat16* p, const float (&v)[N]) {
  static_assert(N == 1 || N == 8, "one value or 16 bytes");
  if constexpr (N == 1)
    *p = __float2bfloat16_rn(v[0]);
  else
    *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                              pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
}
template <int N>
__device__ __forceinline__ void store(float* p, const float (&v)[N]) {
  static_assert(N == 1 || N == 4, "one value or 16 bytes");
  if constexpr (N == 1)
    *p = v[0];
  else
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
}

// max that keeps NaN, as the definition's maximum over a group does
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// Two E4M3 codes, a's in the low byte.
__device__ __forceinline__ uint32_t e4m3x2(float a, float b) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
  return r;
}

// v[i] / s correctly rounded, for s and the largest |v[i]| well inside fp32's
// range, by Markstein's theorem (IBM J. Res. Dev. 34, 1990): from y, 1 / s
// correctly rounded, and q within an ulp of v / s, q + y (v - q s) is v / s
// correctly rounded.  v y may be off by 1.5 ulp, so it takes two such steps.
// Two values to an instruction: 8192 rows of 7168 bf16 with all outputs and a
// flushed L2 in 96.5 us, with a division for each value 102.4.
template <int N>
__device__ __forceinline__ void divide(float (&v)[N], float s) {
  const float y = 1.0f / s;
#pragma unroll
  for (int k = 0; k + 1 < N; k += 2)
    asm("{\n\t.reg .b64 v, q, r, y, s;\n\t"
        "mov.b64 v, {%0, %1};\n\tmov.b64 y, {%2, %2};\n\tmov.b64 s, {%3, %3};\n\t"
        "mul.rn.f32x2 q, v, y;\n\t"
        "fma.rn.f32x2 r, q, s, v;\n\tfma.rn.f32x2 q, r, y, q;\n\t"
        "fma.rn.f32x2 r, q, s, v;\n\tfma.rn.f32x2 q, r, y, q;\n\t"
        "mov.b64 {%0, %1}, q;\n\t}"
        : "+f"(v[k]), "+f"(v[k + 1])
        : "f"(y), "f"(-s));
}

template <int N>
__device__ __forceinline__ void store_codes(uint8_t* p, const float (&q)[N]) {
  if constexpr (N == 8)
    *reinterpret_cast<uint2*>(p) = make_uint2(e4m3x2(q[0], q[1]) | e4m3x2(q[2], q[3]) << 16,
                                              e4m3x2(q[4], q[5]) | e4m3x2(q[6], q[7]) << 16);
  else if constexpr (N == 4)
    *reinterpret_cast<uint32_t*>(p) = e4m3x2(q[0], q[1]) | e4m3x2(q[2], q[3]) << 16;
}

// Pairs of fp32 values, one instruction for both.
typedef unsigned long long pair;
__device__ __forceinline__ pair make_pair2(float a, float b) {
  pair r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void split(pair v, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ pair mul2(pair a, pair b) {
  pair r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ pair fma2(pair a, pair b, pair c) {
  pair r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// Sums of two values over a warp, and over a block's threads; the same in all of
// them.  The halves of a warp first exchange what the other adds up, so that a
// round of the tree serves both values.  A `part`, 64 values, serves one sum at a
// time: with a barrier between two uses of it.
__device__ __forceinline__ float half_sums(float x, float y) {
  const bool low = (threadIdx.x & 31) < 16;
  float v = low ? x : y;
  v += __shfl_xor_sync(0xffffffffu, low ? y : x, 16);
#pragma unroll
  for (int o = 8; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;  // x's in the low half, y's in the high
}
__device__ __forceinline__ float2 both_halves(float v) {
  const float other = __shfl_xor_sync(0xffffffffu, v, 16);
  return (threadIdx.x & 31) < 16 ? make_float2(v, other) : make_float2(other, v);
}
__device__ __forceinline__ float2 warp_sum(float x, float y) { return both_halves(half_sums(x, y)); }
__device__ __forceinline__ float2 block_sum(float x, float y, float* part) {
  const int lane = threadIdx.x & 31;
  float v = half_sums(x, y);
  // the sums of warp i at 2 i and 2 i + 1
  if ((lane & 15) == 0) part[threadIdx.x >> 4] = v;
  __syncthreads();
  const int sums = blockDim.x / 16, i = 2 * (lane & 15) + (lane >> 4);
  v = i < sums ? part[i] : 0.0f;
  if (i + 32 < sums) v += part[i + 32];
#pragma unroll
  for (int o = 8; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return both_halves(v);
}

// N values: one, or N / 2 pairs.
template <int N>
struct Vec {
  static constexpr int M = N / 2;
  pair v[M];
};
template <>
struct Vec<1> {
  float v;
};
template <int N>
__device__ __forceinline__ Vec<N> mul(const Vec<N>& a, const Vec<N>& b) {
  Vec<N> r;
  if constexpr (N == 1)
    r.v = a.v * b.v;
  else
#pragma unroll
    for (int i = 0; i < Vec<N>::M; ++i) r.v[i] = mul2(a.v[i], b.v[i]);
  return r;
}
template <int N>
__device__ __forceinline__ Vec<N> fma(const Vec<N>& a, const Vec<N>& b, const Vec<N>& c) {
  Vec<N> r;
  if constexpr (N == 1)
    r.v = fmaf(a.v, b.v, c.v);
  else
#pragma unroll
    for (int i = 0; i < Vec<N>::M; ++i) r.v[i] = fma2(a.v[i], b.v[i], c.v[i]);
  return r;
}
template <int N>
__device__ __forceinline__ Vec<N> add(const Vec<N>& a, const Vec<N>& b) {
  Vec<N> r;
  if constexpr (N == 1)
    r.v = a.v + b.v;
  else
#pragma unroll
    for (int i = 0; i < Vec<N>::M; ++i)
      asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v[i]) : "l"(a.v[i]), "l"(b.v[i]));
  return r;
}
template <int N>
__device__ __forceinline__ Vec<N> all(float a) {
  Vec<N> r;
  if constexpr (N == 1)
    r.v = a;
  else
#pragma unroll
    for (int i = 0; i < Vec<N>::M; ++i) r.v[i] = make_pair2(a, a);
  return r;
}
template <int N>
__device__ __forceinline__ float total(const Vec<N>& a) {
  if constexpr (N == 1) {
    return a.v;
  } else {
    pair s = a.v[0];
#pragma unroll
    for (int i = 1; i < Vec<N>::M; ++i)
      asm("add.rn.f32x2 %0, %1, %2;" : "=l"(s) : "l"(s), "l"(a.v[i]));
    float x, y;
    split(s, x, y);
    return x + y;
  }
}

// N values of type T in memory, of 2 to 16 bytes, and as a Vec.
template <typename T, int N>
struct Chunk;
template <>
struct Chunk<__nv_bfloat16, 8> { uint4 u; };
template <>
struct Chunk<__nv_bfloat16, 2> { uint32_t u; };
template <>
struct Chunk<__nv_bfloat16, 1> { __nv_bfloat16 u; };
template <>
struct Chunk<float, 4> { float4 u; };
template <>
struct Chunk<float, 1> { float u; };
__device__ __forceinline__ pair bf16_pair(uint32_t w) {
  return make_pair2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
__device__ __forceinline__ uint32_t pair_bf16(pair v) {
  float a, b;
  split(v, a, b);
  return pack_bf16x2(a, b);
}
__device__ __forceinline__ Vec<8> unpack(const Chunk<__nv_bfloat16, 8>& c) {
  return {{bf16_pair(c.u.x), bf16_pair(c.u.y), bf16_pair(c.u.z), bf16_pair(c.u.w)}};
}
__device__ __forceinline__ Vec<2> unpack(const Chunk<__nv_bfloat16, 2>& c) {
  return {{bf16_pair(c.u)}};
}
__device__ __forceinline__ Vec<1> unpack(const Chunk<__nv_bfloat16, 1>& c) {
  return {__bfloat162float(c.u)};
}
__device__ __forceinline__ Vec<4> unpack(const Chunk<float, 4>& c) {
  return {{make_pair2(c.u.x, c.u.y), make_pair2(c.u.z, c.u.w)}};
}
__device__ __forceinline__ Vec<1> unpack(const Chunk<float, 1>& c) { return {c.u}; }
__device__ __forceinline__ void pack(const Vec<8>& v, Chunk<__nv_bfloat16, 8>& c) {
  c.u = make_uint4(pair_bf16(v.v[0]), pair_bf16(v.v[1]), pair_bf16(v.v[2]), pair_bf16(v.v[3]));
}
__device__ __forceinline__ void pack(const Vec<2>& v, Chunk<__nv_bfloat16, 2>& c) {
  c.u = pair_bf16(v.v[0]);
}
__device__ __forceinline__ void pack(const Vec<1>& v, Chunk<__nv_bfloat16, 1>& c) {
  c.u = __float2bfloat16_rn(v.v);
}
__device__ __forceinline__ void pack(const Vec<4>& v, Chunk<float, 4>& c) {
  split(v.v[0], c.u.x, c.u.y);
  split(v.v[1], c.u.z, c.u.w);
}
__device__ __forceinline__ void pack(const Vec<1>& v, Chunk<float, 1>& c) { c.u = v.v; }

// A chunk of global memory into shared memory, past the registers and L1.
template <int kBytes>
__device__ __forceinline__ void copy_async(uint32_t dst, const void* src) {
  if constexpr (kBytes == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(kBytes)
                 : "memory");
}
__device__ __forceinline__ void commit_copies() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}

// Rows that begin inside a chunk.  Chunks that a row of d values reaches into at
// most:
template <int N>
__host__ __device__ constexpr int span_chunks(int d) {
  return (d + 2 * N - 2) / N;
}
// w[at] .. w[at + N - 1], 0 outside [0, d).
template <typename T, int N>
__device__ __forceinline__ Chunk<T, N> gather(const T* w, int at, int d) {
  Vec<N> v;
  float x[N];
#pragma unroll
  for (int k = 0; k < N; ++k)
    x[k] = at + k >= 0 && at + k < d ? static_cast<float>(w[at + k]) : 0.0f;
#pragma unroll
  for (int k = 0; k < N; k += 2) v.v[k / 2] = make_pair2(x[k], x[k + 1]);
  Chunk<T, N> c;
  pack(v, c);
  return c;
}
// `to` in place of the values outside [lo, hi), whatever they are.
template <int N>
__device__ __forceinline__ void clip(Vec<N>& v, int lo, int hi, float to) {
#pragma unroll
  for (int k = 0; k < N; k += 2) {
    float a, b;
    split(v.v[k / 2], a, b);
    v.v[k / 2] = make_pair2(k >= lo && k < hi ? a : to, k + 1 >= lo && k + 1 < hi ? b : to);
  }
}
template <typename T, int N>
__device__ __forceinline__ void clip(Chunk<T, N>& c, int lo, int hi) {
  Vec<N> v = unpack(c);
  clip(v, lo, hi, 0.0f);
  pack(v, c);
}
template <typename T, int N>
__device__ __forceinline__ void store_part(T* to, const Vec<N>& v, int lo, int hi) {
#pragma unroll
  for (int k = 0; k < N; k += 2) {
    float a, b;
    split(v.v[k / 2], a, b);
    const float x[1] = {a}, y[1] = {b};
    if (k >= lo && k < hi) store<1>(to + k, x);
    if (k + 1 >= lo && k + 1 < hi) store<1>(to + k + 1, y);
  }
}

}  // namespace fgs
