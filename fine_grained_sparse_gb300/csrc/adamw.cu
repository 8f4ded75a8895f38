// One AdamW step over many tensors in one launch (moe_adamw).  Per element, in
// fp32 with every operation rounded by itself (no contraction, so that a plain
// program of the same operations gives the same bits):
//   g = grad c,  m = b1 m + (1 - b1) g,  v = b2 v + (1 - b2) g g,  r = sqrt v
//   p = p (1 - lr wd) - (m / (r / sqrt(1 - b2^t) + eps)) lr / (1 - b1^t)
// States in 8 bits: m and r as E4M3 codes with one fp32 scale per 128
// elements, max / 448.  v moves by a hundredth or a thousandth in a step, which
// rounding to nearest would take back every time, so r goes to one of the two
// codes beside it with the probabilities that keep its mean, by 16 random bits
// an element.  A root above 0 has a code above 0: of two codes 0 the update
// m / (0 + eps) of the next step would be unbounded.
// m falls by (1 - b1) of itself where no gradient comes.  E4M3's normal codes are
// at most 1/8 apart, so with b1 up to 29/32 that is 3/4 of a step or more, and
// rounded to nearest m falls.  Its subnormal codes 1 to 4, and with a larger b1
// normal ones too, would come back for ever, while r falls and the weight moves on
// by m / r in every step.  So there, where nearest gives back the stored code, m
// is rounded at random as r is.
// Bound by HBM; the 8-bit form also by its instructions.
#include "common.cuh"
#include "internal.h"
#include "rows.cuh"

namespace fgs {
namespace {

constexpr int kThreads = 256;
constexpr int kStep = 8 * kThreads;  // elements of a block at a time
constexpr int kSteps = 4;            // of a block in large launches

// Eight values of a tensor as they lie in memory, and as fp32.
template <typename T>
struct Raw8;
template <>
struct Raw8<__nv_bfloat16> {
  uint4 u;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) {
    u = *reinterpret_cast<const uint4*>(p);
  }
  __device__ __forceinline__ void unpack(float (&v)[8]) const {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
};
template <>
struct Raw8<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = reinterpret_cast<const float4*>(p)[0];
    b = reinterpret_cast<const float4*>(p)[1];
  }
  __device__ __forceinline__ void unpack(float (&v)[8]) const {
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
    v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  }
};
// Values [at, at + 8) of a tensor of n, 0 beyond its end.
template <typename T>
__device__ __forceinline__ void load_tail(const T* p, int64_t at, int64_t n, float (&v)[8]) {
  if (at + 8 <= n) {
    Raw8<T> x;
    x.load(p + at);
    x.unpack(v);
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = at + k < n ? load<1>(p + at + k).v[0] : 0.0f;
  }
}
template <bool kFull, typename T>
__device__ __forceinline__ void store8(T* p, int64_t at, int64_t n, const float (&v)[8]) {
  if (kFull || at + 8 <= n) {
    if constexpr (sizeof(T) == 2) {
      store<8>(p + at, v);
    } else {
      const float a[4] = {v[0], v[1], v[2], v[3]}, b[4] = {v[4], v[5], v[6], v[7]};
      store<4>(p + at, a);
      store<4>(p + at + 4, b);
    }
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float one[1] = {v[k]};
      if (at + k < n) store<1>(p + at + k, one);
    }
  }
}

// Eight E4M3 codes, 0 beyond the end.
__device__ __forceinline__ uint2 load_codes_tail(const void* codes, int64_t at, int64_t n) {
  const uint8_t* p = static_cast<const uint8_t*>(codes);
  if (at + 8 <= n) return *reinterpret_cast<const uint2*>(p + at);
  uint2 u = make_uint2(0, 0);
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const uint32_t b = at + k < n ? p[at + k] : 0;
    if (k < 4) u.x |= b << 8 * k; else u.y |= b << 8 * (k - 4);
  }
  return u;
}
template <bool kFull>
__device__ __forceinline__ void store_codes8(void* codes, int64_t at, int64_t n, uint2 u) {
  uint8_t* p = static_cast<uint8_t*>(codes);
  if (kFull || at + 8 <= n) {
    *reinterpret_cast<uint2*>(p + at) = u;
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (at + k < n) p[at + k] = static_cast<uint8_t>((k < 4 ? u.x : u.y) >> 8 * (k & 3));
  }
}
// Their values times a scale, each product rounded.
__device__ __forceinline__ void decode(uint2 u, float scale, float (&v)[8]) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const uint16_t two = static_cast<uint16_t>((k < 2 ? u.x : u.y) >> 16 * (k & 1));
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(two));
    asm("{\n\t.reg .f16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
        : "=f"(v[2 * k]), "=f"(v[2 * k + 1])
        : "r"(h));
    v[2 * k] = __fmul_rn(v[2 * k], scale);
    v[2 * k + 1] = __fmul_rn(v[2 * k + 1], scale);
  }
}

// a + b with a rounding of its own: as a 1 + b with a 1 that the compiler does
// not know, as it makes one operation of a product and add.rn.f32x2.
__device__ __forceinline__ pair add2(pair a, float one, pair b) {
  return fma2(a, make_pair2(one, one), b);
}

// Square roots of values in [2^-90, 2^90], correctly rounded: from y, 1 / sqrt v
// to 2^-22, and g = v y, a Newton step of g and the correction (v - g g) y / 2
// (Markstein, IBM J. Res. Dev. 34, 1990); all 2^24 mantissas of both parities
// of the exponent are compared with the exact roots in the tests.
__device__ __forceinline__ pair sqrt2(pair v) {
  float a, b, ya, yb;
  split(v, a, b);
  asm("rsqrt.approx.f32 %0, %1;" : "=f"(ya) : "f"(a));
  asm("rsqrt.approx.f32 %0, %1;" : "=f"(yb) : "f"(b));
  const pair y = make_pair2(ya, yb);
  pair g = mul2(v, y);
  const pair h = mul2(y, make_pair2(0.5f, 0.5f));
  g = fma2(fma2(mul2(h, make_pair2(-1.0f, -1.0f)), g, make_pair2(0.5f, 0.5f)), g, g);
  return fma2(fma2(mul2(g, make_pair2(-1.0f, -1.0f)), g, v), h, g);
}

// 1 / s within half an ulp and 2^-22 of one: the approximation and a Newton step.
__device__ __forceinline__ float reciprocal(float s) {
  float y;
  asm("rcp.approx.f32 %0, %1;" : "=f"(y) : "f"(s));
  return fmaf(fmaf(-s, y, 1.0f), y, y);
}
// a / d from y = reciprocal(d), nd = -d: two residual steps, as in divide().
__device__ __forceinline__ pair quotient2(pair a, pair nd, pair y) {
  pair q = mul2(a, y);
  q = fma2(fma2(nd, q, a), y, q);
  return fma2(fma2(nd, q, a), y, q);
}
__device__ __forceinline__ pair divide2(pair a, pair d) {
  float x, y, rx, ry;
  split(d, x, y);
  asm("rcp.approx.f32 %0, %1;" : "=f"(rx) : "f"(x));
  asm("rcp.approx.f32 %0, %1;" : "=f"(ry) : "f"(y));
  const pair nd = mul2(d, make_pair2(-1.0f, -1.0f));
  const pair r = make_pair2(rx, ry);
  return quotient2(a, nd, fma2(fma2(nd, r, make_pair2(1.0f, 1.0f)), r, r));
}

// The largest of three, NaN if one is.
__device__ __forceinline__ float max3_nan(float a, float b, float c) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ float max8_nan(const float (&v)[8]) {
  return max3_nan(max3_nan(fabsf(v[0]), fabsf(v[1]), fabsf(v[2])),
                  max3_nan(fabsf(v[3]), fabsf(v[4]), fabsf(v[5])), max_nan(fabsf(v[6]), fabsf(v[7])));
}
__device__ __forceinline__ float min3(float a, float b, float c) {
  float r;
  asm("min.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ float min8(const float (&v)[8]) {  // of |v|, past NaN
  return min3(min3(fabsf(v[0]), fabsf(v[1]), fabsf(v[2])),
              min3(fabsf(v[3]), fabsf(v[4]), fabsf(v[5])), fminf(fabsf(v[6]), fabsf(v[7])));
}
// A bound of the smallest of those that are not 0, within an ulp below it; NaN if all are.
__device__ __forceinline__ float min8_not_zero(const float (&v)[8]) {
  uint32_t u = 0xffffffffu;
#pragma unroll
  for (int k = 0; k < 8; ++k) u = min(u, __float_as_uint(v[k]) * 2u - 1u);  // 0 becomes the largest
  return __uint_as_float(u >> 1);
}
// The maximum over the 16 lanes that hold a block of 128.
__device__ __forceinline__ float block_max(float m) {
#pragma unroll
  for (int o = 8; o; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
  return m;
}

// v / scale, correctly rounded; 0 where the scale is 0.  m: the largest |v|.
__device__ __forceinline__ void quotients(float (&v)[8], float m, float scale) {
  if (m > 0x1p-60f && m < 0x1p100f) {
    const float y = reciprocal(scale);
    const pair yy = make_pair2(y, y), ns = make_pair2(-scale, -scale);
#pragma unroll
    for (int k = 0; k < 8; k += 2)
      split(quotient2(make_pair2(v[k], v[k + 1]), ns, yy), v[k], v[k + 1]);
  } else if (scale == 0.0f) {
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = 0.0f;
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = v[k] / scale;
  }
}

// 32 random bits from a pair's number and the tensor's key, already mixed: the
// finaliser of MurmurHash3.
__device__ __forceinline__ uint32_t random_bits(uint32_t h) {
  h = (h ^ h >> 16) * 0x85EBCA6Bu;
  h = (h ^ h >> 13) * 0xC2B2AE35u;
  return h ^ h >> 16;
}

// The E4M3 codes of q in [0, 448], each in the top byte: up with the
// probability of what lies above the code below it, to the nearest 2^-16 (a
// block's largest, whose quotient may be an ulp from 448, keeps its code).
// Times 2^-120 the exponents of both types agree, and E4M3's subnormals are
// fp32's: so the code is bits 20 to 26 of q 2^-120 plus the noise, 16 bits
// below bit 20 and a half of their last.  At least code 1.
__device__ __forceinline__ void random_codes(float a, float b, uint32_t h, uint32_t& ca,
                                             uint32_t& cb) {
  split(mul2(make_pair2(a, b), make_pair2(0x1p-120f, 0x1p-120f)), a, b);
  ca = max(__float_as_uint(a) * 16u + ((h << 8 & 0xffff00u) | 0x80u), 1u << 24);
  cb = max(__float_as_uint(b) * 16u + ((h >> 8 & 0xffff00u) | 0x80u), 1u << 24);
}
__device__ __forceinline__ uint32_t top_bytes(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return __byte_perm(__byte_perm(a, b, 0x0073), __byte_perm(c, d, 0x0073), 0x5410);
}
// Codes of m that nearest gave back, bytes of `code` of the magnitude of `old`'s below
// 8 or (may: 0) of any, take a random code of |m| / scale, q, instead.  h: the random
// bits of the four elements' pairs, of which an element takes the half that its
// neighbour's r takes.
__device__ __forceinline__ uint32_t held_codes(uint32_t code, uint32_t old, uint32_t may,
                                               const float* q, const uint32_t* h) {
  const uint32_t t = ((code ^ old) & 0x7f7f7f7fu) | (old & may);
  const uint32_t held = ~(t + 0x7f7f7f7fu) & 0x80808080u;  // the top bit where a byte of t is 0
  uint32_t c[4];
#pragma unroll
  for (int k = 0; k < 4; k += 2) {
    float a, b;
    split(mul2(make_pair2(q[k], q[k + 1]), make_pair2(0x1p-120f, 0x1p-120f)), a, b);
    // the sign goes; a scale of a few bits, below 2^-133, may leave q above 448
    c[k] = min(__float_as_uint(a) * 16u + ((h[k / 2] >> 8 & 0xffff00u) | 0x80u), 0x7effffffu);
    c[k + 1] = min(__float_as_uint(b) * 16u + ((h[k / 2] << 8 & 0xffff00u) | 0x80u), 0x7effffffu);
  }
  const uint32_t mask = (held >> 7) * 0x7fu;
  return (code & ~mask) | (top_bytes(c[0], c[1], c[2], c[3]) & mask);
}

// What a step reads of eight elements, as it lies in memory: loaded a step
// ahead.  k8: codes and scales, otherwise fp32.
template <typename P, typename G, bool k8>
struct Inputs {
  Raw8<G> g;
  Raw8<P> p;
  Raw8<float> master;
  uint2 mc, vc;
  float ms, vs;
  Raw8<float> m, v;
  __device__ __forceinline__ void load(const AdamwTensor& t, int64_t at) {
    g.load(static_cast<const G*>(t.grad) + at);
    if (t.master)
      master.load(t.master + at);
    else
      p.load(static_cast<const P*>(t.param) + at);
    if constexpr (k8) {
      mc = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(t.m) + at);
      vc = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(t.v) + at);
      ms = t.m_scale[at / kAdamwBlock];
      vs = t.v_scale[at / kAdamwBlock];
    } else {
      m.load(static_cast<const float*>(t.m) + at);
      v.load(static_cast<const float*>(t.v) + at);
    }
  }
};

// Elements [at, at + 8) of a tensor, by a thread; with 8-bit states 16
// neighbouring threads hold a block of 128 (whose lanes are all here).  kFull:
// from `in`; otherwise read here, as far as the tensor goes.
template <typename P, typename G, bool k8, bool kFull>
__device__ __forceinline__ void step8(const AdamwTensor& t, const AdamwScalars& c, float gs,
                                      int64_t at, const Inputs<P, G, k8>& in) {
  const int64_t n = t.n;
  const int64_t block = at / kAdamwBlock;
  float p[8], g[8], m[8], v[8], r[8];
  if constexpr (kFull) {
    in.g.unpack(g);
    if (t.master)
      in.master.unpack(p);
    else
      in.p.unpack(p);
    if constexpr (k8) {
      decode(in.mc, in.ms, m);
      decode(in.vc, in.vs, v);
    } else {
      in.m.unpack(m);
      in.v.unpack(v);
    }
  } else {
    load_tail(static_cast<const G*>(t.grad), at, n, g);
    if (t.master)
      load_tail(static_cast<const float*>(t.master), at, n, p);
    else
      load_tail(static_cast<const P*>(t.param), at, n, p);
    if constexpr (k8) {
      decode(load_codes_tail(t.m, at, n), at < n ? t.m_scale[block] : 0.0f, m);
      decode(load_codes_tail(t.v, at, n), at < n ? t.v_scale[block] : 0.0f, v);
    } else {
      load_tail(static_cast<const float*>(t.m), at, n, m);
      load_tail(static_cast<const float*>(t.v), at, n, v);
    }
  }
#pragma unroll
  for (int k = 0; k < 8; k += 2) {
    const pair gg = mul2(make_pair2(g[k], g[k + 1]), make_pair2(gs, gs));
    const pair mm = add2(mul2(make_pair2(m[k], m[k + 1]), make_pair2(c.b1, c.b1)), c.one,
                         mul2(gg, make_pair2(c.ob1, c.ob1)));
    pair vv = make_pair2(v[k], v[k + 1]);
    if constexpr (k8) vv = mul2(vv, vv);
    vv = add2(mul2(vv, make_pair2(c.b2, c.b2)), c.one,
              mul2(mul2(gg, gg), make_pair2(c.ob2, c.ob2)));
    split(mm, m[k], m[k + 1]);
    split(vv, v[k], v[k + 1]);
  }
  // v and m in a range where no step of the fast forms underflows or overflows: the
  // divisor is in [2^-45, 2^60] (c.vmax), so a quotient in [2^-120, 2^105] and its
  // residual a multiple of 2^-108; an m of 0 gives 0 in any case
  const float vmax = max8_nan(v), mmax = max8_nan(m);
  float mmin = min8(m);
  if (mmin == 0.0f) mmin = min8_not_zero(m);
  const bool tame =
      min8(v) >= 0x1p-90f && vmax <= c.vmax && mmax <= 0x1p60f && !(mmin < 0x1p-60f);
  uint32_t zero[2] = {0, 0};  // bytes 0xff where r is 0
  if (tame) {
#pragma unroll
    for (int k = 0; k < 8; k += 2) {
      const pair rr = sqrt2(make_pair2(v[k], v[k + 1]));
      const pair d = add2(mul2(rr, make_pair2(c.root, c.root)), c.one, make_pair2(c.eps, c.eps));
      const pair u = divide2(make_pair2(m[k], m[k + 1]), d);
      const pair q = add2(mul2(make_pair2(p[k], p[k + 1]), make_pair2(t.decay, t.decay)), c.one,
                          mul2(u, make_pair2(c.nsize, c.nsize)));
      split(rr, r[k], r[k + 1]);
      split(q, p[k], p[k + 1]);
    }
  } else if (vmax == 0.0f && c.eps > 0.0f && mmax == 0.0f) {
    // what no gradient has reached: 0 / eps is m's 0
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      r[k] = 0.0f;
      p[k] = __fadd_rn(__fmul_rn(p[k], t.decay), __fmul_rn(m[k], c.nsize));
    }
    zero[0] = zero[1] = 0xffffffffu;
  } else {
    // v or m of 0, tiny, huge or not finite
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      r[k] = __fsqrt_rn(v[k]);
      const float u = __fdiv_rn(m[k], __fadd_rn(__fmul_rn(r[k], c.root), c.eps));
      p[k] = __fsub_rn(__fmul_rn(p[k], t.decay), __fmul_rn(u, c.size));
      if (r[k] == 0.0f) zero[k / 4] |= 0xffu << 8 * (k & 3);
    }
  }
  if (t.master) store8<kFull>(t.master, at, n, p);
  store8<kFull>(static_cast<P*>(t.param), at, n, p);
  if constexpr (!k8) {
    store8<kFull>(static_cast<float*>(t.m), at, n, m);
    store8<kFull>(static_cast<float*>(t.v), at, n, v);
  } else {
    const float mm = block_max(mmax), rm = block_max(max8_nan(r));
    const float ms = __fmul_rn(mm, 1.0f / 448.0f), rs = __fmul_rn(rm, 1.0f / 448.0f);
    quotients(m, mm, ms);
    const uint64_t j = static_cast<uint64_t>(at) >> 1;  // a multiple of 4
    const uint32_t mixed =
        static_cast<uint32_t>(j) ^ t.key ^ static_cast<uint32_t>(j >> 32) * 0x9E3779B9u;
    uint32_t h[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) h[k] = random_bits(mixed ^ k);
    uint2 code = make_uint2(0x7f7f7f7fu, 0x7f7f7f7fu);  // NaN
    if (rm < __int_as_float(0x7f800000)) {
      quotients(r, rm, rs);
      uint32_t b[8];
#pragma unroll
      for (int k = 0; k < 8; k += 2) random_codes(r[k], r[k + 1], h[k / 2], b[k], b[k + 1]);
      code.x = top_bytes(b[0], b[1], b[2], b[3]) & ~zero[0];
      code.y = top_bytes(b[4], b[5], b[6], b[7]) & ~zero[1];
    }
    uint2 mc = make_uint2(e4m3x2(m[0], m[1]) | e4m3x2(m[2], m[3]) << 16,
                          e4m3x2(m[4], m[5]) | e4m3x2(m[6], m[7]) << 16);
    // a code below 8 is of less than 2^-6 scales (c.held_below; all may be held: inf)
    if (mmin <= __fmul_ru(c.held_below, ms) && mm < __int_as_float(0x7f800000)) {
      // the old codes are still there; read again, as kept they would cost registers
      const uint2 old = kFull ? *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(t.m) + at)
                              : load_codes_tail(t.m, at, n);
      mc.x = held_codes(mc.x, old.x, c.held, m, h);
      mc.y = held_codes(mc.y, old.y, c.held, m + 4, h + 2);
    }
    store_codes8<kFull>(t.m, at, n, mc);
    store_codes8<kFull>(t.v, at, n, code);
    if ((threadIdx.x & 15) == 0 && (kFull || at < n)) {
      t.m_scale[block] = ms;
      t.v_scale[block] = rs;
    }
  }
}

// kMany: kSteps steps a block, each but the first read while the one before it
// is computed; otherwise one, in fewer registers.  352M bf16 elements with a
// master copy and 8-bit states (5.68 GB): 915 us, 6.21 TB/s, 93% of the copy rate,
// with about three quarters of the issue slots taken; without the master copy 134M
// take 349 us, bound by the instructions (about 80 an element).  Of these the range
// check of m and the codes that it is rounded at random are 2 to 4% (895 and 337
// without them), and 17% with beta1 above 29/32, where every code is looked at (398).
// With products and roots one at a time instead of in pairs 938, with the library's
// roots and quotients 1177 (before those two).
template <typename P, typename G, bool k8, bool kMany>
__global__ void __launch_bounds__(kThreads, k8 && kMany ? 3 : 2)
    adamw_kernel(const __grid_constant__ AdamwGroup a) {
  pdl_wait();
  // the tensor of this block: first[lo] <= blockIdx.x < first[lo + 1]
  int lo = a.start[blockIdx.x >> a.shift];
  while (a.first[lo + 1] <= blockIdx.x) ++lo;
  const AdamwTensor& t = a.t[lo];
  const int64_t n = t.n;
  constexpr int kOwn = kMany ? kSteps : 1;
  const int64_t begin = static_cast<int64_t>(blockIdx.x - a.first[lo]) * (kOwn * kStep);
  const int64_t left = n - begin;
  // whole steps of this block, then what is left of the tensor
  const int full = static_cast<int>(min(left / kStep, static_cast<int64_t>(kOwn)));
  int64_t at = begin + threadIdx.x * 8;
  const float gs = a.c.grad_scale ? *a.c.grad_scale : 1.0f;
  Inputs<P, G, k8> in;
  if (full > 0) in.load(t, at);
  for (int step = 0; step < full; ++step, at += kStep) {
    const Inputs<P, G, k8> now = in;
    if (kMany && step + 1 < full) in.load(t, at + kStep);
    step8<P, G, k8, true>(t, a.c, gs, at, now);
    if (!kMany) return;
  }
  if (full < kOwn && at - (threadIdx.x & 31) * 8 < n)  // a warp with something left
    step8<P, G, k8, false>(t, a.c, gs, at, in);
}

// Blocks of a tensor for `steps` steps each.
int64_t blocks_of(int64_t n, int steps) {
  const int64_t chunk = static_cast<int64_t>(kStep) * steps;
  return (n + chunk - 1) / chunk;
}

template <typename P, typename G, bool k8, bool kMany>
cudaError_t launch(AdamwGroup& a, int count, cudaStream_t stream) {
  a.first[0] = 0;
  for (int k = 0; k < count; ++k)
    a.first[k + 1] = a.first[k] + static_cast<uint32_t>(blocks_of(a.t[k].n, kMany ? kSteps : 1));
  const uint32_t blocks = a.first[count];
  if (blocks == 0) return cudaSuccess;  // every tensor is empty
  a.shift = 0;
  while ((blocks - 1) >> a.shift >= kAdamwStarts) ++a.shift;
  for (uint32_t i = 0, lo = 0; i <= (blocks - 1) >> a.shift; ++i) {
    while (a.first[lo + 1] <= i << a.shift) ++lo;
    a.start[i] = static_cast<uint8_t>(lo);
  }
  // launch_pdl, but without further copies of the 19 KB
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(blocks);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl_enabled() ? 1 : 0;
  void* args[] = {&a};
  note_launch();
  return cudaLaunchKernelExC(&cfg, reinterpret_cast<const void*>(adamw_kernel<P, G, k8, kMany>),
                             args);
}

template <typename P, typename G>
cudaError_t launch_states(AdamwGroup& a, int count, bool bits8, bool many, cudaStream_t stream) {
  if (!bits8) return launch<P, G, false, false>(a, count, stream);
  return many ? launch<P, G, true, true>(a, count, stream)
              : launch<P, G, true, false>(a, count, stream);
}

}  // namespace

cudaError_t launch_adamw(AdamwGroup& a, int count, bool param_bf16, bool grad_bf16, bool bits8,
                         int num_sms, int* taken, cudaStream_t stream) {
  int64_t blocks = 0;
  int k = 0;
  for (; k < count; ++k) {
    const int64_t b = blocks_of(a.t[k].n, 1);
    if (k && blocks + b > 0x40000000) break;
    blocks += b;
  }
  *taken = k;
  // 8-bit states: one step a block while there are few blocks, then four (3M
  // elements of bf16 with a master copy 10.7 us with one, 11.5 with four; 16M
  // 53.0 and 47.3; 352M 1065 and 895; eight steps 883, and 49.8 for 16M).
  // 32-bit states need no reading ahead: 134M fp32 523 us with one step in 48
  // registers, 533 with four in 116.
  const bool many = blocks > 16 * num_sms;
  if (param_bf16)
    return grad_bf16 ? launch_states<__nv_bfloat16, __nv_bfloat16>(a, k, bits8, many, stream)
                     : launch_states<__nv_bfloat16, float>(a, k, bits8, many, stream);
  return grad_bf16 ? launch_states<float, __nv_bfloat16>(a, k, bits8, many, stream)
                   : launch_states<float, float>(a, k, bits8, many, stream);
}

}  // namespace fgs
