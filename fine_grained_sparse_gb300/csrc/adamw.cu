// One AdamW step over many tensors in one launch (moe_adamw).  Per element, in
// fp32 with every operation rounded by itself (no contraction, so that a plain
// program of the same operations gives the same bits):
//   g = grad c,  m = b1 m + (1 - b1) g,  v = b2 v + (1 - b2) g g,  r = sqrt v
//   p = p (1 - lr wd) - (m / (r / sqrt(1 - b2^t) + eps)) lr / (1 - b1^t)
// States in 8 bits: m and r as E4M3 codes with one fp32 scale per 128
// elements, max / 448.  m is rounded to nearest: it moves by a tenth of g - m
// in a step, as much as its codes are apart.  v moves by a hundredth or a
// thousandth, which rounding to nearest would take back in every step, so r
// goes to one of the two codes beside it with the probabilities that keep its
// mean, by 16 random bits an element.  A root above 0 has a code above 0: of
// two codes 0 the update m / (0 + eps) of the next step would be unbounded.
// Bound by HBM; the 8-bit form also by its instructions.
#include "common.cuh"
#include "internal.h"
#include "rows.cuh"

namespace fgs {
namespace {

constexpr int kThreads = 256;
constexpr int kStep = 8 * kThreads;  // elements of a block at a time
constexpr int kSteps = 2;
constexpr int64_t kChunk = static_cast<int64_t>(kStep) * kSteps;  // elements of a block

struct AdamwLaunch {
  AdamwTensor t[kAdamwTensors];
  uint32_t first[kAdamwTensors + 1];  // the blocks before each tensor's
  int count;
  AdamwScalars c;
};

// Values [at, at + 8) of a tensor of n, 0 beyond its end.
template <typename T>
__device__ __forceinline__ void load8(const T* p, int64_t at, int64_t n, float (&v)[8]) {
  if (at + 8 <= n) {
    if constexpr (sizeof(T) == 2) {
      const Piece<T, 8> x = load<8>(p + at);
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = x.v[k];
    } else {
      const Piece<T, 4> x = load<4>(p + at), y = load<4>(p + at + 4);
#pragma unroll
      for (int k = 0; k < 4; ++k) v[k] = x.v[k], v[k + 4] = y.v[k];
    }
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = at + k < n ? load<1>(p + at + k).v[0] : 0.0f;
  }
}
template <typename T>
__device__ __forceinline__ void store8(T* p, int64_t at, int64_t n, const float (&v)[8]) {
  if (at + 8 <= n) {
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
__device__ __forceinline__ uint2 load_codes(const uint8_t* p, int64_t at, int64_t n) {
  if (at + 8 <= n) return *reinterpret_cast<const uint2*>(p + at);
  uint2 u = make_uint2(0, 0);
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const uint32_t b = at + k < n ? p[at + k] : 0;
    if (k < 4) u.x |= b << 8 * k; else u.y |= b << 8 * (k - 4);
  }
  return u;
}
__device__ __forceinline__ void store_codes8(uint8_t* p, int64_t at, int64_t n, uint2 u) {
  if (at + 8 <= n) {
    *reinterpret_cast<uint2*>(p + at) = u;
    return;
  }
#pragma unroll
  for (int k = 0; k < 8; ++k)
    if (at + k < n) p[at + k] = static_cast<uint8_t>((k < 4 ? u.x : u.y) >> 8 * (k & 3));
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

// The maximum over the 16 lanes that hold a block of 128, NaN if one is.
__device__ __forceinline__ float block_max(const float (&v)[8]) {
  float m = 0.0f;
#pragma unroll
  for (int k = 0; k < 8; ++k) m = max_nan(m, fabsf(v[k]));
#pragma unroll
  for (int o = 8; o; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
  return m;
}

// v / scale, correctly rounded; 0 where the scale is 0.
__device__ __forceinline__ void quotients(float (&v)[8], float m, float scale) {
  if (m > 0x1p-60f && m < 0x1p126f) {
    divide<8>(v, scale);
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = scale == 0.0f ? 0.0f : v[k] / scale;
  }
}

// 32 random bits of pair j of elements: the finaliser of MurmurHash3.
__device__ __forceinline__ uint32_t random_bits(uint64_t j, uint32_t key) {
  uint32_t h = static_cast<uint32_t>(j) ^ key ^ static_cast<uint32_t>(j >> 32) * 0x9E3779B9u;
  h = (h ^ h >> 16) * 0x85EBCA6Bu;
  h = (h ^ h >> 13) * 0xC2B2AE35u;
  return h ^ h >> 16;
}

// The E4M3 code of q in [0, 448], up with the probability of what lies above
// the code below it, to the nearest 2^-16 (a block's largest, whose quotient
// may be an ulp from 448, keeps its code).  Below 2^-6 codes are 2^-9 apart.
__device__ __forceinline__ uint32_t random_code(float q, uint32_t u, bool some) {
  const int low = static_cast<int>(floorf(__fadd_rn(q * 512.0f, (__uint2float_rn(u) + 0.5f) * 0x1p-16f)));
  const int high = (static_cast<int>(__float_as_uint(q) + (u << 4) + 8) >> 20) - (120 << 3);
  int code = q < 0x1p-6f ? low : high;
  code = min(max(code, some ? 1 : 0), 0x7e);
  return static_cast<uint32_t>(code);
}

template <typename P, typename G, bool k8>
__global__ void __launch_bounds__(kThreads) adamw_kernel(const __grid_constant__ AdamwLaunch a) {
  pdl_wait();
  // the tensor of this block: first[lo] <= blockIdx.x < first[lo + 1]
  int lo = 0, hi = a.count;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a.first[mid] <= blockIdx.x) lo = mid; else hi = mid;
  }
  const AdamwTensor& t = a.t[lo];
  const AdamwScalars& c = a.c;
  const int64_t n = t.n;
  const int64_t begin = static_cast<int64_t>(blockIdx.x - a.first[lo]) * kChunk;
  const float gs = c.grad_scale ? *c.grad_scale : 1.0f;
  for (int step = 0; step < kSteps; ++step) {
    const int64_t start = begin + static_cast<int64_t>(step) * kStep;
    if (start >= n) break;
    const int64_t at = start + threadIdx.x * 8;
    const int64_t block = at / kAdamwBlock;
    float p[8], g[8], m[8], v[8];
    load8(static_cast<const G*>(t.grad), at, n, g);
    if (t.master) {
      load8(static_cast<const float*>(t.master), at, n, p);
    } else {
      load8(static_cast<const P*>(t.param), at, n, p);
    }
    if constexpr (k8) {
      const bool some = at < n;
      decode(load_codes(static_cast<const uint8_t*>(t.m), at, n), some ? t.m_scale[block] : 0.0f, m);
      decode(load_codes(static_cast<const uint8_t*>(t.v), at, n), some ? t.v_scale[block] : 0.0f, v);
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = __fmul_rn(v[k], v[k]);
    } else {
      load8(static_cast<const float*>(t.m), at, n, m);
      load8(static_cast<const float*>(t.v), at, n, v);
    }
    float r[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      g[k] = __fmul_rn(g[k], gs);
      m[k] = __fadd_rn(__fmul_rn(m[k], c.b1), __fmul_rn(g[k], c.ob1));
      v[k] = __fadd_rn(__fmul_rn(v[k], c.b2), __fmul_rn(__fmul_rn(g[k], g[k]), c.ob2));
      r[k] = __fsqrt_rn(v[k]);
      const float u = __fdiv_rn(m[k], __fadd_rn(__fmul_rn(r[k], c.root), c.eps));
      p[k] = __fsub_rn(__fmul_rn(p[k], t.decay), __fmul_rn(u, c.size));
    }
    if (t.master) store8(t.master, at, n, p);
    store8(static_cast<P*>(t.param), at, n, p);
    if constexpr (!k8) {
      store8(static_cast<float*>(t.m), at, n, m);
      store8(static_cast<float*>(t.v), at, n, v);
    } else {
      const float mm = block_max(m), rm = block_max(r);
      const float ms = __fmul_rn(mm, 1.0f / 448.0f), rs = __fmul_rn(rm, 1.0f / 448.0f);
      quotients(m, mm, ms);
      const bool fine = rm < __int_as_float(0x7f800000);
      uint2 code = make_uint2(0x7f7f7f7fu, 0x7f7f7f7fu);  // NaN
      bool some[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) some[k] = r[k] > 0.0f;
      quotients(r, rm, rs);
      if (fine) {
        code = make_uint2(0, 0);
#pragma unroll
        for (int k = 0; k < 8; k += 2) {
          const uint32_t h = random_bits(static_cast<uint64_t>(at + k) >> 1, t.key);
          const uint32_t two = random_code(r[k], h & 0xffff, some[k]) |
                               random_code(r[k + 1], h >> 16, some[k + 1]) << 8;
          if (k < 4) code.x |= two << 8 * k; else code.y |= two << 8 * (k - 4);
        }
      }
      const uint2 mc = make_uint2(e4m3x2(m[0], m[1]) | e4m3x2(m[2], m[3]) << 16,
                                  e4m3x2(m[4], m[5]) | e4m3x2(m[6], m[7]) << 16);
      store_codes8(static_cast<uint8_t*>(t.m), at, n, mc);
      store_codes8(static_cast<uint8_t*>(t.v), at, n, code);
      if ((threadIdx.x & 15) == 0 && at < n) {
        t.m_scale[block] = ms;
        t.v_scale[block] = rs;
      }
    }
  }
}

template <typename P, typename G, bool k8>
cudaError_t launch(const AdamwLaunch& a, cudaStream_t stream) {
  return launch_pdl(adamw_kernel<P, G, k8>, dim3(a.first[a.count]), dim3(kThreads), 0, stream, a);
}

template <typename P, typename G>
cudaError_t launch_bits(const AdamwLaunch& a, bool bits8, cudaStream_t stream) {
  return bits8 ? launch<P, G, true>(a, stream) : launch<P, G, false>(a, stream);
}

}  // namespace

int adamw_group(const AdamwTensor* t, int count) {
  uint64_t blocks = 0;
  int k = 0;
  for (; k < count && k < kAdamwTensors; ++k) {
    const uint64_t b = static_cast<uint64_t>((t[k].n + kChunk - 1) / kChunk);
    if (k && blocks + b > 0x40000000u) break;
    blocks += b;
  }
  return k;
}

cudaError_t launch_adamw(const AdamwTensor* t, int count, const AdamwScalars& c, bool param_bf16,
                         bool grad_bf16, bool bits8, cudaStream_t stream) {
  AdamwLaunch a;
  a.count = count;
  a.c = c;
  a.first[0] = 0;
  for (int k = 0; k < count; ++k) {
    a.t[k] = t[k];
    a.first[k + 1] = a.first[k] + static_cast<uint32_t>((t[k].n + kChunk - 1) / kChunk);
  }
  if (a.first[count] == 0) return cudaSuccess;  // every tensor is empty
  if (param_bf16)
    return grad_bf16 ? launch_bits<__nv_bfloat16, __nv_bfloat16>(a, bits8, stream)
                     : launch_bits<__nv_bfloat16, float>(a, bits8, stream);
  return grad_bf16 ? launch_bits<float, __nv_bfloat16>(a, bits8, stream)
                   : launch_bits<float, float>(a, bits8, stream);
}

}  // namespace fgs
