// Residual sum and root-mean-square norm, with an optional 8-bit output
// (moe_add_rmsnorm).  Per row of d columns:
//   s_i = a_i + r_i,  v_i = w_i s_i / sqrt(mean_i s_i^2 + eps)
//   h = s, y = v, and per 128 columns  scale = max|v| / 448,
//   code_i = e4m3(v_i / scale)
#include "common.cuh"
#include "internal.h"

namespace fgs {
namespace {

constexpr int kNormThreads = 256;
constexpr int kRowGroup = 128;  // columns of a row with one scale

template <typename T>
__device__ __forceinline__ float to_f(T v);
template <>
__device__ __forceinline__ float to_f<float>(float v) {
  return v;
}
template <>
__device__ __forceinline__ float to_f<__nv_bfloat16>(__nv_bfloat16 v) {
  return __bfloat162float(v);
}
template <typename T>
__device__ __forceinline__ T from_f(float v);
template <>
__device__ __forceinline__ float from_f<float>(float v) {
  return v;
}
template <>
__device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float v) {
  return __float2bfloat16_rn(v);
}

// max that keeps NaN, as the definition's maximum over a group does
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

__device__ __forceinline__ uint8_t to_e4m3(float v) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(0.0f), "f"(v));
  return static_cast<uint8_t>(r);
}

// One block a row; a warp takes 128 columns at a time, so that a scale group
// is one warp's values.
template <typename T>
__global__ void __launch_bounds__(kNormThreads)
    add_rmsnorm_kernel(const T* a, const T* r, const T* w, float eps, int d, T* h, T* y,
                       uint8_t* y8, float* ys) {
  pdl_wait();
  __shared__ float part[kNormThreads / 32];
  const int64_t row = blockIdx.x;
  const int64_t base = row * d;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float q = 0.0f;
  for (int c = threadIdx.x; c < d; c += kNormThreads) {
    float s = to_f(a[base + c]);
    if (r) s += to_f(r[base + c]);
    q = fmaf(s, s, q);
  }
  for (int o = 16; o; o >>= 1) q += __shfl_xor_sync(0xffffffffu, q, o);
  if (lane == 0) part[warp] = q;
  __syncthreads();
  q = 0.0f;
  for (int i = 0; i < kNormThreads / 32; ++i) q += part[i];
  const float rs = rsqrtf(q / static_cast<float>(d) + eps);
  for (int c0 = warp * kRowGroup; c0 < d; c0 += kNormThreads / 32 * kRowGroup) {
    float v[4], m = 0.0f;
    for (int i = 0; i < 4; ++i) {
      const int c = c0 + 32 * i + lane;
      v[i] = 0.0f;
      if (c < d) {
        float s = to_f(a[base + c]);
        if (r) s += to_f(r[base + c]);
        if (h) h[base + c] = from_f<T>(s);
        v[i] = s * rs * to_f(w[c]);
        if (y) y[base + c] = from_f<T>(v[i]);
      }
      m = max_nan(m, fabsf(v[i]));
    }
    if (y8) {
      for (int o = 16; o; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
      const float scale = m / 448.0f;
      if (lane == 0) ys[row * (d / kRowGroup) + c0 / kRowGroup] = scale;
      for (int i = 0; i < 4; ++i) {
        const int c = c0 + 32 * i + lane;
        y8[base + c] = to_e4m3(scale == 0.0f ? 0.0f : v[i] / scale);
      }
    }
  }
}

}  // namespace

cudaError_t launch_add_rmsnorm(const NormArgs& n, cudaStream_t stream) {
  if (n.bf16) {
    using B = __nv_bfloat16;
    return launch_pdl(add_rmsnorm_kernel<B>, dim3(static_cast<unsigned>(n.T)), dim3(kNormThreads),
                      0, stream, static_cast<const B*>(n.a), static_cast<const B*>(n.r),
                      static_cast<const B*>(n.w), n.eps, n.d, static_cast<B*>(n.h),
                      static_cast<B*>(n.y), n.y8, n.ys);
  }
  return launch_pdl(add_rmsnorm_kernel<float>, dim3(static_cast<unsigned>(n.T)),
                    dim3(kNormThreads), 0, stream, static_cast<const float*>(n.a),
                    static_cast<const float*>(n.r), static_cast<const float*>(n.w), n.eps, n.d,
                    static_cast<float*>(n.h), static_cast<float*>(n.y), n.y8, n.ys);
}

}  // namespace fgs
