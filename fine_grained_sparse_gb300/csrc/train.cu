// Around the experts' products in training: the rows in expert order
// (moe_gather), and the way back through the weighted combine
// (moe_combine_backward) and through the gate weights (moe_router_backward).
//
// Kernels
//   gather_rows_kernel       x_perm[inv[t K + k]] = x[t], w_perm likewise
//   combine_backward_kernel  y[t] = sum_k w[t, k] Y[inv[t K + k]], so
//                            dY[inv[t K + k]] = w[t, k] dy[t] and
//                            dw[t, k] = <Y[inv[t K + k]], dy[t]>
//   router_backward_kernel   w_k = c p_k, p_k = s_k / (sum_j s_j + 1e-20),
//                            s = sigmoid(z): dp_k/ds_j = (delta_kj - p_k) / S, so
//                            dz_k = c p_k (dw_k - sum_j p_j dw_j) (1 - s_k)
// All are launched with programmatic stream serialization and wait for the
// previous kernel (pdl_wait) before touching global memory.
#include "common.cuh"
#include "internal.h"

namespace fgs {

namespace {

constexpr int kMaxK = 32;

// A CTA per token, or per (token, slice of the row) for small batches.  A row
// is read once and written to the slots of its K pairs; a slot outside
// [0, rows) (inv = -1: a pair that the sort rejected) is left out.  Bound by
// HBM's writes: 8192 x 7168 bf16, K 8 (1.06 GB) 168 us, 6.3 TB/s, 94% of the
// copy rate; the stores are marked as streaming (2000 tokens, whose rows would
// fill L2, 50 us without the mark, 40 with it).
__global__ void __launch_bounds__(128) gather_rows_kernel(
    const uint4* __restrict__ x, int K, int nvec, const int32_t* __restrict__ inv,
    const float* __restrict__ w, int64_t rows, uint4* __restrict__ xp, float* __restrict__ wp) {
  pdl_wait();
  __shared__ int slots[kMaxK];
  const int64_t t = blockIdx.x;
  if (threadIdx.x < K) {
    const int s = __ldg(inv + t * K + threadIdx.x);
    const bool in = s >= 0 && s < rows;
    slots[threadIdx.x] = in ? s : -1;
    if (in && wp && blockIdx.y == 0) wp[s] = __ldg(w + t * K + threadIdx.x);
  }
  __syncthreads();
  const uint4* src = x + t * nvec;
  for (int v = blockIdx.y * blockDim.x + threadIdx.x; v < nvec; v += gridDim.y * blockDim.x) {
    const uint4 u = __ldg(src + v);
    for (int k = 0; k < K; ++k)
      if (slots[k] >= 0) __stcs(xp + static_cast<int64_t>(slots[k]) * nvec + v, u);
  }
}

// Eight values of a row as fp32, 16 or 32 bytes.
template <bool BF16>
struct Row8;
template <>
struct Row8<true> {
  uint4 u;
  __device__ __forceinline__ void load(const void* p, int64_t i) {
    u = __ldcs(reinterpret_cast<const uint4*>(p) + i);
  }
  __device__ __forceinline__ void unpack(float (&v)[8]) const {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      v[2 * q] = __uint_as_float(w[q] << 16);
      v[2 * q + 1] = __uint_as_float(w[q] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ void store(void* p, int64_t i, const float (&v)[8]) {
    __stcs(reinterpret_cast<uint4*>(p) + i, make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                                pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])));
  }
};
template <>
struct Row8<false> {
  float4 a, b;
  __device__ __forceinline__ void load(const void* p, int64_t i) {
    a = __ldcs(reinterpret_cast<const float4*>(p) + 2 * i);
    b = __ldcs(reinterpret_cast<const float4*>(p) + 2 * i + 1);
  }
  __device__ __forceinline__ void unpack(float (&v)[8]) const {
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
    v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  }
  static __device__ __forceinline__ void store(void* p, int64_t i, const float (&v)[8]) {
    __stcs(reinterpret_cast<float4*>(p) + 2 * i, make_float4(v[0], v[1], v[2], v[3]));
    __stcs(reinterpret_cast<float4*>(p) + 2 * i + 1, make_float4(v[4], v[5], v[6], v[7]));
  }
};

// A CTA per token and kB of its pairs.  Each piece of dy is multiplied with
// the same piece of the pairs' rows (dw, summed in fp32: over a thread's
// pieces, the warp, the CTA) and written to their rows of dY, scaled.  dY may
// be Y: an element is read before its thread writes it.
template <bool BF16, int kB, int kThreads>
__global__ void __launch_bounds__(kThreads) combine_backward_kernel(
    const void* __restrict__ dy, const void* Y, const int32_t* __restrict__ inv,
    const float* __restrict__ w, int K, int nvec, int64_t rows, void* dY, float* __restrict__ dw) {
  pdl_wait();
  using R = Row8<BF16>;
  __shared__ int slots[kB];
  __shared__ float wts[kB];
  __shared__ float part[kThreads / 32][kB];
  const int64_t t = blockIdx.x;
  const int k0 = blockIdx.y * kB;
  const int nk = min(kB, K - k0);
  if (threadIdx.x < nk) {
    const int64_t j = t * K + k0 + threadIdx.x;
    const int s = __ldg(inv + j);
    slots[threadIdx.x] = s >= 0 && s < rows ? s : -1;
    wts[threadIdx.x] = w ? __ldg(w + j) : 1.0f;
  }
  __syncthreads();
  float acc[kB];
#pragma unroll
  for (int i = 0; i < kB; ++i) acc[i] = 0.0f;
  for (int v = threadIdx.x; v < nvec; v += kThreads) {
    R d, y[kB];
    d.load(dy, t * nvec + v);
    if (dw) {
#pragma unroll
      for (int i = 0; i < kB; ++i)
        if (i < nk && slots[i] >= 0) y[i].load(Y, static_cast<int64_t>(slots[i]) * nvec + v);
    }
    float g[8], u[8];
    d.unpack(g);
#pragma unroll
    for (int i = 0; i < kB; ++i) {
      if (i >= nk || slots[i] < 0) continue;
      if (dw) {
        y[i].unpack(u);
#pragma unroll
        for (int q = 0; q < 8; ++q) acc[i] = fmaf(u[q], g[q], acc[i]);
      }
      if (dY) {
        const float wk = wts[i];
#pragma unroll
        for (int q = 0; q < 8; ++q) u[q] = wk * g[q];
        R::store(dY, static_cast<int64_t>(slots[i]) * nvec + v, u);
      }
    }
  }
  if (!dw) return;
#pragma unroll
  for (int i = 0; i < kB; ++i) {
#pragma unroll
    for (int o = 16; o; o >>= 1) acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], o);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5][i] = acc[i];
  }
  __syncthreads();
  if (threadIdx.x < nk) {
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < kThreads / 32; ++i) s += part[i][threadIdx.x];
    dw[t * K + k0 + threadIdx.x] = s;
  }
}

// A warp per token: lane k holds pair k.  The row of dz is zeroed, then the
// pairs' entries are written over the zeros; an expert that a token lists
// more than once receives the sum of its pairs, from the first of them.  The
// zeros go out while the loads are under way: 8192 x 896, K 16 (30.9 MB) 6.9 us
// on data in L2, 8.6 among others, of which a launch of 128 tokens takes 2.1;
// zeros first 7.6 and 9.7, the row put together in shared memory 8.2 and 9.8.
constexpr int kRouterWarps = 4;
__global__ void __launch_bounds__(32 * kRouterWarps) router_backward_kernel(
    const float* __restrict__ z, const int32_t* __restrict__ idx, const float* __restrict__ dw,
    int64_t T, int K, int E, float scale, int renorm, float* __restrict__ dz) {
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * kRouterWarps + (threadIdx.x >> 5);
  if (t >= T) return;
  float* row = dz + t * E;
  const int at = lane < K ? __ldg(idx + t * K + lane) : -1;
  const float d0 = lane < K ? __ldg(dw + t * K + lane) : 0.0f;
  const bool in = at >= 0 && at < E;
  const float zk = in ? __ldg(z + t * E + at) : 0.0f;
  if (E % 4 == 0) {
    for (int e = lane; e < E / 4; e += 32)
      reinterpret_cast<float4*>(row)[e] = make_float4(0.f, 0.f, 0.f, 0.f);
  } else {
    for (int e = lane; e < E; e += 32) row[e] = 0.0f;
  }
  float g = 0.0f;
  {
    const float d = in ? d0 : 0.0f;
    // sigmoid(z), times 2^64 so that it holds where e^z is below fp32's range,
    // and 1 - sigmoid(z), each without cancellation
    const float h = expf(-0.5f * fabsf(zk)), e = h * h;
    const float up = 1.0f / (1.0f + e);
    float p = zk >= 0.0f ? 0x1p64f * up : (0x1p32f * h) * (0x1p32f * h) * up;
    const float rest = zk >= 0.0f ? e * up : up;
    if (!in) p = 0.0f;
    float mean = 0.0f;
    if (renorm) {
      float sum = p;
#pragma unroll
      for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      p /= sum + 1e-20f * 0x1p64f;
      mean = p * d;
#pragma unroll
      for (int o = 16; o; o >>= 1) mean += __shfl_xor_sync(0xffffffffu, mean, o);
    } else {
      p *= 0x1p-64f;
    }
    g = in ? scale * p * (d - mean) * rest : 0.0f;
  }
  const unsigned same = __match_any_sync(0xffffffffu, in ? at : E + lane);
  const bool first = (same & ((1u << lane) - 1)) == 0;
  float sum = 0.0f;
  for (int k = 0; k < K; ++k) {
    const float gk = __shfl_sync(0xffffffffu, g, k);
    if (same >> k & 1) sum += gk;
  }
  __syncwarp();  // the zeros come first
  if (in && first) row[at] = sum;
}

template <bool BF16>
cudaError_t combine_backward(const void* dy, const void* Y, const int32_t* inv,
                             const float* w, int64_t T, int K, int D, int num_sms, void* dY,
                             float* dw, cudaStream_t stream) {
  const int64_t rows = T * K;
  auto launch = [&](auto kernel, int kB) {
    return launch_pdl(kernel, dim3(static_cast<unsigned>(T), static_cast<unsigned>((K + kB - 1) / kB)),
                      dim3(128), 0, stream, dy, Y, inv, w, K, D / 8, rows, dY, dw);
  };
  // eight pairs a block, so that dy is read and unpacked once for them (4096 x
  // 3584, K 16: 149 us, with four 157); fewer where blocks would be few (us with
  // one / four / eight: 16 x 7168, K 8 3.2 / 4.4 / 7.0; 500 x 7168 20 / 16 / 19)
  if (K == 1 || T <= num_sms) return launch(combine_backward_kernel<BF16, 1, 128>, 1);
  if (K == 2) return launch(combine_backward_kernel<BF16, 2, 128>, 2);
  if (K <= 4 || (T <= 4 * num_sms && K % 4 == 0))
    return launch(combine_backward_kernel<BF16, 4, 128>, 4);
  return launch(combine_backward_kernel<BF16, 8, 128>, 8);
}

}  // namespace

cudaError_t launch_gather_rows(const void* x, const int32_t* inv, const float* w, int64_t T, int K,
                               int nvec, void* xp, float* wp, cudaStream_t stream) {
  // small batches: several CTAs a row
  const unsigned slices = T < 1024 ? static_cast<unsigned>((nvec + 127) / 128) : 1u;
  return launch_pdl(gather_rows_kernel, dim3(static_cast<unsigned>(T), slices), dim3(128), 0, stream,
                    static_cast<const uint4*>(x), K, nvec, inv, w, T * K, static_cast<uint4*>(xp),
                    wp);
}

cudaError_t launch_combine_backward(const void* dy, const void* Y, const int32_t* inv,
                                    const float* w, int64_t T, int K, int D, bool bf16, int num_sms,
                                    void* dY, float* dw, cudaStream_t stream) {
  return bf16 ? combine_backward<true>(dy, Y, inv, w, T, K, D, num_sms, dY, dw, stream)
              : combine_backward<false>(dy, Y, inv, w, T, K, D, num_sms, dY, dw, stream);
}

cudaError_t launch_router_backward(const float* logits, const int32_t* idx, const float* dw,
                                   int64_t T, int K, int E, float scale, bool renorm, float* dz,
                                   cudaStream_t stream) {
  return launch_pdl(router_backward_kernel,
                    dim3(static_cast<unsigned>((T + kRouterWarps - 1) / kRouterWarps)),
                    dim3(32 * kRouterWarps), 0, stream, logits, idx, dw, T, K, E, scale,
                    renorm ? 1 : 0, dz);
}

}  // namespace fgs
