// Residual sum and layer norm (moe_add_layernorm).  Per row of d columns:
//   s_i = x_i + r_i,  mu = mean s,  v_i = w_i (s_i - mu) / sqrt(mean (s - mu)^2 + eps) + b_i
//   h = s, y = v
// The variance is taken from the differences to the mean, in a second pass
// over the row's registers: sums of squares lose it where |mu| is large.
// Bound by HBM for many rows (each input read once, each output written
// once) and by latency for few.
#include "common.cuh"
#include "internal.h"
#include "rows.cuh"

namespace fgs {
namespace {

constexpr int kRowsPerBlock = 8;

// As add_rmsnorm_kernel: a block a row, or (kWarpRow) a warp a row; N values at
// a time; kKeep pieces of a thread's part stay in registers, a wider row
// (kKeep == 0) is read three times.  Reads of an element come before the writes
// of it, so h and y may be the inputs.
template <typename T, int N, bool kWarpRow, int kKeep, int kMaxThreads, int kMinBlocks>
__global__ void __launch_bounds__(kMaxThreads, kMinBlocks)
    add_layernorm_kernel(const LayerNormArgs p) {
  __shared__ float part[2][32];
  pdl_wait();
  const int d = p.d;
  const int threads = kWarpRow ? 32 : blockDim.x;
  const int tid = kWarpRow ? threadIdx.x & 31 : threadIdx.x;
  const int64_t row = kWarpRow
                          ? static_cast<int64_t>(blockIdx.x) * kRowsPerBlock + threadIdx.x / 32
                          : blockIdx.x;
  const bool live = row < p.T;
  const int64_t base = row * d;
  const T* a = static_cast<const T*>(p.a) + base;
  const T* r = p.r ? static_cast<const T*>(p.r) + base : nullptr;
  const int pieces = live ? d / N : 0;
  const uint32_t wide = pieces;  // unsigned: a step beyond the last piece may pass 2^31

  auto sum = [&](int i) {
    Piece<T, N> s = load<N>(a + static_cast<int64_t>(i) * N);
    if (r) {
      const Piece<T, N> b = load<N>(r + static_cast<int64_t>(i) * N);
#pragma unroll
      for (int k = 0; k < N; ++k) s.v[k] += b.v[k];
    }
    return s;
  };
  auto mean = [&](float q, int use) {
#pragma unroll
    for (int o = 16; o; o >>= 1) q += __shfl_xor_sync(0xffffffffu, q, o);
    if constexpr (!kWarpRow) {
      if ((tid & 31) == 0) part[use][tid >> 5] = q;
      __syncthreads();
      q = (tid & 31) < threads / 32 ? part[use][tid & 31] : 0.0f;
#pragma unroll
      for (int o = 16; o; o >>= 1) q += __shfl_xor_sync(0xffffffffu, q, o);
    }
    return q / static_cast<float>(d);
  };
  Piece<T, N> keep[kKeep ? kKeep : 1];
  float q = 0.0f, mu, rs;
  if constexpr (kKeep > 0) {
#pragma unroll
    for (int j = 0; j < kKeep; ++j)
      if (tid + j * threads < pieces) keep[j] = sum(tid + j * threads);
#pragma unroll
    for (int j = 0; j < kKeep; ++j)
      if (tid + j * threads < pieces)
#pragma unroll
        for (int k = 0; k < N; ++k) q += keep[j].v[k];
    mu = mean(q, 0);
    q = 0.0f;
#pragma unroll
    for (int j = 0; j < kKeep; ++j)
      if (tid + j * threads < pieces)
#pragma unroll
        for (int k = 0; k < N; ++k) q = fmaf(keep[j].v[k] - mu, keep[j].v[k] - mu, q);
  } else {
    for (uint32_t i = tid; i < wide; i += threads) {
      const Piece<T, N> s = sum(i);
#pragma unroll
      for (int k = 0; k < N; ++k) q += s.v[k];
    }
    mu = mean(q, 0);
    q = 0.0f;
    for (uint32_t i = tid; i < wide; i += threads) {
      const Piece<T, N> s = sum(i);
#pragma unroll
      for (int k = 0; k < N; ++k) q = fmaf(s.v[k] - mu, s.v[k] - mu, q);
    }
  }
  rs = rsqrtf(mean(q, 1) + p.eps);

  auto finish = [&](int i, const Piece<T, N>& s) {
    const int64_t at = static_cast<int64_t>(i) * N;
    const Piece<T, N> g = load<N>(static_cast<const T*>(p.w) + at);
    float v[N];
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] = (s.v[k] - mu) * rs * g.v[k];
    if (p.b) {
      const Piece<T, N> b = load<N>(static_cast<const T*>(p.b) + at);
#pragma unroll
      for (int k = 0; k < N; ++k) v[k] += b.v[k];
    }
    if (p.h) store<N>(static_cast<T*>(p.h) + base + at, s.v);
    store<N>(static_cast<T*>(p.y) + base + at, v);
  };
  if constexpr (kKeep > 0) {
#pragma unroll
    for (int j = 0; j < kKeep; ++j)
      if (tid + j * threads < pieces) finish(tid + j * threads, keep[j]);
  } else {
    for (uint32_t i = tid; i < wide; i += threads) finish(i, sum(i));
  }
}

template <typename T, int N, bool kWarpRow, int kKeep, int kMaxThreads, int kMinBlocks = 1>
cudaError_t launch(const LayerNormArgs& n, int threads, cudaStream_t stream) {
  const int64_t blocks = kWarpRow ? (n.T + kRowsPerBlock - 1) / kRowsPerBlock : n.T;
  return launch_pdl(add_layernorm_kernel<T, N, kWarpRow, kKeep, kMaxThreads, kMinBlocks>,
                    dim3(static_cast<unsigned>(blocks)),
                    dim3(kWarpRow ? 32 * kRowsPerBlock : threads), 0, stream, n);
}

template <typename T, int N>
cudaError_t dispatch(const LayerNormArgs& n, int num_sms, cudaStream_t stream) {
  const int pieces = n.d / N;
  auto round32 = [](int v) { return (v + 31) / 32 * 32; };
  if (pieces <= 32) return launch<T, N, true, 1, 32 * kRowsPerBlock>(n, 32, stream);
  if (pieces <= 128) return launch<T, N, false, 1, 1024>(n, round32(pieces), stream);
  if (pieces <= 1024)
    return n.T < 2 * num_sms ? launch<T, N, false, 1, 1024>(n, round32(pieces), stream)
                             : launch<T, N, false, 2, 512, 3>(n, round32((pieces + 1) / 2), stream);
  if (pieces <= 4096) return launch<T, N, false, 4, 1024>(n, round32((pieces + 3) / 4), stream);
  return launch<T, N, false, 0, 1024>(n, 1024, stream);
}

}  // namespace

cudaError_t launch_add_layernorm(const LayerNormArgs& n, int num_sms, cudaStream_t stream) {
  if (n.bf16)
    return n.d % 8 ? dispatch<__nv_bfloat16, 1>(n, num_sms, stream)
                   : dispatch<__nv_bfloat16, 8>(n, num_sms, stream);
  return n.d % 4 ? dispatch<float, 1>(n, num_sms, stream) : dispatch<float, 4>(n, num_sms, stream);
}

}  // namespace fgs
