// Residual sum and root-mean-square norm, with an optional 8-bit output
// (moe_add_rmsnorm).  Per row of d columns:
//   s_i = a_i + r_i,  v_i = w_i s_i / sqrt(mean_i s_i^2 + eps)
//   h = s, y = v, and per 128 columns  scale = max|v| / 448,
//   code_i = e4m3(v_i / scale), the quotient rounded to fp32 first
// Bound by HBM for many rows (each input read once, each output written
// once) and by latency for few.
#include "common.cuh"
#include "internal.h"
#include "rows.cuh"

namespace fgs {
namespace {

struct NormPtrs {
  const void* a;
  const void* r;
  const void* w;
  void* h;
  void* y;
  uint8_t* y8;
  float* ys;
};

// A block a row, or (kWarpRow) a warp a row and kRowsPerBlock rows a block;
// N values at a time.  kKeep pieces of a thread's part stay in registers
// between the sum and the outputs; a wider row (kKeep == 0) is read twice, the
// second time mostly from L2.  Reads of an element come before the writes of
// it, so h and y may be the inputs.
constexpr int kRowsPerBlock = 8;

template <typename T, int N, bool kWarpRow, int kKeep, int kMaxThreads, int kMinBlocks>
__global__ void __launch_bounds__(kMaxThreads, kMinBlocks)
    add_rmsnorm_kernel(const NormPtrs p, float eps, int d, int64_t rows) {
  __shared__ float part[32];
  pdl_wait();
  const int threads = kWarpRow ? 32 : blockDim.x;
  const int tid = kWarpRow ? threadIdx.x & 31 : threadIdx.x;
  const int64_t row = kWarpRow
                          ? static_cast<int64_t>(blockIdx.x) * kRowsPerBlock + threadIdx.x / 32
                          : blockIdx.x;
  const bool live = row < rows;
  const int64_t base = row * d;
  const T* a = static_cast<const T*>(p.a) + base;
  const T* r = p.r ? static_cast<const T*>(p.r) + base : nullptr;
  const T* w = static_cast<const T*>(p.w);
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
  Piece<T, N> keep[kKeep ? kKeep : 1];
  float q = 0.0f;
  if constexpr (kKeep > 0) {
#pragma unroll
    for (int j = 0; j < kKeep; ++j)
      if (tid + j * threads < pieces) keep[j] = sum(tid + j * threads);
#pragma unroll
    for (int j = 0; j < kKeep; ++j)
      if (tid + j * threads < pieces)
#pragma unroll
        for (int k = 0; k < N; ++k) q = fmaf(keep[j].v[k], keep[j].v[k], q);
  } else {
    for (uint32_t i = tid; i < wide; i += threads) {
      const Piece<T, N> s = sum(i);
#pragma unroll
      for (int k = 0; k < N; ++k) q = fmaf(s.v[k], s.v[k], q);
    }
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) q += __shfl_xor_sync(0xffffffffu, q, o);
  if constexpr (!kWarpRow) {
    if ((tid & 31) == 0) part[tid >> 5] = q;
    __syncthreads();
    q = (tid & 31) < threads / 32 ? part[tid & 31] : 0.0f;
#pragma unroll
    for (int o = 16; o; o >>= 1) q += __shfl_xor_sync(0xffffffffu, q, o);
  }
  const float rs = rsqrtf(q / static_cast<float>(d) + eps);

  // a scale group is 128 / N neighbouring lanes of a warp, whose pieces all
  // exist or none does
  auto finish = [&](int i, const Piece<T, N>& s) {
    const int64_t at = static_cast<int64_t>(i) * N;
    const Piece<T, N> g = load<N>(w + at);
    float v[N];
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] = s.v[k] * rs * g.v[k];
    if (p.h) store<N>(static_cast<T*>(p.h) + base + at, s.v);
    if (p.y) store<N>(static_cast<T*>(p.y) + base + at, v);
    if constexpr (N > 1) {
      if (p.y8) {
        constexpr int kLanes = kRowGroup / N;
        float m = 0.0f;
#pragma unroll
        for (int k = 0; k < N; ++k) m = max_nan(m, fabsf(v[k]));
        const uint32_t mask = kLanes == 32 ? 0xffffffffu
                                           : ((1u << (kLanes & 31)) - 1) << (threadIdx.x & 31 & ~(kLanes - 1));
#pragma unroll
        for (int o = kLanes / 2; o; o >>= 1) m = max_nan(m, __shfl_xor_sync(mask, m, o));
        const float scale = m / 448.0f;
        if (m > 0x1p-60f && m < 0x1p126f) {
          divide<N>(v, scale);
        } else {  // zero, tiny and non-finite groups
#pragma unroll
          for (int k = 0; k < N; ++k) v[k] = scale == 0.0f ? 0.0f : v[k] / scale;
        }
        store_codes<N>(p.y8 + base + at, v);
        if ((tid & (kLanes - 1)) == 0) p.ys[row * (d / kRowGroup) + at / kRowGroup] = scale;
      }
    }
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
cudaError_t launch(const NormArgs& n, int threads, cudaStream_t stream) {
  const NormPtrs p = {n.a, n.r, n.w, n.h, n.y, n.y8, n.ys};
  const int64_t blocks = kWarpRow ? (n.T + kRowsPerBlock - 1) / kRowsPerBlock : n.T;
  return launch_pdl(add_rmsnorm_kernel<T, N, kWarpRow, kKeep, kMaxThreads, kMinBlocks>,
                    dim3(static_cast<unsigned>(blocks)),
                    dim3(kWarpRow ? 32 * kRowsPerBlock : threads), 0, stream, p, n.eps, n.d, n.T);
}

// Threads of a row.  Few rows are a matter of latency: a thread a piece.
// Many (two an SM) are one of bandwidth: two pieces a thread, with the
// registers held to three blocks of 512 an SM (8192 x 7168 bf16 with all
// outputs, 530 MB: 448 threads x 2 so held 90.4 us, not held 108.0; 896 x 1
// 91.5; 224 x 4 held to 6 blocks 91.9, not held 100.6; 128 x 7 104.7; the copy
// rate allows 78.4).
template <typename T, int N>
cudaError_t dispatch(const NormArgs& n, int num_sms, cudaStream_t stream) {
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

cudaError_t launch_add_rmsnorm(const NormArgs& n, int num_sms, cudaStream_t stream) {
  if (n.bf16)
    return n.d % 8 ? dispatch<__nv_bfloat16, 1>(n, num_sms, stream)
                   : dispatch<__nv_bfloat16, 8>(n, num_sms, stream);
  return n.d % 4 ? dispatch<float, 1>(n, num_sms, stream) : dispatch<float, 4>(n, num_sms, stream);
}

}  // namespace fgs
