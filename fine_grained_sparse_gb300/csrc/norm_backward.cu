// Gradients of the residual RMS norm and layer norm (moe_norm_backward).  Per
// row of d columns, with s = x + residual, g = w dy and dh the gradient that
// reaches s past the norm:
//   RMS:    u = s r,         r = 1 / sqrt(mean s^2 + eps),
//           dx = r (g - u mean(g u)) + dh
//   layer:  u = (s - mu) r,  r = 1 / sqrt(mean (s - mu)^2 + eps),
//           dx = r (g - mean g - u mean(g u)) + dh
//   dweight = sum over the rows of dy u,  dbias = sum over the rows of dy
// mean(g u) is r mean(g s) (r mean(g (s - mu))), so the RMS form needs one
// reduction over a row and the layer form two.  Bound by HBM for many rows,
// by latency for few.
//
// The rows are dealt to at most kNormParts blocks; each sums its rows' dweight
// and dbias in registers and writes one partial row of each, and a second
// launch adds the partial rows up in a fixed order, so results do not depend
// on timing, nor on the device.
#include "common.cuh"
#include "internal.h"
#include "rows.cuh"

namespace fgs {
namespace {

struct BackwardPtrs {
  const void* a;
  const void* r;
  const void* w;
  const void* dy;
  const void* dh;
  void* dx;
  float* pw;  // [gridDim.x, d] partial dweight, or null
  float* pb;  // and dbias
  float2* stats;  // wide rows: (mu, r) of every row
};

template <typename T, int N>
__device__ __forceinline__ Piece<T, N> row_sum(const T* a, const T* r, int64_t at) {
  Piece<T, N> s = load<N>(a + at);
  if (r) {
    const Piece<T, N> b = load<N>(r + at);
#pragma unroll
    for (int k = 0; k < N; ++k) s.v[k] += b.v[k];
  }
  return s;
}

// Sums of two values over a block's threads (or a warp's), the same in all of
// them.  Callers alternate `buf`: one barrier then separates the uses.
template <bool kWarp>
__device__ __forceinline__ float2 block_sum(float x, float y, float2 (*part)[32], int buf) {
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    x += __shfl_xor_sync(0xffffffffu, x, o);
    y += __shfl_xor_sync(0xffffffffu, y, o);
  }
  if constexpr (!kWarp) {
    const int lane = threadIdx.x & 31;
    if (lane == 0) part[buf][threadIdx.x >> 5] = make_float2(x, y);
    __syncthreads();
    const float2 v = lane < blockDim.x / 32 ? part[buf][lane] : make_float2(0.f, 0.f);
    x = v.x, y = v.y;
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      x += __shfl_xor_sync(0xffffffffu, x, o);
      y += __shfl_xor_sync(0xffffffffu, y, o);
    }
  }
  return make_float2(x, y);
}

// A block a row, or (kWarpRow) a warp a row; a thread holds the same kP pieces
// of N columns of each of its rows.
constexpr int kRowWarps = 8;

template <typename T, int N, int kP, bool kLayer, bool kWarpRow, int kMaxThreads>
__global__ void __launch_bounds__(kMaxThreads)
    norm_backward_kernel(const BackwardPtrs p, float eps, int d, int64_t rows) {
  __shared__ float2 part[2][32];
  pdl_wait();
  const int threads = kWarpRow ? 32 : blockDim.x;
  const int tid = kWarpRow ? threadIdx.x & 31 : threadIdx.x;
  const int teams = kWarpRow ? kRowWarps : 1;
  const int team = kWarpRow ? threadIdx.x / 32 : 0;
  const int pieces = d / N;
  const T* w = static_cast<const T*>(p.w);
  const float inv_d = 1.0f / static_cast<float>(d);
  float dw[kP][N], db[kLayer ? kP : 1][N];
#pragma unroll
  for (int j = 0; j < kP; ++j)
#pragma unroll
    for (int k = 0; k < N; ++k) {
      dw[j][k] = 0.0f;
      if constexpr (kLayer) db[j][k] = 0.0f;
    }
  int buf = 0;
  for (int64_t row = static_cast<int64_t>(blockIdx.x) * teams + team; row < rows;
       row += static_cast<int64_t>(gridDim.x) * teams) {
    const int64_t base = row * d;
    Piece<T, N> s[kP], y[kP];
#pragma unroll
    for (int j = 0; j < kP; ++j) {
      const int i = tid + j * threads;
      if (i < pieces) {
        s[j] = row_sum<T, N>(static_cast<const T*>(p.a),
                             static_cast<const T*>(p.r), base + static_cast<int64_t>(i) * N);
        y[j] = load<N>(static_cast<const T*>(p.dy) + base + static_cast<int64_t>(i) * N);
      } else {
#pragma unroll
        for (int k = 0; k < N; ++k) s[j].v[k] = y[j].v[k] = 0.0f;
      }
    }
    float x0 = 0.0f, x1 = 0.0f, mu = 0.0f, mg = 0.0f;
    if constexpr (kLayer) {
#pragma unroll
      for (int j = 0; j < kP; ++j) {
        const int i = tid + j * threads;
        if (i >= pieces) continue;
        const Piece<T, N> g = load<N>(w + static_cast<int64_t>(i) * N);
#pragma unroll
        for (int k = 0; k < N; ++k) {
          x0 += s[j].v[k];
          x1 = fmaf(y[j].v[k], g.v[k], x1);
        }
      }
      const float2 t = block_sum<kWarpRow>(x0, x1, part, buf);
      buf ^= 1;
      mu = t.x * inv_d;
      mg = t.y * inv_d;
      x0 = x1 = 0.0f;
    }
#pragma unroll
    for (int j = 0; j < kP; ++j) {
      const int i = tid + j * threads;
      if (i >= pieces) continue;
      const Piece<T, N> g = load<N>(w + static_cast<int64_t>(i) * N);
#pragma unroll
      for (int k = 0; k < N; ++k) {
        if constexpr (kLayer) s[j].v[k] -= mu;
        x0 = fmaf(s[j].v[k], s[j].v[k], x0);
        x1 = fmaf(y[j].v[k] * g.v[k], s[j].v[k], x1);
      }
    }
    const float2 t = block_sum<kWarpRow>(x0, x1, part, buf);
    buf ^= 1;
    const float rs = rsqrtf(t.x * inv_d + eps);
    const float c = rs * t.y * inv_d;  // mean(g u)
#pragma unroll
    for (int j = 0; j < kP; ++j) {
      const int i = tid + j * threads;
      if (i >= pieces) continue;
      const int64_t at = base + static_cast<int64_t>(i) * N;
#pragma unroll
      for (int k = 0; k < N; ++k) {
        s[j].v[k] *= rs;
        dw[j][k] = fmaf(y[j].v[k], s[j].v[k], dw[j][k]);
        if constexpr (kLayer) db[j][k] += y[j].v[k];
      }
      if (p.dx) {
        const Piece<T, N> g = load<N>(w + static_cast<int64_t>(i) * N);
        float v[N];
#pragma unroll
        for (int k = 0; k < N; ++k) {
          float f = fmaf(y[j].v[k], g.v[k], -s[j].v[k] * c);
          if constexpr (kLayer) f -= mg;
          v[k] = rs * f;
        }
        if (p.dh) {
          const Piece<T, N> h = load<N>(static_cast<const T*>(p.dh) + at);
#pragma unroll
          for (int k = 0; k < N; ++k) v[k] += h.v[k];
        }
        store<N>(static_cast<T*>(p.dx) + at, v);
      }
    }
  }

  // the block's partial rows; with a warp a row, its warps' in their order
  auto write = [&](float* to, const float (*acc)[N]) {
    if (!to) return;
    to += static_cast<int64_t>(blockIdx.x) * d;
    if constexpr (kWarpRow) {
      __shared__ float sum[32 * kP * N];
      for (int turn = 0; turn < kRowWarps; ++turn) {
        __syncthreads();
        if (turn != team) continue;
#pragma unroll
        for (int j = 0; j < kP; ++j)
#pragma unroll
          for (int k = 0; k < N; ++k) {
            float& at = sum[(j * 32 + tid) * N + k];
            at = turn ? at + acc[j][k] : acc[j][k];
          }
      }
      __syncthreads();
      for (int i = threadIdx.x; i < d; i += blockDim.x) to[i] = sum[i];
      __syncthreads();
    } else {
#pragma unroll
      for (int j = 0; j < kP; ++j) {
        const int i = tid + j * threads;
        if (i >= pieces) continue;
#pragma unroll
        for (int k = 0; k < N; ++k) to[static_cast<int64_t>(i) * N + k] = acc[j][k];
      }
    }
  };
  write(p.pw, dw);
  if constexpr (kLayer) write(p.pb, db);
}

// Rows too wide for registers: dx and the rows' statistics, a block a row,
// reading the row once for each of its sums and once for the output.
template <typename T, int N, bool kLayer>
__global__ void __launch_bounds__(1024)
    norm_backward_wide_kernel(const BackwardPtrs p, float eps, int d) {
  __shared__ float2 part[2][32];
  pdl_wait();
  const int64_t row = blockIdx.x, base = row * d;
  const uint32_t pieces = d / N;
  const T* a = static_cast<const T*>(p.a) + base;
  const T* r = p.r ? static_cast<const T*>(p.r) + base : nullptr;
  const T* w = static_cast<const T*>(p.w);
  const T* dy = static_cast<const T*>(p.dy) + base;
  const float inv_d = 1.0f / static_cast<float>(d);
  float mu = 0.0f, mg = 0.0f, x0 = 0.0f, x1 = 0.0f;
  if constexpr (kLayer) {
    for (uint32_t i = threadIdx.x; i < pieces; i += blockDim.x) {
      const int64_t at = static_cast<int64_t>(i) * N;
      const Piece<T, N> s = row_sum<T, N>(a, r, at), y = load<N>(dy + at), g = load<N>(w + at);
#pragma unroll
      for (int k = 0; k < N; ++k) {
        x0 += s.v[k];
        x1 = fmaf(y.v[k], g.v[k], x1);
      }
    }
    const float2 t = block_sum<false>(x0, x1, part, 0);
    mu = t.x * inv_d;
    mg = t.y * inv_d;
    x0 = x1 = 0.0f;
  }
  for (uint32_t i = threadIdx.x; i < pieces; i += blockDim.x) {
    const int64_t at = static_cast<int64_t>(i) * N;
    const Piece<T, N> s = row_sum<T, N>(a, r, at), y = load<N>(dy + at), g = load<N>(w + at);
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const float u = s.v[k] - mu;
      x0 = fmaf(u, u, x0);
      x1 = fmaf(y.v[k] * g.v[k], u, x1);
    }
  }
  const float2 t = block_sum<false>(x0, x1, part, 1);
  const float rs = rsqrtf(t.x * inv_d + eps);
  const float c = rs * t.y * inv_d;
  if (threadIdx.x == 0 && p.stats) p.stats[row] = make_float2(mu, rs);
  if (!p.dx) return;  // a row's sums are taken before any of it is written: dx may be an input
  for (uint32_t i = threadIdx.x; i < pieces; i += blockDim.x) {
    const int64_t at = static_cast<int64_t>(i) * N;
    const Piece<T, N> s = row_sum<T, N>(a, r, at), y = load<N>(dy + at), g = load<N>(w + at);
    float v[N];
#pragma unroll
    for (int k = 0; k < N; ++k) {
      float f = fmaf(y.v[k], g.v[k], -((s.v[k] - mu) * rs) * c);
      if constexpr (kLayer) f -= mg;
      v[k] = rs * f;
    }
    if (p.dh) {
      const Piece<T, N> h = load<N>(static_cast<const T*>(p.dh) + base + at);
#pragma unroll
      for (int k = 0; k < N; ++k) v[k] += h.v[k];
    }
    store<N>(static_cast<T*>(p.dx) + base + at, v);
  }
}

// Their dweight and dbias: a thread a column, gridDim.y parts of the rows.
template <typename T, bool kLayer>
__global__ void __launch_bounds__(256)
    norm_backward_columns_kernel(const BackwardPtrs p, int d, int64_t rows) {
  pdl_wait();
  const int64_t c = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (c >= d) return;
  const T* a = static_cast<const T*>(p.a);
  const T* r = static_cast<const T*>(p.r);
  float dw = 0.0f, db = 0.0f;
  for (int64_t row = blockIdx.y; row < rows; row += gridDim.y) {
    const float2 st = p.stats[row];
    const float y = load<1>(static_cast<const T*>(p.dy) + row * d + c).v[0];
    dw = fmaf(y, (row_sum<T, 1>(a, r, row * d + c).v[0] - st.x) * st.y, dw);
    if constexpr (kLayer) db += y;
  }
  if (p.pw) p.pw[static_cast<int64_t>(blockIdx.y) * d + c] = dw;
  if constexpr (kLayer)
    if (p.pb) p.pb[static_cast<int64_t>(blockIdx.y) * d + c] = db;
}

// out[c] = the sum of `parts` rows of partials, 32 columns a block: warp w
// adds rows w, w + 32, ..., then the warps' sums are added in their order.
__global__ void __launch_bounds__(1024)
    column_sum_kernel(const float* __restrict__ pw, const float* __restrict__ pb, int parts, int d,
                      float* __restrict__ dw, float* __restrict__ db) {
  __shared__ float sums[32][33];
  pdl_wait();
  const float* p = blockIdx.y ? pb : pw;
  float* out = blockIdx.y ? db : dw;
  if (!out) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t c = static_cast<int64_t>(blockIdx.x) * 32 + lane;
  float s = 0.0f;
  if (c < d)
    for (int i = warp; i < parts; i += 32) s += p[static_cast<int64_t>(i) * d + c];
  sums[warp][lane] = s;
  __syncthreads();
  s = sums[lane][warp];  // lane: the adding warp, warp: the column
#pragma unroll
  for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  const int64_t col = static_cast<int64_t>(blockIdx.x) * 32 + warp;
  if (lane == 0 && col < d) out[col] = s;
}

constexpr int kWideParts = 32;  // parts of the rows of norm_backward_columns_kernel

template <typename T, int N, int kP, bool kLayer, bool kWarpRow, int kMaxThreads>
cudaError_t launch(const NormBackwardArgs& n, int threads, const BackwardPtrs& p, int parts,
                   cudaStream_t stream) {
  return launch_pdl(norm_backward_kernel<T, N, kP, kLayer, kWarpRow, kMaxThreads>,
                    dim3(static_cast<unsigned>(parts)),
                    dim3(kWarpRow ? 32 * kRowWarps : threads), 0, stream, p, n.eps, n.d, n.T);
}

template <typename T, int N, bool kLayer>
cudaError_t dispatch(const NormBackwardArgs& n, cudaStream_t stream) {
  const int pieces = n.d / N;
  const bool sums = n.dw || n.db;
  BackwardPtrs p = {n.a, n.r, n.w, n.dy, n.dh, n.dx, nullptr, nullptr, nullptr};
  auto round32 = [](int v) { return (v + 31) / 32 * 32; };
  constexpr int kMaxP = N == 8 ? 2 : N == 4 ? 4 : 8;
  const bool wide = pieces > 1024 * kMaxP;
  const bool warp = pieces <= 128;
  int parts = static_cast<int>(n.T < kNormParts ? n.T : kNormParts);
  if (warp) {
    const int64_t b = (n.T + kRowWarps - 1) / kRowWarps;
    parts = static_cast<int>(b < kNormParts ? b : kNormParts);
  }
  if (wide) parts = n.T < kWideParts ? static_cast<int>(n.T) : kWideParts;
  float* ws = n.partials;
  if (sums) {
    p.pw = ws;
    p.pb = ws + static_cast<int64_t>(parts) * n.d;
  }
  if (!n.dw) p.pw = nullptr;
  if (!n.db) p.pb = nullptr;
  cudaError_t err;
  if (wide) {
    // the rows' statistics, the columns' sums, then dx, which may be an input
    const dim3 grid(static_cast<unsigned>(n.T));
    if (sums) {
      p.stats = n.stats;
      p.dx = nullptr;
      err = launch_pdl(norm_backward_wide_kernel<T, N, kLayer>, grid, dim3(1024), 0, stream, p,
                       n.eps, n.d);
      if (err != cudaSuccess) return err;
      err = launch_pdl(norm_backward_columns_kernel<T, kLayer>,
                       dim3(static_cast<unsigned>((static_cast<int64_t>(n.d) + 255) / 256), parts),
                       dim3(256), 0, stream, p, n.d, n.T);
      if (err != cudaSuccess) return err;
      p.stats = nullptr;
      p.dx = n.dx;
    }
    err = p.dx ? launch_pdl(norm_backward_wide_kernel<T, N, kLayer>, grid, dim3(1024), 0, stream, p,
                            n.eps, n.d)
               : cudaSuccess;
  } else if (pieces <= 32) {
    err = launch<T, N, 1, kLayer, true, 32 * kRowWarps>(n, 32, p, parts, stream);
  } else if (warp) {
    err = launch<T, N, 4, kLayer, true, 32 * kRowWarps>(n, 32, p, parts, stream);
  } else if (pieces <= 512) {
    err = launch<T, N, 1, kLayer, false, 512>(n, round32(pieces), p, parts, stream);
  } else if (pieces <= 1024) {
    err = launch<T, N, 2, kLayer, false, 512>(n, round32((pieces + 1) / 2), p, parts, stream);
  } else if (N < 8 && pieces <= 2048) {
    err = launch<T, N, 4, kLayer, false, 512>(n, round32((pieces + 3) / 4), p, parts, stream);
  } else {
    err = launch<T, N, kMaxP, kLayer, false, 1024>(n, round32((pieces + kMaxP - 1) / kMaxP), p,
                                                   parts, stream);
  }
  if (err != cudaSuccess || !sums) return err;
  const float *pw = p.pw, *pb = p.pb;
  return launch_pdl(column_sum_kernel,
                    dim3(static_cast<unsigned>((static_cast<int64_t>(n.d) + 31) / 32), n.db ? 2 : 1),
                    dim3(1024), 0, stream, pw, pb, parts, n.d, n.dw, n.db);
}

template <typename T, int N>
cudaError_t dispatch_kind(const NormBackwardArgs& n, cudaStream_t stream) {
  return n.layer ? dispatch<T, N, true>(n, stream) : dispatch<T, N, false>(n, stream);
}

}  // namespace

int64_t norm_partial_floats(int64_t T, int64_t d) {
  return 2 * d * (T < kNormParts ? T : kNormParts);
}

cudaError_t launch_norm_backward(const NormBackwardArgs& n, cudaStream_t stream) {
  if (n.bf16)
    return n.d % 8 ? dispatch_kind<__nv_bfloat16, 1>(n, stream)
                   : dispatch_kind<__nv_bfloat16, 8>(n, stream);
  return n.d % 4 ? dispatch_kind<float, 1>(n, stream) : dispatch_kind<float, 4>(n, stream);
}

}  // namespace fgs
