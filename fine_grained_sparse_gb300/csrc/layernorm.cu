// Residual sum and layer norm (moe_add_layernorm).  Per row of d columns:
//   s_i = x_i + r_i,  mu = mean s,  v_i = w_i (s_i - mu) / sqrt(mean (s - mu)^2 + eps) + b_i
//   h = s, y = v
// The variance is taken from the differences to the mean, in a second pass
// over the row's registers, or to a pivot near it: sums of squares lose it where
// |mu| is large.
// Bound by HBM for many rows (each input read once, each output written
// once) and by latency for few.
#include "common.cuh"
#include "internal.h"
#include "rows.cuh"

namespace fgs {
namespace {

constexpr int kRowWarps = 8;

// A block kR neighbouring rows, or (kWarpRow) a warp; a thread the same kP
// chunks of N columns of each, in registers.  Two rows share the barriers and
// trees of their sums, and the weights.  Reads of an element come before the
// writes of it, so h and y may be the inputs.
template <typename T, int N, int kP, int kR, bool kWarpRow, int kMaxThreads, int kMinBlocks>
__global__ void __launch_bounds__(kMaxThreads, kMinBlocks)
    add_layernorm_kernel(const LayerNormArgs p) {
  using C = Chunk<T, N>;
  using V = Vec<N>;
  __shared__ float part[64], part_mean[64];
  pdl_wait();
  const int threads = kWarpRow ? 32 : blockDim.x;
  const int tid = kWarpRow ? threadIdx.x & 31 : threadIdx.x;
  const int64_t row0 = kR * (kWarpRow ? static_cast<int64_t>(blockIdx.x) * kRowWarps + threadIdx.x / 32
                                      : blockIdx.x);
  if (kWarpRow && row0 >= p.T) return;
  const int live = static_cast<int>(min(static_cast<int64_t>(kR), p.T - row0));
  const int chunks = p.d / N;
  const float inv_d = 1.0f / static_cast<float>(p.d);
  auto sums = [&](const V (&a)[kR], float (&x)[kR], float (&to)[64]) {
    const float one = total(a[0]), two = kR > 1 ? total(a[kR - 1]) : 0.0f;
    const float2 t = kWarpRow ? warp_sum(one, two) : block_sum(one, two, to);
    x[0] = t.x * inv_d;
    x[kR - 1] = kR > 1 ? t.y * inv_d : x[0];
  };
  V s[kR][kP], a[kR];
  {
    C x[kR][kP], r[kR][kP];
#pragma unroll
    for (int k = 0; k < kR; ++k)
#pragma unroll
      for (int j = 0; j < kP; ++j) {
        const int i = tid + j * threads;
        if (i >= chunks || k >= live) continue;
        const int64_t at = (row0 + k) * chunks + i;
        x[k][j] = static_cast<const C*>(p.a)[at];
        if (p.r) r[k][j] = static_cast<const C*>(p.r)[at];
      }
#pragma unroll
    for (int k = 0; k < kR; ++k) {
      a[k] = all<N>(0.0f);
#pragma unroll
      for (int j = 0; j < kP; ++j) {
        if (tid + j * threads < chunks && k < live) {
          s[k][j] = unpack(x[k][j]);
          if (p.r) s[k][j] = add(s[k][j], unpack(r[k][j]));
          a[k] = add(a[k], s[k][j]);
        } else {
          s[k][j] = all<N>(0.0f);
        }
      }
    }
  }
  if (p.h) {
#pragma unroll
    for (int k = 0; k < kR; ++k)
#pragma unroll
      for (int j = 0; j < kP; ++j) {
        const int i = tid + j * threads;
        if (i >= chunks || k >= live) continue;
        C out;
        pack(s[k][j], out);
        static_cast<C*>(p.h)[(row0 + k) * chunks + i] = out;
      }
  }
  float mu[kR], rs[kR];
  sums(a, mu, part_mean);
#pragma unroll
  for (int k = 0; k < kR; ++k) {
    a[k] = all<N>(0.0f);
#pragma unroll
    for (int j = 0; j < kP; ++j) {
      if (tid + j * threads >= chunks) continue;
      s[k][j] = add(s[k][j], all<N>(-mu[k]));
      a[k] = fma(s[k][j], s[k][j], a[k]);
    }
  }
  sums(a, rs, part);
#pragma unroll
  for (int k = 0; k < kR; ++k) rs[k] = rsqrtf(rs[k] + p.eps);
#pragma unroll
  for (int j = 0; j < kP; ++j) {
    const int i = tid + j * threads;
    if (i >= chunks) continue;
    const V g = unpack(static_cast<const C*>(p.w)[i]);
    const V b = p.b ? unpack(static_cast<const C*>(p.b)[i]) : all<N>(0.0f);
#pragma unroll
    for (int k = 0; k < kR; ++k) {
      if (k >= live) continue;
      C out;
      pack(fma(mul(s[k][j], all<N>(rs[k])), g, b), out);
      static_cast<C*>(p.y)[(row0 + k) * chunks + i] = out;
    }
  }
}

// Many rows that are not whole 16-byte chunks.  A block's rows are a multiple of N
// apart, so that each begins at the same value of its first chunk: the block holds
// the weights for that shift, reads the chunks that a row reaches into, the next
// row's while it works on one, and clears what there belongs to the rows beside it.
// The sums are taken about a pivot, the mean of the row's first 32 values:
//   mu = pivot + m, m = mean(s - pivot), variance v = mean (s - pivot)^2 - m^2
// Taking m^2 off multiplies the roundings by (v + m^2) / v, up to d / 32 where the first
// values are unlike the rest, and the sum's are those of values of m: so where m^2 exceeds
// v / 4 they are taken once more, about mu.
// 8192 x 7001 bf16 with a residual 106 us, 4.3 TB/s, by single values 231; 16384 x
// 1001 32.5 and 55.7; 4096 x 7001 fp32 106 and 204.
template <typename T, int kP, int kMaxThreads, int kMinBlocks>
__global__ void __launch_bounds__(kMaxThreads, kMinBlocks)
    add_layernorm_shift_kernel(const LayerNormArgs p) {
  constexpr int N = 16 / sizeof(T);
  using C = Chunk<T, N>;
  using V = Vec<N>;
  __shared__ float part[2][64];  // of sums in turn
  pdl_wait();
  const int tid = threadIdx.x, threads = blockDim.x, d = p.d;
  const int shift = static_cast<int>(blockIdx.x * static_cast<int64_t>(d) % N);
  const int chunks = (shift + d + N - 1) / N;
  const float inv_d = 1.0f / static_cast<float>(d);
  auto edge = [&](int j, int& lo, int& hi) {
    const int c = tid + j * threads;
    lo = c ? 0 : shift, hi = min(N, shift + d - c * N);
    return hi - lo < N;
  };
  // the weights and two rows; a thread's chunks, which it alone reads (in
  // registers the weights would be kept as fp32 values)
  extern __shared__ uint4 ring[];
  const int tensors = p.r ? 2 : 1;
  auto slot = [&](int stage, int t, int j) {
    return reinterpret_cast<C*>(ring) + ((2 + stage * tensors + t) * kP + j) * threads + tid;
  };
  auto weight = [&](int t, int j) { return reinterpret_cast<C*>(ring) + (t * kP + j) * threads + tid; };
#pragma unroll
  for (int j = 0; j < kP; ++j) {
    const int at = (tid + j * threads) * N - shift;
    *weight(0, j) = gather<T, N>(static_cast<const T*>(p.w), at, d);
    *weight(1, j) = gather<T, N>(static_cast<const T*>(p.b), at, p.b ? d : 0);
  }
  float first = 0.0f;
  auto fetch = [&](int64_t row, int stage) {
    const int64_t at = row * d / N;
    // the last row's last chunk may reach past the tensors' end
    const bool cut = row == p.T - 1 && p.T * d % N;
    auto one = [&](const void* from, int t) {
#pragma unroll
      for (int j = 0; j < kP; ++j) {
        const int c = tid + j * threads;
        if (c >= chunks) continue;
        if (cut && c == chunks - 1) {
          const int at = c * N - shift;
#pragma unroll 1
          for (int k = 0; at + k < d; ++k)
            reinterpret_cast<T*>(slot(stage, t, j))[k] = static_cast<const T*>(from)[row * d + at + k];
        } else
          copy_async<16>(smem_u32(slot(stage, t, j)), static_cast<const C*>(from) + at + c);
      }
      first += static_cast<float>(static_cast<const T*>(from)[row * d + (tid & 31)]);
    };
    first = 0.0f;
    one(p.a, 0);
    if (p.r) one(p.r, 1);
  };
  int64_t row = blockIdx.x;
  if (row < p.T) fetch(row, 0);
  commit_copies();
  __syncthreads();  // h may be an input: no warp writes the row before all have its first values
  int sum = 0;  // the part of the next sums
  for (int turn = 0; row < p.T; row += gridDim.x, turn ^= 1) {
    float pivot = first;
#pragma unroll
    for (int o = 16; o; o >>= 1) pivot += __shfl_xor_sync(0xffffffffu, pivot, o);
    pivot *= 1.0f / 32;
    if (row + gridDim.x < p.T) fetch(row + gridDim.x, turn ^ 1);
    commit_copies();
    asm volatile("cp.async.wait_group 1;" ::: "memory");
    V s[kP];
#pragma unroll
    for (int j = 0; j < kP; ++j) {
      if (tid + j * threads >= chunks) continue;
      s[j] = unpack(*slot(turn, 0, j));
      if (p.r) s[j] = add(s[j], unpack(*slot(turn, 1, j)));
    }
    const int64_t at = row * d / N;
    auto put = [&](void* to, int j, const V& v) {
      C* const dst = static_cast<C*>(to) + at + tid + j * threads;
      C out;
      pack(v, out);
      int lo, hi;
      if (edge(j, lo, hi)) {
        C* const own = slot(turn, 0, j);  // its values are in registers by now
        *own = out;
#pragma unroll 1
        for (int k = lo; k < hi; ++k)
          reinterpret_cast<T*>(dst)[k] = reinterpret_cast<const T*>(own)[k];
      } else {
        *dst = out;
      }
    };
    if (p.h) {
#pragma unroll
      for (int j = 0; j < kP; ++j)
        if (tid + j * threads < chunks) put(p.h, j, s[j]);
    }
    // s, the row, less `at`, and the sums of it and of its squares
    auto sums = [&](float at) {
      V m = all<N>(0.0f), q = m;
      const V na = all<N>(-at);
#pragma unroll
      for (int j = 0; j < kP; ++j) {
        if (tid + j * threads >= chunks) continue;
        int lo, hi;
        if (edge(j, lo, hi)) clip(s[j], lo, hi, at);  // 0 to the sums
        s[j] = add(s[j], na);
        m = add(m, s[j]);
        q = fma(s[j], s[j], q);
      }
      sum ^= 1;
      return block_sum(total(m), total(q), part[sum]);
    };
    float2 t = sums(pivot);
    float mu = t.x * inv_d, var = fmaf(-mu, mu, t.y * inv_d);
    if (4.0f * mu * mu > var) {  // the same in all threads
      t = sums(mu);
      mu = t.x * inv_d, var = fmaf(-mu, mu, t.y * inv_d);
    }
    const V rs = all<N>(rsqrtf(var + p.eps)), nm = all<N>(-mu);
#pragma unroll
    for (int j = 0; j < kP; ++j)
      if (tid + j * threads < chunks)
        put(p.y, j, fma(mul(add(s[j], nm), rs), unpack(*weight(0, j)), unpack(*weight(1, j))));
  }
}

// Rows too wide for registers: a block a row, which it reads three times.
template <typename T, int N>
__global__ void __launch_bounds__(1024) add_layernorm_wide_kernel(const LayerNormArgs p) {
  __shared__ float part[64], part_mean[64];
  pdl_wait();
  const int64_t base = blockIdx.x * static_cast<int64_t>(p.d);
  const T* a = static_cast<const T*>(p.a) + base;
  const T* r = p.r ? static_cast<const T*>(p.r) + base : nullptr;
  const uint32_t pieces = p.d / N;  // unsigned: a step beyond the last piece may pass 2^31
  const float inv_d = 1.0f / static_cast<float>(p.d);
  auto sum = [&](int64_t at) {
    Piece<T, N> s = load<N>(a + at);
    if (r) {
      const Piece<T, N> b = load<N>(r + at);
#pragma unroll
      for (int k = 0; k < N; ++k) s.v[k] += b.v[k];
    }
    return s;
  };
  float q = 0.0f;
  for (uint32_t i = threadIdx.x; i < pieces; i += 1024) {
    const Piece<T, N> s = sum(static_cast<int64_t>(i) * N);
#pragma unroll
    for (int k = 0; k < N; ++k) q += s.v[k];
  }
  const float mu = block_sum(q, 0.0f, part_mean).x * inv_d;
  q = 0.0f;
  for (uint32_t i = threadIdx.x; i < pieces; i += 1024) {
    const Piece<T, N> s = sum(static_cast<int64_t>(i) * N);
#pragma unroll
    for (int k = 0; k < N; ++k) q = fmaf(s.v[k] - mu, s.v[k] - mu, q);
  }
  const float rs = rsqrtf(block_sum(q, 0.0f, part).x * inv_d + p.eps);
  for (uint32_t i = threadIdx.x; i < pieces; i += 1024) {
    const int64_t at = static_cast<int64_t>(i) * N;
    const Piece<T, N> s = sum(at), g = load<N>(static_cast<const T*>(p.w) + at);
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
  }
}

template <typename T, int N, int kP, int kR, bool kWarpRow, int kMaxThreads, int kMinBlocks = 1>
cudaError_t launch(const LayerNormArgs& n, int threads, cudaStream_t stream) {
  constexpr int kRows = kR * (kWarpRow ? kRowWarps : 1);
  return launch_pdl(add_layernorm_kernel<T, N, kP, kR, kWarpRow, kMaxThreads, kMinBlocks>,
                    dim3(static_cast<unsigned>((n.T + kRows - 1) / kRows)), dim3(threads), 0, stream,
                    n);
}

template <typename T, int N>
cudaError_t dispatch(const LayerNormArgs& n, int num_sms, cudaStream_t stream) {
  // threads of a row with at most Q values each
  auto threads = [&](int Q) { return (n.d + 32 * Q - 1) / (32 * Q) * 32; };
  constexpr int kWarps = 32 * kRowWarps;
  if (n.d > 16384) {
    constexpr int W = N == 2 ? 1 : N;  // a Piece is one value or 16 bytes
    return launch_pdl(add_layernorm_wide_kernel<T, W>, dim3(static_cast<unsigned>(n.T)), dim3(1024),
                      0, stream, n);
  }
  if (n.d > 8192) return launch<T, N, 16 / N, 1, false, 1024>(n, threads(16), stream);
  if (n.T < 2 * num_sms)
    return n.d <= 256 ? launch<T, N, 8 / N, 1, true, kWarps>(n, kWarps, stream)
                      : launch<T, N, 8 / N, 1, false, 1024>(n, threads(8), stream);
  if constexpr (N == 1) {
    // (8192 x 7002, in pairs of values, 111 us and 104 here, 16384 x 1002 30.1 and 32.6;
    // 32768 x 501, a warp two rows, 36.8 and 52.8)
    constexpr int kChunk = 16 / sizeof(T), kMost = sizeof(T) == 2 ? 512 : 1024;
    const int wide = (span_chunks<kChunk>(n.d) + 63) / 64 * 32;
    if (n.d > 512 && wide <= kMost) {
      int64_t blocks = static_cast<int64_t>(num_sms) * (1024 / wide < 16 ? 1024 / wide : 16);
      if (blocks > n.T) blocks = n.T;
      auto kernel = add_layernorm_shift_kernel<T, 2, kMost, 1024 / kMost>;
      const size_t bytes = (2 + 2 * (n.r ? 2 : 1)) * 2 * 16 * static_cast<size_t>(wide);
      const cudaError_t err =
          cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 200 * 1024);
      if (err != cudaSuccess) return err;
      return launch_pdl(kernel, dim3(static_cast<unsigned>((blocks + 7) / 8 * 8)), dim3(wide), bytes,
                        stream, n);
    }
  }
  // many rows: two at a time where bf16 makes the instructions count (8192 x 7168
  // with a residual, 470 MB: 70.1 us, the copy rate; a row a block, without pairs
  // of values, 82.3; three such blocks an SM spill, 137), one where fp32 does not
  // (8191 x 3584, 235 MB: 38.8 us, 90% of it; 32768 x 1000 40.6, 96%)
  if (n.d <= 256) return launch<T, N, 8 / N, 2, true, kWarps>(n, kWarps, stream);
  if constexpr (sizeof(T) == 4) {
    if (n.d <= 2048) return launch<T, N, 8 / N, 1, false, 256, 8>(n, threads(8), stream);
    if (n.d <= 4096) return launch<T, N, 16 / N, 1, false, 256, 4>(n, threads(16), stream);
    return launch<T, N, 16 / N, 1, false, 512, 1>(n, threads(16), stream);
  } else {
    if (n.d <= 512) return launch<T, N, 16 / N, 2, true, kWarps>(n, kWarps, stream);
    if (n.d <= 1024) return launch<T, N, 32 / N, 2, true, kWarps>(n, kWarps, stream);
    // up to 448 threads a block may have more registers than with 512: 8192 x 7168 69.8 and
    // 70.5 us, without a residual 47.3 and 48.7, 6144 columns 60.7 and 62.2, 7002 110 and 118
    // (but 4096 without a residual 29.4 and 26.0, 5002 92 and 79; rows by pairs or single
    // values spill 30 to 140 bytes a thread in either)
    if (n.d <= 7168) return launch<T, N, 16 / N, 2, false, 448, 2>(n, threads(16), stream);
    return launch<T, N, 16 / N, 2, false, 512, 2>(n, threads(16), stream);
  }
}

}  // namespace

cudaError_t launch_add_layernorm(const LayerNormArgs& n, int num_sms, cudaStream_t stream) {
  if (n.bf16)
    return n.d % 8 == 0   ? dispatch<__nv_bfloat16, 8>(n, num_sms, stream)
           : n.d % 2 == 0 ? dispatch<__nv_bfloat16, 2>(n, num_sms, stream)
                          : dispatch<__nv_bfloat16, 1>(n, num_sms, stream);
  return n.d % 4 == 0 ? dispatch<float, 4>(n, num_sms, stream)
                      : dispatch<float, 1>(n, num_sms, stream);
}

}  // namespace fgs
