// Gradients of the residual RMS norm and layer norm (moe_norm_backward).  Per
// row of d columns, with s = x + residual, g = w dy and dh the gradient that
// reaches s past the norm:
//   RMS:    u = s r,         r = 1 / sqrt(mean s^2 + eps),
//           dx = r (g - u mean(g u)) + dh
//   layer:  u = (s - mu) r,  r = 1 / sqrt(mean (s - mu)^2 + eps),
//           dx = r (g - mean g - u mean(g u)) + dh
//   dweight = sum over the rows of dy u,  dbias = sum over the rows of dy
// mean(g u) is r mean(g s) (r mean(g (s - mu))), so the RMS form needs one
// reduction over a row; the layer form two, or one about a pivot (below).
//
// Kernels
//   norm_backward_stream_kernel   many rows of more than 512 columns (layer form
//       256): blocks that stay sum their rows' dweight and dbias in registers
//       and write one partial row of each; column_sum_kernel adds those up.
//       8192 x 7168 bf16 with dh (470 MB): RMS 73.9 us, 6.36 TB/s, 95% of the copy
//       rate; layer form 77.1 us, 91%; 4096 x 7168 fp32 RMS 72.7 us, 97%; 57344 x
//       1024 75.3 and 76.4.  What is lost is the launch of the sums of the partial
//       rows and the start of the copies.
//   norm_backward_warps_kernel    many shorter rows, the same with a warp a row
//   norm_backward_rows_kernel, norm_backward_columns_kernel   few rows: dx and
//       the rows' statistics, then the sums from a second reading, which comes
//       from L2.  777 x 1000 fp32 layer form 6.8 us: two launches.
//   norm_backward_wide_kernel     rows of more than 16384 columns
// Every sum is taken in an order that the sizes, the types and the given arguments
// decide, so results depend neither on timing nor on the device.
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

// Wait until at most `left` (< kMaxStages) of the thread's groups of copies are
// under way.
constexpr int kMaxStages = 4, kStreamStages = 4;
__device__ __forceinline__ void wait_copies(int left) {
  if (left == 0)
    asm volatile("cp.async.wait_group 0;" ::: "memory");
  else if (left == 1)
    asm volatile("cp.async.wait_group 1;" ::: "memory");
  else if (left == 2)
    asm volatile("cp.async.wait_group 2;" ::: "memory");
  else
    asm volatile("cp.async.wait_group 3;" ::: "memory");
}

// Many short rows: a warp a row, a lane the same kP chunks of N columns of each
// of its rows.  But for single bf16 values a lane keeps the chunks of its next
// `stages` rows on their way into shared memory, where it alone reads them: no
// barrier, and no register holds what is under way.
//   dx = r g - (r mean(g u)) u + dh, and for the layer form
//   dx = r g - (r mean(g u)) u + (dh - r mean g)
// with u = s r taken first: r r mean(g s) by itself overflows for rows of values
// below 2^-64.
constexpr int kRowWarps = 8;

template <typename T, int N, int kP, bool kLayer, int kMinBlocks>
__global__ void __launch_bounds__(32 * kRowWarps, kMinBlocks)
    norm_backward_warps_kernel(const BackwardPtrs p, float eps, int d, int64_t rows, int stages) {
  using C = Chunk<T, N>;
  using V = Vec<N>;
  extern __shared__ uint4 ring_bytes[];
  C* const ring = reinterpret_cast<C*>(ring_bytes);
  constexpr bool kRing = sizeof(C) >= 4;
  pdl_wait();
  const int lane = threadIdx.x & 31, team = threadIdx.x / 32;
  const int chunks = d / N;
  const C* const w = static_cast<const C*>(p.w);
  const float inv_d = 1.0f / static_cast<float>(d);
  const int64_t first = static_cast<int64_t>(blockIdx.x) * kRowWarps + team;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * kRowWarps;
  V dw[kP], db[kLayer ? kP : 1];
#pragma unroll
  for (int j = 0; j < kP; ++j) {
    dw[j] = all<N>(0.0f);
    if constexpr (kLayer) db[j] = all<N>(0.0f);
  }
  // a stage: dy, x, then the residual and dh where there are any
  const bool with_r = p.r, with_dh = p.dh && p.dx;
  const int tensors = 2 + with_r + with_dh;
  const int pitch = kP * 32 * kRowWarps;  // chunks of a tensor in a stage
  const int64_t step = stride * chunks;
  int64_t ahead = first * chunks + lane;  // of the thread's first chunk to fetch
  int64_t left = rows - first;           // rows from there on
  uint32_t fill = smem_u32(ring + threadIdx.x);
  const uint32_t begin = fill, stage_bytes = tensors * pitch * sizeof(C);
  const uint32_t end = begin + stages * stage_bytes;
  auto fetch = [&]() {
    if (left > 0) {
      uint32_t to = fill;
      auto one = [&](const void* from) {
        const C* src = static_cast<const C*>(from) + ahead;
#pragma unroll
        for (int j = 0; j < kP; ++j)
          if (lane + 32 * j < chunks)
            copy_async<sizeof(C)>(to + j * 32 * kRowWarps * static_cast<uint32_t>(sizeof(C)),
                                  src + 32 * j);
        to += pitch * sizeof(C);
      };
      one(p.dy);
      one(p.a);
      if (with_r) one(p.r);
      if (with_dh) one(p.dh);
    }
    commit_copies();
    ahead += step;
    left -= stride;
    fill += stage_bytes;
    if (fill == end) fill = begin;
  };
  if constexpr (kRing)
    for (int i = 0; i < stages; ++i) fetch();

  int stage = 0;
  for (int64_t row = first; row < rows; row += stride) {
    const int64_t base = row * chunks + lane;
    if constexpr (kRing) wait_copies(stages - 1);
    const C* from = ring + stage * tensors * pitch + threadIdx.x;
    // chunk j of tensor t; the last of them is dh
    auto chunk = [&](const void* global, int t, int j) {
      if constexpr (kRing)
        return from[t * pitch + j * 32 * kRowWarps];
      else
        return static_cast<const C*>(global)[base + 32 * j];
    };
    auto sum = [&](int j) {
      V s = unpack(chunk(p.a, 1, j));
      if (with_r) s = add(s, unpack(chunk(p.r, 2, j)));
      return s;
    };
    float mu = 0.0f, mg = 0.0f;
    if constexpr (kLayer) {
      V a = all<N>(0.0f), b = a;
#pragma unroll
      for (int j = 0; j < kP; ++j) {
        if (lane + 32 * j >= chunks) continue;
        a = add(a, sum(j));
        b = fma(unpack(chunk(p.dy, 0, j)), unpack(w[lane + 32 * j]), b);
      }
      const float2 t = warp_sum(total(a), total(b));
      mu = t.x * inv_d;
      mg = t.y * inv_d;
    }
    const V vmu = all<N>(-mu);
    V a = all<N>(0.0f), b = a;
#pragma unroll
    for (int j = 0; j < kP; ++j) {
      if (lane + 32 * j >= chunks) continue;
      V s = sum(j);
      if constexpr (kLayer) s = add(s, vmu);
      a = fma(s, s, a);
      b = fma(mul(unpack(chunk(p.dy, 0, j)), unpack(w[lane + 32 * j])), s, b);
    }
    const float2 t = warp_sum(total(a), total(b));
    const float rs = rsqrtf(t.x * inv_d + eps);
    const float c = -rs * (rs * (t.y * inv_d));
    const V vrs = all<N>(rs), vc = all<N>(c), vg = all<N>(-rs * mg);
#pragma unroll
    for (int j = 0; j < kP; ++j) {
      if (lane + 32 * j >= chunks) continue;
      V s = sum(j);
      if constexpr (kLayer) s = add(s, vmu);
      const V y = unpack(chunk(p.dy, 0, j));
      s = mul(s, vrs);
      dw[j] = fma(y, s, dw[j]);
      if constexpr (kLayer) db[j] = add(db[j], y);
      if (p.dx) {
        V v = with_dh ? unpack(chunk(p.dh, tensors - 1, j)) : all<N>(0.0f);
        if constexpr (kLayer) v = add(v, vg);
        v = fma(mul(y, unpack(w[lane + 32 * j])), vrs, fma(s, vc, v));
        C out;
        pack(v, out);
        static_cast<C*>(p.dx)[base + 32 * j] = out;
      }
    }
    if constexpr (kRing) {
      fetch();
      if (++stage == stages) stage = 0;
    }
  }
  pdl_release();  // the sum of the partial rows waits for them itself

  // the block's partial rows, its warps' sums in their order
  auto write = [&](float* to, const V* acc) {
    if (!to) return;
    V* const sum = reinterpret_cast<V*>(ring_bytes);
    for (int turn = 0; turn < kRowWarps; ++turn) {
      __syncthreads();
      if (turn != team) continue;
#pragma unroll
      for (int j = 0; j < kP; ++j)
        sum[32 * j + lane] = turn ? add(sum[32 * j + lane], acc[j]) : acc[j];
    }
    __syncthreads();
    to += static_cast<int64_t>(blockIdx.x) * d;
    for (int i = threadIdx.x; i < chunks; i += blockDim.x) reinterpret_cast<V*>(to)[i] = sum[i];
    __syncthreads();
  };
  write(p.pw, dw);
  if constexpr (kLayer) write(p.pb, db);
}

// Sums of four values over a block of at most 16 warps, as block_sum takes two;
// `part` of 64 values.
__device__ __forceinline__ float4 block_sum4(float v0, float v1, float v2, float v3,
                                             float* part) {
  const int lane = threadIdx.x & 31;
  const bool high = lane & 16, odd = lane & 8;
  float a = high ? v2 : v0, b = high ? v3 : v1;
  a += __shfl_xor_sync(0xffffffffu, high ? v0 : v2, 16);
  b += __shfl_xor_sync(0xffffffffu, high ? v1 : v3, 16);
  float v = odd ? b : a;
  v += __shfl_xor_sync(0xffffffffu, odd ? a : b, 8);
#pragma unroll
  for (int o = 4; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  // value k of warp i at 4 i + k
  if ((lane & 7) == 0) part[threadIdx.x >> 3] = v;
  __syncthreads();
  const int sums = blockDim.x / 8;
  v = lane < sums ? part[lane] : 0.0f;
  if (lane + 32 < sums) v += part[lane + 32];
#pragma unroll
  for (int o = 4; o <= 16; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return make_float4(__shfl_sync(0xffffffffu, v, 0), __shfl_sync(0xffffffffu, v, 1),
                     __shfl_sync(0xffffffffu, v, 2), __shfl_sync(0xffffffffu, v, 3));
}

// Many rows, a block a row at a time, a thread the same kP 16-byte chunks of each
// (kFull: all of them in the row).  One thread keeps bulk copies
// of the next rows under way into a ring of shared memory; a stage is free again
// at the barrier of its row's sums, as every thread then holds its chunks of it, x
// as fp32 values.  (bf16, 8192 x 7168: unpacked for each use 79.6 us, two rows at a
// time so that they share a barrier 77.9; layer form 102.3 and 96.1.)
//
// The layer form takes its sums about a pivot P, the mean of the row's first 32
// values:
//   mean(s - P) = m, mu = P + m, mean (s - mu)^2 = mean (s - P)^2 - m^2,
//   sum g (s - mu) = sum g (s - P) - m sum g
// which needs one reduction (77.8 us, with four rows a ring) and not two (83.4).
// Taking m^2 off multiplies the roundings of the mean square by (v + m^2) / v, v the
// variance: by 1.03 for rows like one another's values, whose m is a fifth of a
// standard deviation, but by up to d / 32 where the first values are unlike the rest.
// And the roundings of the sum of s - P, of values of m where most of the row lies there,
// are those of m.  So where m^2 exceeds v / 4 (one row in 200 of like values) the block
// takes the sums once more, about mu.  (s - P is off by half an ulp of at most sqrt(d / 32)
// + |s - mu| / sigma standard deviations.)
//
// kShift: rows that are not whole chunks begin inside one.  A block's rows are a
// multiple of N apart, so that all of them begin at the same value of their first
// chunk: the block holds the weights and sums for that shift, copies the chunks that
// the row reaches into, and clears what there belongs to the rows beside it.
// (8192 x 7001 bf16 RMS 77.8 us, layer form 104; from two readings of single values
// 246 and 264.)
template <typename T, int kP, bool kLayer, bool kRes, bool kFull, bool kShift>
__global__ void __launch_bounds__(512, 1)
    norm_backward_stream_kernel(const BackwardPtrs p, float eps, int d, int64_t rows, int stages,
                                int* status) {
  constexpr int N = 16 / sizeof(T);
  using C = Chunk<T, N>;
  using V = Vec<N>;
  extern __shared__ uint4 ring_bytes[];
  __shared__ uint64_t full[kStreamStages];
  __shared__ int aborted;
  __shared__ float part[2][64];  // of sums in turn: a barrier then separates the uses of each
  pdl_wait();
  const int tid = threadIdx.x, threads = blockDim.x;
  // values before the row in its first chunk, the chunks it reaches into, and the
  // most that any row does
  const int shift = kShift ? static_cast<int>(blockIdx.x * static_cast<int64_t>(d) % N) : 0;
  const int chunks = kShift ? (shift + d + N - 1) / N : d / N;
  const int pitch = kShift ? span_chunks<N>(d) : chunks;
  auto chunk_of = [&](int64_t row) { return kShift ? row * d / N : row * chunks; };
  // the last row's last chunk may reach past the tensor's end
  auto cut = [&](int64_t row) { return kShift && row == rows - 1 && rows * d % N; };
  // the values of chunk j that are the row's, where they are not all
  auto edge = [&](int j, int& lo, int& hi) {
    const int c = tid + j * threads;
    lo = c ? 0 : shift, hi = min(N, shift + d - c * N);
    return kShift && hi - lo < N;
  };
  const float inv_d = 1.0f / static_cast<float>(d);
  const bool with_dh = p.dh && p.dx;
  const int tensors = 2 + kRes + with_dh;
  if (tid == 0) {
    aborted = 0;
    for (int i = 0; i < stages; ++i) mbar_init(smem_u32(&full[i]), 1);
    fence_mbarrier_init();
  }
  __syncthreads();
  const uint64_t policy = l2_policy_evict_first();
  auto fetch = [&](int64_t row, int stage) {
    const uint32_t bar = smem_u32(&full[stage]);
    uint32_t to = smem_u32(ring_bytes + stage * tensors * pitch);
    const uint32_t bytes = (chunks - cut(row)) * 16u;
    const int64_t at = chunk_of(row);
    mbar_arrive_expect_tx(bar, bytes * tensors);
    auto one = [&](const void* from) {
      bulk_load(to, static_cast<const C*>(from) + at, bytes, bar, policy);
      to += pitch * 16u;
    };
    one(p.dy);
    one(p.a);
    if (kRes) one(p.r);
    if (with_dh) one(p.dh);
  };
  int64_t row = blockIdx.x;
  if (tid == 0)
    for (int i = 0; i < stages; ++i) {
      const int64_t at = row + static_cast<int64_t>(i) * gridDim.x;
      if (at < rows) fetch(at, i);
    }

  auto has = [&](int j) { return kFull || tid + j * threads < chunks; };
  C cw[kP];
  V dw[kP], db[kLayer ? kP : 1];
#pragma unroll
  for (int j = 0; j < kP; ++j) {
    dw[j] = all<N>(0.0f);
    if constexpr (kLayer) db[j] = all<N>(0.0f);
    if (!has(j)) continue;
    if constexpr (kShift)
      cw[j] = gather<T, N>(static_cast<const T*>(p.w), (tid + j * threads) * N - shift, d);
    else
      cw[j] = static_cast<const C*>(p.w)[tid + j * threads];
  }
  int stage = 0, turn = 0;
  uint32_t parity = 0;
  for (; row < rows; row += gridDim.x) {
    if (!__all_sync(0xffffffffu,
                    mbar_wait_bounded(smem_u32(&full[stage]), parity, &aborted, status)))
      break;
    C cy[kP], ch[kP];
    V vs[kP], vy[kLayer ? 1 : kP];
    C* const base = reinterpret_cast<C*>(ring_bytes) + stage * tensors * pitch;
    if (cut(row)) {
      const int have = (chunks - 1) * N;
      const int64_t at = rows * d - (shift + d - have) + tid;
      auto one = [&](const void* src, int t) {
        if (tid < shift + d - have)
          reinterpret_cast<T*>(base + t * pitch)[have + tid] = static_cast<const T*>(src)[at];
      };
      one(p.dy, 0);
      one(p.a, 1);
      if (kRes) one(p.r, 2);
      if (with_dh) one(p.dh, tensors - 1);
      __syncthreads();
    }
    float pivot = 0.0f;
    if constexpr (kLayer) {
      const T* v = reinterpret_cast<const T*>(base + pitch) + shift + (tid & 31);
      pivot = static_cast<float>(*v);
      if constexpr (kRes) pivot += static_cast<float>(v[pitch * N]);
#pragma unroll
      for (int o = 16; o; o >>= 1) pivot += __shfl_xor_sync(0xffffffffu, pivot, o);
      pivot *= 1.0f / 32;
    }
    const C* from = base + tid;
#pragma unroll
    for (int j = 0; j < kP; ++j) {
      if (!has(j)) continue;
      const C* at = from + j * threads;
      cy[j] = *at;
      vs[j] = unpack(at[pitch]);
      if constexpr (kRes) vs[j] = add(vs[j], unpack(at[2 * pitch]));
      if (with_dh) ch[j] = at[(tensors - 1) * pitch];
      int lo, hi;
      if (edge(j, lo, hi)) {
        clip(cy[j], lo, hi);
        clip(vs[j], lo, hi, pivot);  // 0 to the sums
      }
      if constexpr (!kLayer) vy[j] = unpack(cy[j]);
    }
    auto dy = [&](int j) {
      if constexpr (kLayer)
        return unpack(cy[j]);
      else
        return vy[j];
    };
    auto refill = [&]() {  // after the first barrier that follows the loads
      const int64_t next = row + static_cast<int64_t>(stages) * gridDim.x;
      if (tid == 0 && next < rows) fetch(next, stage);
    };
    float mg = 0.0f, ms, gs;
    if constexpr (kLayer) {
      // vs, the row, less `at`, and the means of it, of its squares, of g and of g vs
      auto sums = [&](float at) {
        const V np = all<N>(-at);
        V m = all<N>(0.0f), g = m, p = m, q = m;
#pragma unroll
        for (int j = 0; j < kP; ++j) {
          if (!has(j)) continue;
          const V y = mul(dy(j), unpack(cw[j]));
          vs[j] = add(vs[j], np);
          m = add(m, vs[j]);
          p = fma(vs[j], vs[j], p);
          g = add(g, y);
          q = fma(y, vs[j], q);
        }
        return block_sum4(total(p), total(q), total(m), total(g), part[turn]);
      };
      float4 t = sums(pivot);
      refill();
      float mu = t.z * inv_d;
      ms = fmaf(-mu, mu, t.x * inv_d);
      if (4.0f * mu * mu > ms) {  // the same in all threads
        turn ^= 1;
        // what is not the row's takes mu, for 0 to the sums
#pragma unroll
        for (int j = 0; j < kP; ++j) {
          int lo, hi;
          if (has(j) && edge(j, lo, hi)) clip(vs[j], lo, hi, mu);
        }
        t = sums(mu);
        mu = t.z * inv_d;
        ms = fmaf(-mu, mu, t.x * inv_d);
      }
      mg = t.w * inv_d;
      gs = fmaf(-mu, t.w, t.y);
      const V nm = all<N>(-mu);
#pragma unroll
      for (int j = 0; j < kP; ++j)
        if (has(j)) vs[j] = add(vs[j], nm);
    } else {
      V a = all<N>(0.0f), b = a;
#pragma unroll
      for (int j = 0; j < kP; ++j) {
        if (!has(j)) continue;
        a = fma(vs[j], vs[j], a);
        b = fma(mul(dy(j), unpack(cw[j])), vs[j], b);
      }
      const float2 t = block_sum(total(a), total(b), part[turn]);
      ms = t.x * inv_d;
      gs = t.y;
    }
    turn ^= 1;
    if constexpr (!kLayer) refill();
    const float rs = rsqrtf(ms + eps);
    const V vrs = all<N>(rs), c = all<N>(-rs * (rs * (gs * inv_d))), vg = all<N>(-rs * mg);
#pragma unroll
    for (int j = 0; j < kP; ++j) {
      if (!has(j)) continue;
      const V y = dy(j), s = mul(vs[j], vrs);
      dw[j] = fma(y, s, dw[j]);
      if constexpr (kLayer) db[j] = add(db[j], y);
      if (p.dx) {
        V v = with_dh ? unpack(ch[j]) : all<N>(0.0f);
        if constexpr (kLayer) v = add(v, vg);
        v = fma(mul(y, unpack(cw[j])), vrs, fma(s, c, v));
        C* const to = static_cast<C*>(p.dx) + chunk_of(row) + tid + j * threads;
        int lo, hi;
        if (edge(j, lo, hi)) {
          store_part(reinterpret_cast<T*>(to), v, lo, hi);
        } else {
          C out;
          pack(v, out);
          *to = out;
        }
      }
    }
    if (++stage == stages) {
      stage = 0;
      parity ^= 1;
    }
  }
  // After a wait that expired: no copy of the block's may be under way at its end.
  if (tid == 0)
    for (int i = 0; i < stages && row < rows; ++i, row += gridDim.x) {
      int own = 0;
      if (!mbar_wait_bounded(smem_u32(&full[stage]), parity, &own, status)) break;
      if (++stage == stages) {
        stage = 0;
        parity ^= 1;
      }
    }
  pdl_release();  // the sum of the partial rows waits for them itself
#pragma unroll
  for (int j = 0; j < kP; ++j) {
    if (!has(j)) continue;
    const int64_t at = static_cast<int64_t>(blockIdx.x) * d;
    const int i = tid + j * threads;
    auto write = [&](float* to, const V& v) {
      int lo = 0, hi = N;
      edge(j, lo, hi);
      if constexpr (kShift)
        store_part(to + at + i * N - shift, v, lo, hi);
      else
        reinterpret_cast<V*>(to + at)[i] = v;
    };
    if (p.pw) write(p.pw, dw[j]);
    if constexpr (kLayer)
      if (p.pb) write(p.pb, db[j]);
  }
}

// dx and the rows' statistics of tensors that stay in L2, where dweight and
// dbias are summed from a second reading (norm_backward_columns_kernel): no
// partial rows, and every row under way at once.  A block a row, or (kWarpRow) a
// warp a row; a thread kP chunks of it, loaded together and kept.
template <typename T, int N, int kP, bool kLayer, bool kWarpRow, int kMaxThreads>
__global__ void __launch_bounds__(kMaxThreads)
    norm_backward_rows_kernel(const BackwardPtrs p, float eps, int d, int64_t rows) {
  using C = Chunk<T, N>;
  using V = Vec<N>;
  __shared__ float part[64], part_mean[64];
  pdl_wait();
  const int threads = kWarpRow ? 32 : blockDim.x;
  const int tid = kWarpRow ? threadIdx.x & 31 : threadIdx.x;
  const int64_t row =
      kWarpRow ? static_cast<int64_t>(blockIdx.x) * kRowWarps + threadIdx.x / 32 : blockIdx.x;
  if (kWarpRow && row >= rows) return;
  const int chunks = d / N;
  const float inv_d = 1.0f / static_cast<float>(d);
  const int64_t base = row * chunks;
  C cy[kP], cs[kP], cr[kP], ch[kP], cw[kP];
#pragma unroll
  for (int j = 0; j < kP; ++j) {
    const int i = tid + j * threads;
    if (i < chunks) {
      cy[j] = static_cast<const C*>(p.dy)[base + i];
      cs[j] = static_cast<const C*>(p.a)[base + i];
      cw[j] = static_cast<const C*>(p.w)[i];
      if (p.r) cr[j] = static_cast<const C*>(p.r)[base + i];
      if (p.dh && p.dx) ch[j] = static_cast<const C*>(p.dh)[base + i];
    }
  }
  V s[kP], g[kP];
  V a = all<N>(0.0f), b = a;
#pragma unroll
  for (int j = 0; j < kP; ++j) {
    if (tid + j * threads < chunks) {
      s[j] = unpack(cs[j]);
      if (p.r) s[j] = add(s[j], unpack(cr[j]));
      g[j] = mul(unpack(cy[j]), unpack(cw[j]));
    } else {
      s[j] = g[j] = all<N>(0.0f);
    }
    if constexpr (kLayer) {
      a = add(a, s[j]);
      b = add(b, g[j]);
    }
  }
  float mu = 0.0f, mg = 0.0f;
  if constexpr (kLayer) {
    const float2 t = kWarpRow ? warp_sum(total(a), total(b)) : block_sum(total(a), total(b), part_mean);
    mu = t.x * inv_d;
    mg = t.y * inv_d;
    a = b = all<N>(0.0f);
  }
#pragma unroll
  for (int j = 0; j < kP; ++j) {
    if constexpr (kLayer)
      if (tid + j * threads < chunks) s[j] = add(s[j], all<N>(-mu));
    a = fma(s[j], s[j], a);
    b = fma(g[j], s[j], b);
  }
  const float2 t = kWarpRow ? warp_sum(total(a), total(b)) : block_sum(total(a), total(b), part);
  const float rs = rsqrtf(t.x * inv_d + eps);
  const float c = -rs * (rs * (t.y * inv_d));
  if (p.stats && tid == 0) p.stats[row] = make_float2(mu, rs);
  if (!p.dx) return;
#pragma unroll
  for (int j = 0; j < kP; ++j) {
    const int i = tid + j * threads;
    if (i >= chunks) continue;
    V v = p.dh ? unpack(ch[j]) : all<N>(0.0f);
    if constexpr (kLayer) v = add(v, all<N>(-rs * mg));
    C out;
    pack(fma(g[j], all<N>(rs), fma(mul(s[j], all<N>(rs)), all<N>(c), v)), out);
    static_cast<C*>(p.dx)[base + i] = out;
  }
}

// Sums of two values over a block of 1024 threads.
__device__ __forceinline__ float2 wide_sum(float x, float y, float2 (*part)[32], int buf) {
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    x += __shfl_xor_sync(0xffffffffu, x, o);
    y += __shfl_xor_sync(0xffffffffu, y, o);
  }
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
  return make_float2(x, y);
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
    const float2 t = wide_sum(x0, x1, part, 0);
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
  const float2 t = wide_sum(x0, x1, part, 1);
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

// dweight and dbias from the rows and their statistics.  A cluster of eight
// blocks sums 32 N columns: a lane a chunk, the rows dealt to the blocks' warps;
// the warps' sums are added in each block, then the blocks' through distributed
// shared memory, an eighth of the columns by each.
constexpr int kColumnBlocks = 8, kColumnWarps = 8;

template <typename T, int N, bool kLayer>
__global__ void __cluster_dims__(1, kColumnBlocks, 1) __launch_bounds__(32 * kColumnWarps)
    norm_backward_columns_kernel(const BackwardPtrs p, int d, int64_t rows, float* out_w,
                                 float* out_b) {
  using C = Chunk<T, N>;
  using V = Vec<N>;
  constexpr int kCols = 32 * N;
  __shared__ __align__(16) float warps[kLayer ? 2 : 1][kColumnWarps][kCols];
  __shared__ float sums[kLayer ? 2 : 1][kCols];
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t chunks = d / N, i = static_cast<int64_t>(blockIdx.x) * 32 + lane;
  const int rank = blockIdx.y;
  V dw = all<N>(0.0f), db = dw;
  if (i < chunks) {
    constexpr int kAhead = 4, kStep = kColumnBlocks * kColumnWarps;
    for (int64_t row = rank * kColumnWarps + warp; row < rows; row += kAhead * kStep) {
      C y[kAhead], s[kAhead], r[kAhead];
      float2 st[kAhead];
#pragma unroll
      for (int a = 0; a < kAhead; ++a) {
        const int64_t at = row + a * kStep;
        if (at < rows) {
          y[a] = static_cast<const C*>(p.dy)[at * chunks + i];
          s[a] = static_cast<const C*>(p.a)[at * chunks + i];
          if (p.r) r[a] = static_cast<const C*>(p.r)[at * chunks + i];
          st[a] = p.stats[at];
        }
      }
#pragma unroll
      for (int a = 0; a < kAhead; ++a) {
        if (row + a * kStep >= rows) continue;
        V u = unpack(s[a]);
        if (p.r) u = add(u, unpack(r[a]));
        if constexpr (kLayer) u = add(u, all<N>(-st[a].x));
        const V v = unpack(y[a]);
        dw = fma(v, mul(u, all<N>(st[a].y)), dw);
        if constexpr (kLayer) db = add(db, v);
      }
    }
  }
  reinterpret_cast<V*>(warps[0][warp])[lane] = dw;
  if constexpr (kLayer) reinterpret_cast<V*>(warps[1][warp])[lane] = db;
  __syncthreads();
  for (int c = threadIdx.x; c < kCols; c += 32 * kColumnWarps) {
#pragma unroll
    for (int k = 0; k < (kLayer ? 2 : 1); ++k) {
      float t = 0.0f;
#pragma unroll
      for (int w = 0; w < kColumnWarps; ++w) t += warps[k][w][c];
      sums[k][c] = t;
    }
  }
  cluster_sync_all();
  constexpr int kMine = kCols / kColumnBlocks;
  if (threadIdx.x < kMine * (kLayer ? 2 : 1)) {
    const int k = threadIdx.x / kMine, c = rank * kMine + threadIdx.x % kMine;
    const uint32_t at = smem_u32(&sums[k][c]);
    float t = 0.0f;
#pragma unroll
    for (int q = 0; q < kColumnBlocks; ++q) {
      float v;
      asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(cluster_map(at, q)) : "memory");
      t += v;
    }
    float* out = k ? out_b : out_w;
    const int64_t col = static_cast<int64_t>(blockIdx.x) * kCols + c;
    if (out && col < d) out[col] = t;
  }
  cluster_sync_all();  // no block ends while another reads its sums
}

// out[c] = the sum of `parts` rows of partials: a thread adds C neighbouring
// columns, a block's 32 warps the rows 32 apart, eight of them in flight; then
// the warps' sums are added in their order.
constexpr int kSumWarps = 32;
template <int C>
__global__ void __launch_bounds__(32 * kSumWarps)
    column_sum_kernel(const float* __restrict__ pw, const float* __restrict__ pb, int parts, int d,
                      float* __restrict__ dw, float* __restrict__ db) {
  __shared__ float sums[kSumWarps][32 * C];
  pdl_wait();
  const float* p = blockIdx.y ? pb : pw;
  float* out = blockIdx.y ? db : dw;
  if (!out) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t c = (static_cast<int64_t>(blockIdx.x) * 32 + lane) * C;
  float s[C];
#pragma unroll
  for (int k = 0; k < C; ++k) s[k] = 0.0f;
  if (c < d) {
    constexpr int kAhead = 8;
    for (int i = warp; i < parts; i += kAhead * kSumWarps) {
      Piece<float, C> v[kAhead];
#pragma unroll
      for (int a = 0; a < kAhead; ++a)
        if (i + a * kSumWarps < parts)
          v[a] = load<C>(p + static_cast<int64_t>(i + a * kSumWarps) * d + c);
#pragma unroll
      for (int a = 0; a < kAhead; ++a)
        if (i + a * kSumWarps < parts)
#pragma unroll
          for (int k = 0; k < C; ++k) s[k] += v[a].v[k];
    }
  }
#pragma unroll
  for (int k = 0; k < C; ++k) sums[warp][lane * C + k] = s[k];
  __syncthreads();
  for (int i = threadIdx.x; i < 32 * C; i += 32 * kSumWarps) {
    float t = 0.0f;
#pragma unroll
    for (int a = 0; a < kSumWarps; ++a) t += sums[a][i];
    const int64_t col = static_cast<int64_t>(blockIdx.x) * 32 * C + i;
    if (col < d) out[col] = t;
  }
}

template <typename T, int N, int kP, bool kLayer, int kMinBlocks>
cudaError_t launch_warps(const NormBackwardArgs& n, const BackwardPtrs& p, int parts,
                         cudaStream_t stream) {
  auto kernel = norm_backward_warps_kernel<T, N, kP, kLayer, kMinBlocks>;
  constexpr int kThreads = 32 * kRowWarps;
  int stages = 0;
  size_t bytes = 32 * kP * N * sizeof(float);  // the sums at the end
  if (N * sizeof(T) >= 4) {
    // as many as leave room for a second block on the SM
    const int one = (2 + (p.r ? 1 : 0) + (p.dh && p.dx ? 1 : 0)) * kP * kThreads *
                    static_cast<int>(N * sizeof(T));
    stages = 110 * 1024 / one;
    stages = stages < 1 ? 1 : stages > kMaxStages ? kMaxStages : stages;
    if (bytes < static_cast<size_t>(stages) * one) bytes = static_cast<size_t>(stages) * one;
  }
  const cudaError_t err =
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 160 * 1024);
  if (err != cudaSuccess) return err;
  return launch_pdl(kernel, dim3(static_cast<unsigned>(parts)), dim3(kThreads), bytes, stream, p,
                    n.eps, n.d, n.T, stages);
}

// Blocks of an SM that share its registers and shared memory in the stream
// kernel.  With rows of at most 512 columns a block is a warp: 16 of them where
// each has at least 8 rows (57344 x 512 layer form 45.2 us, with 8 blocks 49.3; 8192
// x 512 15.5 and 13.4).
int stream_blocks(int64_t T, int64_t d) {
  return d > 4096 ? 1 : d > 2048 ? 2 : d > 1024 ? 4 : d > 512 || T < 8 * 16 * 152 ? 8 : 16;
}

template <typename T, bool kLayer, bool kRes, bool kShift>
cudaError_t launch_stream(const NormBackwardArgs& n, const BackwardPtrs& p, int parts,
                          cudaStream_t stream) {
  constexpr int N = 16 / sizeof(T), kP = 16 / N;
  const int chunks = kShift ? span_chunks<N>(n.d) : n.d / N;
  const int threads = (chunks + 32 * kP - 1) / (32 * kP) * 32;
  auto kernel = norm_backward_stream_kernel<T, kP, kLayer, kRes, false, kShift>;
  if (!kShift && threads * kP == chunks)
    kernel = norm_backward_stream_kernel<T, kP, kLayer, kRes, !kShift, kShift>;
  const int one = (2 + kRes + (p.dh && p.dx ? 1 : 0)) * chunks * 16;
  // What is under way on an SM: 132 KB, and two rows at least where they fit (room).
  // Less leaves the memory waiting, more makes reads and writes get in each other's way
  // (8192 x 7168 RMS, of 43 KB a row, two rows 75.5 us, three 73.7, four 77.6, five 80.3;
  // 57344 x 1024, of 48 KB in eight blocks, two 75.1, three 78.8, four 81.1).  fp32 rows
  // with a residual and dh have room for one in the upper sixth of each range of
  // stream_blocks (865 to 1024 columns, 1729 to 2048, 3457 to 4096, 6913 to 8192): a
  // block then copies no row ahead (4096 x 7168 layer form 102 us, 86% of the copy rate).
  const int room = 216 * 1024 / stream_blocks(n.T, n.d) / one;
  int stages = 132 * 1024 / stream_blocks(n.T, n.d) / one;
  stages = stages < 2 ? 2 : stages > kStreamStages ? kStreamStages : stages;
  if (stages > room) stages = room;
  const cudaError_t err =
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 220 * 1024);
  if (err != cudaSuccess) return err;
  return launch_pdl(kernel, dim3(static_cast<unsigned>(parts)), dim3(threads),
                    static_cast<size_t>(stages) * one, stream, p, n.eps, n.d, n.T, stages, n.status);
}

// Statistics and dx by `rows`, and the sums over the rows, before dx is written
// where it is an input of theirs.
template <typename T, int N, bool kLayer, typename Rows>
cudaError_t two_passes(const NormBackwardArgs& n, BackwardPtrs p, cudaStream_t stream, Rows rows) {
  const bool sums = n.dw || n.db;
  if (!sums) return rows(p);
  const bool in_place = p.dx && (p.dx == p.dy || p.dx == p.a || p.dx == p.r);
  p.stats = n.stats;
  if (in_place) p.dx = nullptr;
  cudaError_t err = rows(p);
  if (err != cudaSuccess) return err;
  const int64_t chunks = n.d / N;
  err = launch_pdl(norm_backward_columns_kernel<T, N, kLayer>,
                   dim3(static_cast<unsigned>((chunks + 31) / 32), kColumnBlocks),
                   dim3(32 * kColumnWarps), 0, stream, p, n.d, n.T, n.dw, n.db);
  if (err != cudaSuccess || !in_place) return err;
  p.stats = nullptr;
  p.dx = n.dx;
  return rows(p);
}

// Two readings or partial rows.  A second reading of few rows that stay in L2
// is the faster (us with it / with partial rows, bf16: layer form, 1100 x 2048
// 9.0 / 10.5, 1100 x 4096 13.0 / 14.1, 1500 x 2048 10.6 / 11.8, 1500 x 4096 16.0 / 16.0;
// RMS 700 x 4096 8.4 / 9.6, 1000 x 2048 7.7 / 7.7), but for short rows, a warp each
// (1000 x 256 6.3 / 5.4).  With more of them it loses (RMS 700 x 7168 12.5 / 11.0,
// 1000 x 4096 10.7 / 9.8; layer form 2000 x 1024 10.7 / 10.0, 2000 x 4096 20.4 / 17.6,
// fp32 1500 x 1024 9.6 / 8.0): a warp of the second launch has more rows, and the
// tensors leave L2.
// Rows of no whole chunks take more of them (2000 x 1001 layer form 10.9 / 13.6, RMS
// 10.1 / 11.1, 3000 x 1001 14.5 / 14.2 and 13.4 / 11.7).
template <typename T, int N, bool kLayer>
constexpr int64_t kTwoPassRows = N * sizeof(T) < 16    ? (kLayer ? 3000 : 2048)
                                 : kLayer && sizeof(T) == 2 ? 1536
                                                            : 1024;
template <bool kLayer>
constexpr int64_t kTwoPassBytes = (kLayer ? 24ll : 13ll) << 20;
constexpr int kShort = 256;

template <typename T, int N, bool kLayer>
cudaError_t dispatch(const NormBackwardArgs& n, cudaStream_t stream) {
  const bool sums = n.dw || n.db;
  BackwardPtrs p = {n.a, n.r, n.w, n.dy, n.dh, n.dx, nullptr, nullptr, nullptr};
  if (n.d > 16384)
    return two_passes<T, N, kLayer>(n, p, stream, [&](const BackwardPtrs& q) {
      constexpr int W = N == 2 ? 1 : N;  // a Piece is one value or 16 bytes
      return launch_pdl(norm_backward_wide_kernel<T, W, kLayer>, dim3(static_cast<unsigned>(n.T)),
                        dim3(1024), 0, stream, q, n.eps, n.d);
    });
  constexpr bool kShift = N * sizeof(T) < 16;
  const bool few = n.T <= (n.d <= kShort ? 256 : kTwoPassRows<T, N, kLayer>) &&
                   2 * n.T * n.d * static_cast<int64_t>(sizeof(T)) <= kTwoPassBytes<kLayer>;
  // rows of no whole chunks are streamed up to the kernel's 512 threads
  const int most_d = kShift ? 8192 - 2 * 16 / static_cast<int>(sizeof(T)) : 8192;
  if (!sums || few || n.d > most_d)
    return two_passes<T, N, kLayer>(n, p, stream, [&](const BackwardPtrs& q) {
      // threads of a row with at most Q values each
      auto threads = [&](int Q) { return dim3((n.d + 32 * Q - 1) / (32 * Q) * 32); };
      const dim3 rows(static_cast<unsigned>(n.T));
      if (n.d <= kShort)
        return launch_pdl(norm_backward_rows_kernel<T, N, 8 / N, kLayer, true, 32 * kRowWarps>,
                          dim3(static_cast<unsigned>((n.T + kRowWarps - 1) / kRowWarps)),
                          dim3(32 * kRowWarps), 0, stream, q, n.eps, n.d, n.T);
      if (n.d <= 8192)
        return launch_pdl(norm_backward_rows_kernel<T, N, 8 / N, kLayer, false, 1024>, rows,
                          threads(8), 0, stream, q, n.eps, n.d, n.T);
      return launch_pdl(norm_backward_rows_kernel<T, N, 16 / N, kLayer, false, 1024>, rows,
                        threads(16), 0, stream, q, n.eps, n.d, n.T);
    });
  // A block's rows from bulk copies, or a warp a row (bf16 RMS, 8192 x 512 11.2 and
  // 10.6 us, 4096 x 1024 11.1 / 10.4, 8192 x 1024 14.2 / 13.9, 16384 x 1024 21.5 / 30,
  // 57344 x 1024 75 / 84; layer form 8192 x 512 13.4 / 23).  Of short rows a block has
  // four at least: fewer make more partial rows than pay (2500 x 512 10.3 and 9.2 us).
  const bool streamed =
      kLayer || kShift ? n.d > kShort
             : n.d > 1024 ||
                   (n.d > 512 && n.T * n.d * static_cast<int64_t>(sizeof(T)) > 16 << 20);
  const int64_t teams = streamed ? (n.T + 3) / 4 : (n.T + kRowWarps - 1) / kRowWarps;
  const int64_t most = streamed ? 152 * stream_blocks(n.T, n.d) : kNormParts;
  int parts = static_cast<int>(teams < most ? teams : most);
  if (kShift && streamed) parts = (parts + 7) / 8 * 8;  // `most` is a multiple of 8
  p.pw = n.dw ? n.partials : nullptr;
  p.pb = n.db ? n.partials + static_cast<int64_t>(parts) * n.d : nullptr;
  cudaError_t err = cudaSuccess;
  if (n.d <= kShort) {
    err = launch_warps<T, N, 8 / N, kLayer, 2>(n, p, parts, stream);
  } else if (!streamed) {
    if constexpr (!kShift && !kLayer) err = launch_warps<T, N, 32 / N, false, 1>(n, p, parts, stream);
  } else {
    err = n.r ? launch_stream<T, kLayer, true, kShift>(n, p, parts, stream)
              : launch_stream<T, kLayer, false, kShift>(n, p, parts, stream);
  }
  if (err != cudaSuccess) return err;
  const float *pw = p.pw, *pb = p.pb;
  // A thread sums one column or four: with few columns more blocks share the work
  // (bf16 layer form, 8192 x 512 2.6 us less with one, 57344 x 1024 3.1), with many
  // the loads are wide (8192 x 7168 3 us less with four).
  constexpr int kWide = N >= 4 ? 4 : 1;
  const int C = n.d > 2048 ? kWide : 1;
  const dim3 grid(static_cast<unsigned>((n.d + 32 * C - 1) / (32 * C)), n.db ? 2 : 1);
  return launch_pdl(C == 1 ? column_sum_kernel<1> : column_sum_kernel<kWide>, grid,
                    dim3(32 * kSumWarps), 0, stream, pw, pb, parts, n.d, n.dw, n.db);
}

template <typename T, int N>
cudaError_t dispatch_kind(const NormBackwardArgs& n, cudaStream_t stream) {
  return n.layer ? dispatch<T, N, true>(n, stream) : dispatch<T, N, false>(n, stream);
}

}  // namespace

int64_t norm_partial_floats(int64_t T, int64_t d) {
  if (d > 8192) return 0;  // read twice
  const int64_t blocks = 152 * stream_blocks(T, d), most = blocks < kNormParts ? kNormParts : blocks;
  return 2 * d * (T < most ? T : most);
}

cudaError_t launch_norm_backward(const NormBackwardArgs& n, cudaStream_t stream) {
  if (n.bf16)
    return n.d % 8 == 0   ? dispatch_kind<__nv_bfloat16, 8>(n, stream)
           : n.d % 2 == 0 ? dispatch_kind<__nv_bfloat16, 2>(n, stream)
                          : dispatch_kind<__nv_bfloat16, 1>(n, stream);
  return n.d % 4 == 0 ? dispatch_kind<float, 4>(n, stream) : dispatch_kind<float, 1>(n, stream);
}

}  // namespace fgs
