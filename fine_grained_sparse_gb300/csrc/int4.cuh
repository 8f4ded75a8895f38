// What the two kernels for 4-bit weights share: the packed records, the
// conversions of x to f16, and the lists of the groups that have rows.
#pragma once

#include "common.cuh"
#include "internal.h"

namespace fgs {

constexpr int kChunk = 128;       // columns of one packed record
constexpr int kBlockRows = 16;    // rows of one packed record
constexpr int kCodeBytes = kChunk * kBlockRows / 2;

__host__ __device__ constexpr int record_bytes(int group) {
  return kCodeBytes + kBlockRows * (kChunk / group) * 2;
}

// Eight E4M3 codes to four f16 pairs (exact).
__device__ __forceinline__ uint4 e4m3x8_to_f16(uint2 v) {
  uint4 o;
  asm("{\n\t.reg .b16 a, b, c, d;\n\tmov.b32 {a, b}, %4;\n\tmov.b32 {c, d}, %5;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t"
      "cvt.rn.f16x2.e4m3x2 %2, c;\n\tcvt.rn.f16x2.e4m3x2 %3, d;\n\t}"
      : "=r"(o.x), "=r"(o.y), "=r"(o.z), "=r"(o.w)
      : "r"(v.x), "r"(v.y));
  return o;
}

// Eight bf16 values per lane of a half warp (128 columns) to f16, scaled by
// 2^(141 - e) where e is the biased exponent of the largest of the 128.  An
// infinity or NaN counts as the largest finite value, and maxima below 2^-112
// are left small.
__device__ __forceinline__ uint4 bf16x8_to_f16(uint4 v, uint32_t& e) {
  uint32_t w[4] = {v.x, v.y, v.z, v.w}, m = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) m = __vmaxu2(m, w[i] & 0x7fff7fffu);
#pragma unroll
  for (int o = 8; o; o >>= 1) m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, o));
  m = max(m & 0xffffu, m >> 16);
  e = min(max(m >> 7, 15u), 254u);
  const float up = __uint_as_float((268u - e) << 23);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float lo = __uint_as_float(w[i] << 16) * up;
    const float hi = __uint_as_float(w[i] & 0xffff0000u) * up;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(hi), "f"(lo));
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

// Division of 32-bit numbers by one known to the host, as a product with
// inv = ceil(2^64 / d): exact for every 32-bit x.  (A launch of a few
// microseconds notices the divisions of its beginning.)
struct Divisor {
  uint32_t d;
  uint64_t inv;
};
inline Divisor divisor(uint32_t d) { return {d, d > 1 ? ~0ull / d + 1 : 0}; }
__device__ __forceinline__ uint32_t divide(uint32_t x, const Divisor& by) {
  if (by.d == 1) return x;
  const uint64_t high = static_cast<uint64_t>(x) * static_cast<uint32_t>(by.inv >> 32);
  const uint64_t low = static_cast<uint64_t>(x) * static_cast<uint32_t>(by.inv);
  return static_cast<uint32_t>((high + (low >> 32)) >> 32);
}

// What waits for the end of the kernel before this one: nothing, a tile's x,
// or its weights (and routing) too.
enum { kWaitNone = 0, kWaitX = 1, kWaitWeights = 2 };

struct Int4Launch {
  Int4Segment seg[2];
  int nseg;
  int most;    // gemv: groups of more rows are left to gemm; gemm: those of no more to gemv
  int wait;    // kWait...
  int cap[2];  // gemv: tokens of a tile
  Divisor chunks[2], ctas;  // gemv: seg[i].chunks, the CTAs
  int smem;    // bytes of shared memory
  int* status; // device status word; null: the library's
};
cudaError_t launch_gemv_int4(const Int4Launch& p, bool swiglu, int group, int num_sms,
                             cudaStream_t stream);
cudaError_t launch_gemm_int4(const Int4Launch& p, bool swiglu, int group, int num_sms,
                             cudaStream_t stream);

// Over the groups that have work (groups of the second segment numbered
// after the first's): the cost before each [groups + 1] and its number; and
// the first row of every group with explicit rows [groups + 1].
constexpr int kMaxGroups = 1024 + 8;
struct GroupLists {
  int64_t* before;
  int32_t* first;
  uint16_t* number;
};
__host__ __device__ inline int group_list_bytes(int groups) { return 14 * (groups + 1); }
__device__ __forceinline__ GroupLists group_lists(int64_t* at, int groups) {
  GroupLists l;
  l.before = at;
  l.first = reinterpret_cast<int32_t*>(at + groups + 1);
  l.number = reinterpret_cast<uint16_t*>(l.first + groups + 1);
  return l;
}

struct GroupPlan {
  int present;    // groups with work
  int64_t total;  // their cost
};

// Fills the lists, all threads of the block.  cost(segment, rows): of one
// group, 0 if it has no work here; with(total) runs in every thread once the
// total is known; place(position, before, cost) for each group with work, in
// one thread.  Ends with a barrier.
template <int kThreads, typename Cost, typename With, typename Place>
__device__ __forceinline__ GroupPlan plan_groups(const Int4Launch& p, const GroupLists& l,
                                                 int64_t* warp_sum, Cost cost, With with,
                                                 Place place) {
  // costs of neighbouring groups in a thread, then a scan of them and of the
  // number of groups (in the low bits of the same word)
  constexpr int kPer = (kMaxGroups + kThreads - 1) / kThreads, kCountBits = 11;
  static_assert(kMaxGroups < 1 << kCountBits, "");
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int n0 = p.seg[0].groups, groups = n0 + (p.nseg > 1 ? p.seg[1].groups : 0);
  if (groups == 1 && !p.seg[0].offsets) {  // a linear map: nothing to scan
    GroupPlan one;
    one.total = cost(0, static_cast<int>(p.seg[0].rows));
    one.present = one.total > 0;
    with(one.total);
    if (tid == 0 && one.present) {
      l.before[0] = 0;
      l.before[1] = one.total;
      l.number[0] = 0;
      place(0, static_cast<int64_t>(0), one.total);
    }
    __syncthreads();
    return one;
  }
  int64_t mine[kPer], sum = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int k = tid * kPer + i, si = k >= n0;
    mine[i] = 0;
    if (k >= groups) continue;
    const Int4Segment& s = p.seg[si];
    int n = static_cast<int>(s.rows);
    if (s.offsets) {
      const int32_t a = s.offsets[k], b = s.offsets[k + 1];
      l.first[k] = a;
      if (k == n0 - 1) l.first[n0] = b;
      n = b - a;
    }
    const int64_t c = cost(si, n);
    if (c) mine[i] = c << kCountBits | 1;
    sum += mine[i];
  }
  int64_t incl = sum;
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) warp_sum[warp] = incl;
  __syncthreads();
  int64_t at = incl - sum, total = 0;
#pragma unroll
  for (int v = 0; v < kThreads / 32; ++v) {
    const int64_t w = warp_sum[v];
    if (v < warp) at += w;
    total += w;
  }
  GroupPlan plan;
  plan.present = static_cast<int>(total & ((1 << kCountBits) - 1));
  plan.total = total >> kCountBits;
  with(plan.total);
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    if (!mine[i]) continue;
    const int pos = static_cast<int>(at & ((1 << kCountBits) - 1));
    l.before[pos] = at >> kCountBits;
    l.number[pos] = static_cast<uint16_t>(tid * kPer + i);
    place(pos, at >> kCountBits, mine[i] >> kCountBits);
    at += mine[i];
  }
  if (tid == 0) l.before[plan.present] = plan.total;
  __syncthreads();
  return plan;
}

}  // namespace fgs
