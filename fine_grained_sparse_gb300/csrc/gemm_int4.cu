// Products of more than a few rows with 4-bit weights, on the tensor cores
// (tcgen05): the groups that gemv_int4.cu leaves.  128 weight rows by up to
// 128 tokens a unit, in one of two forms:
//
//  bf16 rows   gemm_int4_bf16_kernel   weights as two bf16 values, sums over
//              all of K in TMEM
//  E4M3 rows   gemm_int4_bytes_kernel  both operands stay bytes, the sums over
//              a scale's columns are scaled in fp32
//
// All products are exact.  What bounds both is making the first operand:
// a block of 128 x 128 weights is 16 to 18 KB of HBM, but some 4500 warp
// instructions from codes to swizzled operand to sums (96 tokens and 17
// experts' groups of which 11 come here: 4580 with bf16 rows at 2.5 a cycle
// and SM, tensor pipe 39% active, shared-memory pipe 48%; E4M3 rows 4460 with
// groups of 128, 5740 with groups of 32).  It is made once for all of a unit's
// tokens, so the form pays from kGemvRows rows on.
#include "int4.cuh"

namespace fgs {
namespace {

// Where a launch that brings no status word (a linear map has no workspace)
// records that a wait expired, at its end: one word of the library's on each
// device.
__device__ int library_status;

constexpr int kWorkers = 16;  // warps that make the operands and add up the chunks' sums
constexpr int kThreads = 32 * (kWorkers + 1);  // and the one that issues the MMAs
constexpr int kBlocks = 8;    // row blocks of a unit
constexpr int kRows = 16 * kBlocks;
constexpr int kTokens = 128;
constexpr int kDepth = 4;         // half records of a worker's ring
constexpr int kAtom = 128 * 128;  // bytes of 128 swizzled rows of 128 bytes

// Half a record (64 columns) with all of its scales.
__host__ __device__ constexpr int half_bytes(int group) { return record_bytes(group) - kCodeBytes / 2; }
__host__ __device__ constexpr int ring_bytes(int group) {
  return kWorkers * kDepth * half_bytes(group);
}

// One unit: a row tile of a group against a tile of its tokens.
struct Unit {
  int seg;         // -1: none
  int blocks;      // 16-row blocks, up to 8
  int first_block;
  int n;           // tokens
  int chunks;
  const uint8_t* W;  // the tile's first record
  int64_t out_row, x_row;
};

// Unit u of the launch; pos: where in the group lists to look from (units
// are asked for in ascending order).  Token tiles run fastest, so that the
// CTAs that read the same weights do so at the same time.
template <int kMostTokens>
__device__ __forceinline__ Unit unit_at(const Int4Launch& p, const GroupLists& l, GroupPlan plan,
                                        int u, int& pos, int rec) {
  Unit x;
  x.seg = -1;
  x.n = x.chunks = x.blocks = 0;
  if (u >= plan.total) return x;
  while (l.before[pos + 1] <= u) ++pos;
  const int n0 = p.seg[0].groups, k = l.number[pos];
  x.seg = k >= n0;
  const Int4Segment& s = p.seg[x.seg];
  const int grp = x.seg ? k - n0 : k;
  const int first = s.offsets ? l.first[k] : 0;
  const int n = s.offsets ? l.first[k + 1] - first : static_cast<int>(s.rows);
  const uint32_t tiles = (n + kMostTokens - 1u) / kMostTokens;
  const uint32_t local = u - static_cast<int>(l.before[pos]);
  const int m = local / tiles, t = local - m * tiles;
  const int row0 = static_cast<int>(static_cast<int64_t>(n) * t / tiles);
  x.n = static_cast<int>(static_cast<int64_t>(n) * (t + 1) / tiles) - row0;
  x.first_block = m * kBlocks;
  x.blocks = min(kBlocks, s.blocks - x.first_block);
  x.chunks = s.chunks;
  x.W = s.W + (static_cast<int64_t>(grp) * s.blocks + x.first_block) * s.chunks * rec;
  x.out_row = row0 + (s.offsets ? first : grp * s.out_group_rows);
  x.x_row = row0 + (s.offsets ? first : grp * s.x_group_rows);
  return x;
}

// A CTA's first unit, and the one after u.  The round that does not fill the
// grid (the first `rest` units) comes first, so that a shared expert's units,
// which are the last and often the longer ones, fall to CTAs that sit it out (301
// tokens of 64 experts, the shared one twice as wide: 102.1 -> 98.6 us; where
// all units are equal, 128 and 512 tokens, within 0.1%).
__device__ __forceinline__ int first_unit(int rest) {
  const int b = blockIdx.x;
  return b < rest ? b : b + rest;
}
__device__ __forceinline__ int next_unit(int u, int rest) {
  return u + (u < rest ? rest : static_cast<int>(gridDim.x));
}

// o[i] += f[i] (r v[i]) for four tokens, two to an instruction.
__device__ __forceinline__ void add_scaled4(float* o, float4 f, float r, const uint32_t* v) {
  asm("{\n\t.reg .b64 a, b, x, y, s, t, u;\n\t"
      "mov.b64 a, {%0, %1};\n\tmov.b64 b, {%2, %3};\n\t"
      "mov.b64 s, {%4, %5};\n\tmov.b64 t, {%6, %7};\n\tmov.b64 u, {%8, %8};\n\t"
      "mov.b64 x, {%9, %10};\n\tmov.b64 y, {%11, %12};\n\t"
      "mul.rn.f32x2 x, x, u;\n\tmul.rn.f32x2 y, y, u;\n\t"
      "fma.rn.f32x2 a, s, x, a;\n\tfma.rn.f32x2 b, t, y, b;\n\t"
      "mov.b64 {%0, %1}, a;\n\tmov.b64 {%2, %3}, b;\n\t}"
      : "+f"(o[0]), "+f"(o[1]), "+f"(o[2]), "+f"(o[3])
      : "f"(f.x), "f"(f.y), "f"(f.z), "f"(f.w), "f"(r), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]));
}

// A unit's outputs from the sums of row `row` and tokens t0 .. t0 + cols - 1
// (cols 16 or 32); weight: the row weight of token t0 + lane.
template <bool kSwiglu>
__device__ __forceinline__ void write_unit(const Int4Segment& s, const Unit& x,
                                           const float (&acc)[kTokens / 4], float weight, int t0,
                                           int cols, int row, int lane) {
  const bool live = row / 16 < x.blocks;
  const int block = x.first_block + row / 16;
  if (kSwiglu) {
    // rows r < 8 of a block are gate rows, r + 8 the up rows of the same
    // features: lanes 8 apart swap halves and each finishes half the tokens
    const bool up = lane & 8;
    __nv_bfloat16* out = s.out + (x.out_row + t0) * s.out_ld + block * 8 + (lane & 7);
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      // with 16 tokens, j and j + 8; with 32, j and j + 16
      if (cols == 16 && j >= 8) break;
      const float low = acc[j], high = cols == 16 ? acc[(j + 8) & 31] : acc[j + 16];
      const float got = __shfl_xor_sync(0xffffffffu, up ? low : high, 8);
      const float gate = up ? got : low, lin = up ? high : got;
      const int t = j + (up ? cols / 2 : 0);
      if (live && t0 + t < x.n)  // H is rounded to bf16, the type of the layer's activations
        out[t * s.out_ld] = __float2bfloat16_rn(silu_f(gate) * lin);
    }
  } else {
    const int64_t o = (x.out_row + t0) * s.out_ld + block * 16 + (lane & 15);
#pragma unroll
    for (int j = 0; j < 32; ++j) {
      if (j >= cols) break;
      float v = __shfl_sync(0xffffffffu, weight, j) * acc[j];
      if (live && t0 + j < x.n) {
        if (s.add) v += __bfloat162float(s.add[o + j * s.out_ld]);
        s.out[o + j * s.out_ld] = __float2bfloat16_rn(v);
      }
    }
  }
}

// ------------------------------------------------------------- bf16 rows
// With x in bf16 both operands are bf16 and nothing is left to apply to the
// sums: b is x as it lies in memory, a weight (c - 8) s is the sum of two bf16
// values (its rounding and the rest, at most 11 significant bits together),
// and the MMAs of both run over all of K in TMEM accumulators of their own,
// issued by two warps: one thread takes about 100 cycles for each MMA beside
// the workers, and eight a stage held everything up (linear 7168-18432, 64
// tokens: 70 us).
// Stages are 64 columns (a high, a low, b): four where no group has more than
// 64 rows, so that each parity has two (linear 7168-18432, 64 tokens: 53.3 us,
// 54.4 with the three of 128 tokens); three otherwise.
__host__ __device__ constexpr int stages(int tokens) { return tokens == 64 ? 4 : 3; }
__host__ __device__ constexpr int stage_bytes(int tokens) { return 2 * kAtom + tokens * 128; }
constexpr int kThreadsB = 32 * (kWorkers + 2);
constexpr int kTmemColsB = 4 * kTokens;     // [unit parity][high, low][tokens]

struct HeaderB {
  uint64_t full[4], empty[4], tfull[2], tempty[2], drain;
  uint32_t tmem;
  int abort;
  int at_first, pad;
  int64_t warp_sum[kThreadsB / 32];
  int64_t lists[1];
};

inline int smem_bytes_b(int tokens, int groups, int group) {
  return 1024 + stages(tokens) * stage_bytes(tokens) + ring_bytes(group) +
         (static_cast<int>(sizeof(HeaderB)) + group_list_bytes(groups) + 15) / 16 * 16;
}

// Half h of a record, at `rec` (codes, then the scales; this lane's
// g = lane / 4 and c = lane % 4), into the two halves of the a operand at
// hi_to and lo_to (rows row and row + 8, row = 16 w + g).  Lanes of odd g take
// the half's two 32-column parts in the other order, which puts the rows that
// are stored together on different banks.
template <int kGroup>
__device__ __forceinline__ void make_a_split(const uint8_t* rec, uint8_t* hi_to, uint8_t* lo_to,
                                             int row, int h, int lane) {
  const int g = lane >> 2, c = lane & 3, odd = g & 1;
  const uint8_t* scales = rec + kCodeBytes / 2;
  uint32_t s[2][2];  // [row g, row g + 8][part in order], bf16 pairs
  if (kGroup == 128) {
    const uint32_t sc = *reinterpret_cast<const uint32_t*>(scales + g * 4);
    s[0][0] = s[0][1] = __byte_perm(sc, 0, 0x1010);
    s[1][0] = s[1][1] = __byte_perm(sc, 0, 0x3232);
  } else {
    const uint2 a = *reinterpret_cast<const uint2*>(scales + g * 16);
    const uint2 b = *reinterpret_cast<const uint2*>(scales + g * 16 + 8);
    const uint32_t v0 = h ? a.y : a.x, v1 = h ? b.y : b.x;
    const uint32_t first = odd ? 0x3232u : 0x1010u, second = odd ? 0x1010u : 0x3232u;
    s[0][0] = __byte_perm(v0, 0, first);
    s[0][1] = __byte_perm(v0, 0, second);
    s[1][0] = __byte_perm(v1, 0, first);
    s[1][1] = __byte_perm(v1, 0, second);
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint2 v = *reinterpret_cast<const uint2*>(rec + lane * 16 + ((i ^ odd) << 3));
    uint32_t hi[2][4], lo[2][4];  // [row g, row g + 8], eight columns
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const uint32_t w = j ? v.y : v.x;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        uint32_t q = ((w >> (4 * k)) & 0x000f000fu) | 0x43004300u;  // 128 + c
        uint32_t& o = hi[k & 1][2 * j + (k >> 1)];
        uint32_t& r = lo[k & 1][2 * j + (k >> 1)];
        asm("sub.rn.bf16x2 %0, %0, %1;" : "+r"(q) : "r"(0x43084308u));
        asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(o) : "r"(q), "r"(s[k & 1][i]));
        asm("{\n\t.reg .b32 n;\n\tneg.bf16x2 n, %1;\n\tfma.rn.bf16x2 %0, %2, %3, n;\n\t}"
            : "=r"(r)
            : "r"(o), "r"(q), "r"(s[k & 1][i]));
      }
    }
    const int at = ((4 * (i ^ odd) + c) ^ g) << 4;
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      *reinterpret_cast<uint4*>(hi_to + (row + 8 * b) * 128 + at) =
          make_uint4(hi[b][0], hi[b][1], hi[b][2], hi[b][3]);
      *reinterpret_cast<uint4*>(lo_to + (row + 8 * b) * 128 + at) =
          make_uint4(lo[b][0], lo[b][1], lo[b][2], lo[b][3]);
    }
  }
}

// Stage j of the CTA's units is 64 columns; the workers of parity j mod 2
// (one for each row block) make it: they start the copies of b, convert a and
// hand it over when the copies have landed.  A unit's outputs are written
// while the next unit's first stages run, from the other half of TMEM.
template <bool kSwiglu, int kGroup, int kMostTokens>
__global__ void __launch_bounds__(kThreadsB, 1)
    gemm_int4_bf16_kernel(const __grid_constant__ Int4Launch p) {
  constexpr int kStages = stages(kMostTokens), kStageBytes = stage_bytes(kMostTokens);
  constexpr int kRec = record_bytes(kGroup), kHalf = half_bytes(kGroup);
  extern __shared__ __align__(16) uint8_t raw[];
  uint8_t* smem = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
  uint8_t* ring_base = smem + kStages * kStageBytes;
  HeaderB* hd = reinterpret_cast<HeaderB*>(ring_base + ring_bytes(kGroup));
  const int groups = p.seg[0].groups + (p.nseg > 1 ? p.seg[1].groups : 0);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile int* abort_flag = &hd->abort;
  auto bar = [](uint64_t& b) { return smem_u32(&b); };

  if (warp == 0) {
    tmem_alloc(smem_u32(&hd->tmem), kTmemColsB);
    tmem_relinquish();
  }
  if (warp == kWorkers && lane == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(bar(hd->full[i]), kWorkers / 2);
      mbar_init(bar(hd->empty[i]), 2);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(hd->tfull[i]), 2);
      mbar_init(bar(hd->tempty[i]), kWorkers);
    }
    mbar_init(bar(hd->drain), 2);
    hd->abort = 0;
    fence_mbarrier_init();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = hd->tmem;

  if (p.wait == kWaitWeights) pdl_wait();
  pdl_release();
  const GroupLists lists = group_lists(hd->lists, groups);
  int u0 = 0, rest = 0;
  const GroupPlan plan = plan_groups<kThreadsB>(
      p, lists, hd->warp_sum,
      [&](int si, int n) -> int64_t {
        if (n <= p.most) return 0;
        return static_cast<int64_t>((p.seg[si].blocks + kBlocks - 1) / kBlocks) *
               ((n + kMostTokens - 1u) / kMostTokens);
      },
      [&](int64_t total) {
        rest = static_cast<int>(total % gridDim.x);
        u0 = first_unit(rest);
      },
      [&](int pos, int64_t before, int64_t cost) {
        if (before <= u0 && u0 < before + cost) hd->at_first = pos;
      });
  int pos = u0 < plan.total ? hd->at_first : 0;

  if (warp < kWorkers) {
    const int parity = warp & 1, a_block = warp >> 1, g = lane >> 2;
    const int piece = lane & 7, sub = 4 * a_block + (lane >> 3);  // of b: tokens 32 k + sub
    const int quarter = warp & 3, row = 32 * quarter + lane;      // of the outputs
    uint8_t* const ring = ring_base + warp * kDepth * kHalf;
    constexpr int kTasks = kMostTokens / 32;

    // the outputs of unit `of`, the seq-th of the CTA; false: gave up
    auto finish = [&](const Unit& of, int seq) {
      const int buf = seq & 1;
      if (!mbar_wait_bounded(bar(hd->tfull[buf]), seq >> 1 & 1, abort_flag, p.status)) return false;
      __syncwarp();
      tc_fence_after();
      const Int4Segment& s = p.seg[of.seg];
      const int cols = of.n > 64 ? 32 : 16, t0 = (warp >> 2) * cols;
      const bool live = row / 16 < of.blocks;
      const int block = of.first_block + row / 16;
      float weight = 1.0f;
      if (!kSwiglu && s.row_w && t0 + lane < of.n)
        weight = s.row_w[s.row_perm[of.out_row + t0 + lane]];
#pragma unroll
      for (int b = 0; b < kMostTokens / 64; ++b) {
        if (16 * b >= cols) break;
        uint32_t v[16], v2[16];
        const uint32_t from = tmem + 2 * buf * kTokens + t0 + 16 * b +
                              (static_cast<uint32_t>(32 * quarter) << 16);
        tmem_ld_x16(from, v);
        tmem_ld_x16(from + kTokens, v2);
        tmem_ld_wait(v);
        tmem_ld_wait(v2);
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          // An infinity of x has met the weights' high parts, which are zero
          // where the weight is and have its sign; against the rests, which
          // may be zero or of the other sign, it says nothing.
          const float high = __uint_as_float(v[j]), rest = __uint_as_float(v2[j]);
          v[j] = __float_as_uint(isfinite(high) ? high + rest : high);
        }
        if (kSwiglu) {
          // rows r < 8 of a block are gate rows, r + 8 the up rows of the
          // same features: lanes 8 apart swap and each finishes half the tokens
          const bool up = lane & 8;
          const int first = t0 + 16 * b + (up ? 8 : 0);
          __nv_bfloat16* out = s.out + (of.out_row + first) * s.out_ld + block * 8 + (lane & 7);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float low = __uint_as_float(v[j]), high = __uint_as_float(v[j + 8]);
            const float got = __shfl_xor_sync(0xffffffffu, up ? low : high, 8);
            const float gate = up ? got : low, lin = up ? high : got;
            if (live && first + j < of.n)  // H is rounded to bf16, the type of the activations
              out[j * s.out_ld] = __float2bfloat16_rn(silu_f(gate) * lin);
          }
        } else {
          const int64_t o = (of.out_row + t0 + 16 * b) * s.out_ld + block * 16 + (lane & 15);
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            float r = __shfl_sync(0xffffffffu, weight, 16 * b + j) * __uint_as_float(v[j]);
            if (live && t0 + 16 * b + j < of.n) {
              if (s.add) r += __bfloat162float(s.add[o + j * s.out_ld]);
              s.out[o + j * s.out_ld] = __float2bfloat16_rn(r);
            }
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(hd->tempty[buf]));
      return true;
    };

    bool ok = true;
    int seq = 0, slot = parity, phase = 0;
    Unit of;  // whose outputs are to be written
    of.seg = -1;
    for (int u = u0; u < plan.total && ok; u = next_unit(u, rest), ++seq) {
      const Unit x = unit_at<kMostTokens>(p, lists, plan, u, pos, kRec);
      const Int4Segment& s = p.seg[x.seg];
      const bool has_a = a_block < x.blocks;
      const uint8_t* w = x.W + (has_a ? static_cast<int64_t>(a_block) * x.chunks * kRec : 0) +
                         parity * (kCodeBytes / 2) + lane * 16;
      auto fetch = [&](int ch) {
        if (has_a && ch < x.chunks) {
          const uint32_t to = smem_u32(ring + (ch & (kDepth - 1)) * kHalf) + lane * 16;
          const uint8_t* from = w + ch * kRec;
          cp_async16(to, from);
          if (lane < (kRec - kCodeBytes) / 16)
            cp_async16(to + kCodeBytes / 2, from + kCodeBytes - parity * (kCodeBytes / 2));
        }
      };
#pragma unroll
      for (int c = 0; c < kDepth - 1; ++c) {
        fetch(c);
        asm volatile("cp.async.commit_group;" ::: "memory");
      }
      if (seq == 0 && p.wait == kWaitX) pdl_wait();
      const uint8_t* xp[kTasks];  // this lane's piece of its tokens' rows
      {
        const int t = 32 * (lane >> 2 & (kTasks - 1)) + 4 * a_block + (lane & 3);
        const int64_t at = x.x_row + min(t, x.n - 1);
        const int mine = static_cast<int>(s.perm ? s.perm[at] / s.perm_div : at);
#pragma unroll
        for (int k = 0; k < kTasks; ++k)
          xp[k] = static_cast<const uint8_t*>(s.x) +
                  static_cast<int64_t>(__shfl_sync(0xffffffffu, mine, 4 * k + (lane >> 3))) *
                      x.chunks * (2 * kChunk) + parity * kChunk + piece * 16;
      }
      for (int ch = 0; ch < x.chunks; ++ch) {
        asm volatile("cp.async.wait_group %0;" ::"n"(kDepth - 2) : "memory");
        __syncwarp();
        if (!mbar_wait_bounded(bar(hd->empty[slot]), phase ^ 1, abort_flag, p.status)) {
          ok = false;
          break;
        }
        uint8_t* st = smem + slot * kStageBytes;
#pragma unroll
        for (int k = 0; k < kTasks; ++k) {
          const int t = 32 * k + sub;
          if (t < x.n)
            cp_async16(smem_u32(st + 2 * kAtom) + t * 128 + ((piece ^ (t & 7)) << 4),
                       xp[k] + ch * (2 * kChunk));
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        fetch(ch + kDepth - 1);
        asm volatile("cp.async.commit_group;" ::: "memory");
        if (has_a)
          make_a_split<kGroup>(ring + (ch & (kDepth - 1)) * kHalf, st, st + kAtom, 16 * a_block + g,
                               parity, lane);
        // b has landed, and every half record but the one just asked for
        asm volatile("cp.async.wait_group 1;" ::: "memory");
        fence_proxy_async_smem();  // the tensor cores read the operands next
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(hd->full[slot]));
        if ((slot += 2) >= kStages) {
          slot -= kStages;
          phase ^= 1;
        }
        if (of.seg >= 0 && ch == min(1, x.chunks - 1)) {
          if (!finish(of, seq - 1)) {
            ok = false;
            break;
          }
          of.seg = -1;
        }
      }
      of = x;
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    if (ok && of.seg >= 0) finish(of, seq - 1);
  } else {
    if (lane == 0) {
      const int low = warp - kWorkers;  // 1: the rests
      int slot = 0, phase = 0, seq = 0;
      bool ok = true;
      for (int u = u0; ok && u < plan.total; u = next_unit(u, rest), ++seq) {
        const Unit x = unit_at<kMostTokens>(p, lists, plan, u, pos, kRec);
        const uint32_t idesc = idesc_bf16_f32(128, x.n > 64 ? 128 : 64);
        const uint32_t d = tmem + (2 * (seq & 1) + low) * kTokens;
        if (!mbar_wait_bounded(bar(hd->tempty[seq & 1]), (seq >> 1 & 1) ^ 1, abort_flag, p.status))
          break;
        for (int j = 0; j < 2 * x.chunks; ++j) {
          if (!mbar_wait_bounded(bar(hd->full[slot]), phase, abort_flag, p.status)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t st = smem_u32(smem + slot * kStageBytes);
          const uint64_t a = smem_desc_sw128(st + low * kAtom), b = smem_desc_sw128(st + 2 * kAtom);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            tc_mma_bf16(d, a + 2u * kk, b + 2u * kk, idesc, (j | kk) != 0);
          tc_commit(bar(hd->empty[slot]));
          if (++slot == kStages) {
            slot = 0;
            phase ^= 1;
          }
        }
        tc_commit(bar(hd->tfull[seq & 1]));
      }
      // nothing is in flight when the CTA gives its TMEM back
      tc_commit(bar(hd->drain));
      int own_abort = 0;
      if (!mbar_wait_bounded(bar(hd->drain), 0, &own_abort, p.status)) hd->abort = 1;
    }
    __syncwarp();
  }
  if (p.wait != kWaitWeights) pdl_wait();  // a kernel ends after the one before it has
  tc_fence_before();
  __syncthreads();
  if (threadIdx.x == 0 && hd->abort && !p.status) record_status(&library_status, MOE_ERR_TIMEOUT);
  if (warp == 0) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, kTmemColsB);
  }
}

// ------------------------------------------------------------- E4M3 rows
// The operands can stay bytes (kind::f8f6f4): b is x as it lies in memory, and
// a code c as an E4M3 byte is c 2^-9 (subnormals and the first normal binade
// are evenly spaced), so that masks make a from the codes.  A constant first
// operand of -8 2^-9 adds what makes the codes signed.  The sums over the
// columns of one scale come to registers, where both scales are applied and
// the chunks are added up in fp32.  With scales of 32 columns, one step of
// the MMA's K, a chunk has four accumulators.  7168 to 18432 columns: 64
// tokens 63 us with scales of 128 columns, 73 with 32; 2048 tokens 1110 and
// 1354.  (As f16, (c - 8) s needs one accumulator a chunk in either case, but
// holds a row's four scales together only while they are within 2^24 of one
// another; it took 82 and 1377 us.)
constexpr int kStagesC = 3;
constexpr int kStageBytesC = 2 * kAtom;  // a, b: 128 rows of 128 bytes

// A chunk's accumulators, one for each scale, and the chunks whose sums TMEM
// holds: two, or one with four accumulators, whose MMAs have the time in which
// the workers make the next chunk.
__host__ __device__ constexpr int scales(int group) { return kChunk / group; }
__host__ __device__ constexpr int buffers(int group) { return group == 32 ? 1 : 2; }
__host__ __device__ constexpr int tmem_cols_c(int group) {
  return buffers(group) * scales(group) * kTokens;
}

// b and f are asked for a chunk ahead, when sums four chunks back may still be
// read: eight chunks' factors are kept.
constexpr int kFactorsC = 8;

template <int kGroup>
struct HeaderC {
  float f[kFactorsC][kTokens];
  float r[kFactorsC][scales(kGroup)][kRows];
  uint64_t full[kStagesC], empty[kStagesC], tfull[2], tempty[2], drain;
  uint32_t tmem;
  int abort;
  int at_first, pad;
  int64_t warp_sum[kThreads / 32];
  int64_t lists[1];
};

template <int kGroup>
int smem_bytes_c(int groups) {
  return 1024 + kStagesC * kStageBytesC + kAtom + ring_bytes(kGroup) +
         (static_cast<int>(sizeof(HeaderC<kGroup>)) + group_list_bytes(groups) + 15) / 16 * 16;
}

// The sums of one scale's columns are below 2^10 in units of the codes' 2^-9;
// the scales enter times 2^-10, so that no product with a sum leaves fp32's
// range where the weights are inside it, and a unit's outputs are brought back.
constexpr float kSmall = 0x1p-10f, kBack = 0x1p19f;

// Both operands E4M3 (format 0), K-major, fp32 sums, M = 128, N = n.
__device__ __forceinline__ uint32_t idesc_e4m3_f32(uint32_t n) {
  return (1u << 4) | ((n >> 3) << 17) | ((128u >> 4) << 24);
}

// D[tmem] (+)= A[smem] * B[smem]^T, E4M3 inputs, fp32 accumulator, M = 128.
__device__ __forceinline__ void tc_mma_e4m3(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                            uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// v0[i] = r0 v0[i] + r1 v1[i] for four tokens, two to an instruction.
__device__ __forceinline__ void join4(uint32_t* v0, float r0, const uint32_t* v1, float r1) {
  asm("{\n\t.reg .b64 x, y, s, t, u, w;\n\t"
      "mov.b64 u, {%4, %4};\n\tmov.b64 w, {%5, %5};\n\t"
      "mov.b64 x, {%0, %1};\n\tmov.b64 y, {%2, %3};\n\t"
      "mul.rn.f32x2 x, x, u;\n\tmul.rn.f32x2 y, y, u;\n\t"
      "mov.b64 s, {%6, %7};\n\tmov.b64 t, {%8, %9};\n\t"
      "fma.rn.f32x2 x, s, w, x;\n\tfma.rn.f32x2 y, t, w, y;\n\t"
      "mov.b64 {%0, %1}, x;\n\tmov.b64 {%2, %3}, y;\n\t}"
      : "+r"(v0[0]), "+r"(v0[1]), "+r"(v0[2]), "+r"(v0[3])
      : "f"(r0), "f"(r1), "r"(v1[0]), "r"(v1[1]), "r"(v1[2]), "r"(v1[3]));
}

// o[i] += f[i] (x[i] + r0 v0[i] + r1 v1[i]) for four tokens.
__device__ __forceinline__ void add_joined4(float* o, float4 f, const uint32_t* x0, float r0,
                                            const uint32_t* v0, float r1, const uint32_t* v1) {
  asm("{\n\t.reg .b64 a, b, x, y, s, t, u, w;\n\t"
      "mov.b64 u, {%8, %8};\n\tmov.b64 w, {%9, %9};\n\t"
      "mov.b64 x, {%10, %11};\n\tmov.b64 y, {%12, %13};\n\t"
      "mov.b64 s, {%14, %15};\n\tmov.b64 t, {%16, %17};\n\t"
      "fma.rn.f32x2 x, s, u, x;\n\tfma.rn.f32x2 y, t, u, y;\n\t"
      "mov.b64 s, {%18, %19};\n\tmov.b64 t, {%20, %21};\n\t"
      "fma.rn.f32x2 x, s, w, x;\n\tfma.rn.f32x2 y, t, w, y;\n\t"
      "mov.b64 a, {%0, %1};\n\tmov.b64 b, {%2, %3};\n\t"
      "mov.b64 s, {%4, %5};\n\tmov.b64 t, {%6, %7};\n\t"
      "fma.rn.f32x2 a, s, x, a;\n\tfma.rn.f32x2 b, t, y, b;\n\t"
      "mov.b64 {%0, %1}, a;\n\tmov.b64 {%2, %3}, b;\n\t}"
      : "+f"(o[0]), "+f"(o[1]), "+f"(o[2]), "+f"(o[3])
      : "f"(f.x), "f"(f.y), "f"(f.z), "f"(f.w), "f"(r0), "f"(r1), "r"(x0[0]), "r"(x0[1]),
        "r"(x0[2]), "r"(x0[3]), "r"(v0[0]), "r"(v0[1]), "r"(v0[2]), "r"(v0[3]), "r"(v1[0]),
        "r"(v1[1]), "r"(v1[2]), "r"(v1[3]));
}

// 32 lanes x 8 consecutive 32-bit columns of two accumulators of TMEM into
// registers, and the wait for them.
__device__ __forceinline__ void tmem_ld_two_x8(uint32_t from0, uint32_t from1, uint32_t (&v0)[8],
                                               uint32_t (&v1)[8]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%16];\n\t"
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%8, %9, %10, %11, %12, %13, %14, %15}, [%17];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=&r"(v0[0]), "=&r"(v0[1]), "=&r"(v0[2]), "=&r"(v0[3]), "=&r"(v0[4]), "=&r"(v0[5]),
        "=&r"(v0[6]), "=&r"(v0[7]), "=&r"(v1[0]), "=&r"(v1[1]), "=&r"(v1[2]), "=&r"(v1[3]),
        "=&r"(v1[4]), "=&r"(v1[5]), "=&r"(v1[6]), "=&r"(v1[7])
      : "r"(from0), "r"(from1)
      : "memory");
}

// Sixteen worker warps make the operands of chunk i (half of a row block of
// the weights each, and four tokens' rows of each 64) and then add up the sums
// of chunk i - 1 (a quarter of the rows, a quarter of the tokens), while the
// MMAs of chunk i run; one more warp issues those.  Sixteen warps of both
// kinds of work, not eight of each: a scheduler has four to choose from, and
// two could not hide the latencies (a chunk of 64 tokens took 3900 cycles).
template <bool kSwiglu, int kGroup>
__global__ void __launch_bounds__(kThreads, 1)
    gemm_int4_bytes_kernel(const __grid_constant__ Int4Launch p) {
  constexpr int kRec = record_bytes(kGroup), kHalf = half_bytes(kGroup);
  constexpr int kScales = scales(kGroup), kBuffers = buffers(kGroup);
  constexpr int kTmemCols = tmem_cols_c(kGroup);
  extern __shared__ __align__(16) uint8_t raw[];
  uint8_t* smem = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
  uint8_t* bias = smem + kStagesC * kStageBytesC;
  uint8_t* ring_base = bias + kAtom;
  using Header = HeaderC<kGroup>;
  Header* hd = reinterpret_cast<Header*>(ring_base + ring_bytes(kGroup));
  const int groups = p.seg[0].groups + (p.nseg > 1 ? p.seg[1].groups : 0);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile int* abort_flag = &hd->abort;
  auto bar = [](uint64_t& b) { return smem_u32(&b); };

  if (warp == 0) {
    tmem_alloc(smem_u32(&hd->tmem), kTmemCols);
    tmem_relinquish();
  }
  if (warp == kWorkers && lane == 0) {
    for (int i = 0; i < kStagesC; ++i) {
      mbar_init(bar(hd->full[i]), kWorkers);
      mbar_init(bar(hd->empty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(hd->tfull[i]), 1);
      mbar_init(bar(hd->tempty[i]), kWorkers);
    }
    mbar_init(bar(hd->drain), 1);
    hd->abort = 0;
    fence_mbarrier_init();
  }
  for (int i = threadIdx.x; i < kAtom / 16; i += kThreads)
    reinterpret_cast<uint4*>(bias)[i] = make_uint4(0x88888888u, 0x88888888u, 0x88888888u, 0x88888888u);
  fence_proxy_async_smem();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = hd->tmem;

  if (p.wait == kWaitWeights) pdl_wait();
  pdl_release();
  const GroupLists lists = group_lists(hd->lists, groups);
  int u0 = 0, rest = 0;
  const GroupPlan plan = plan_groups<kThreads>(
      p, lists, hd->warp_sum,
      [&](int si, int n) -> int64_t {
        if (n <= p.most) return 0;
        return static_cast<int64_t>((p.seg[si].blocks + kBlocks - 1) / kBlocks) *
               ((n + kTokens - 1u) / kTokens);
      },
      [&](int64_t total) {
        rest = static_cast<int>(total % gridDim.x);
        u0 = first_unit(rest);
      },
      [&](int pos, int64_t before, int64_t cost) {
        if (before <= u0 && u0 < before + cost) hd->at_first = pos;
      });
  int pos = u0 < plan.total ? hd->at_first : 0;

  if (warp < kWorkers) {
    const int a_block = warp >> 1, a_half = warp & 1, g = lane >> 2, c = lane & 3;
    const int piece = lane & 7, sub = 4 * warp + (lane >> 3);  // of b: tokens 64 k + sub
    const int quarter = warp & 3, row = 32 * quarter + lane;   // of the sums
    uint8_t* const ring = ring_base + warp * kDepth * kHalf;
    bool ok = true;
    int i = 0, seq = 0;
    int slot = 0;               // stage of chunk i
    int bslot = 0, bphase = 0;  // that of the chunk whose b is asked for next, its round's parity
    int aslot = 0, aphase = 0;  // and those of the chunk whose sums are added next
    for (int u = u0; u < plan.total && ok; u = next_unit(u, rest), ++seq) {
      const Unit x = unit_at<kTokens>(p, lists, plan, u, pos, kRec);
      const Int4Segment& s = p.seg[x.seg];
      const bool has_a = a_block < x.blocks;
      const uint8_t* w = x.W + (has_a ? static_cast<int64_t>(a_block) * x.chunks * kRec : 0) +
                         a_half * (kCodeBytes / 2) + lane * 16;
      auto fetch = [&](int ch) {
        if (has_a && ch < x.chunks) {
          const uint32_t to = smem_u32(ring + (ch & (kDepth - 1)) * kHalf) + lane * 16;
          const uint8_t* from = w + ch * kRec;
          cp_async16(to, from);
          if (lane < (kRec - kCodeBytes) / 16)
            cp_async16(to + kCodeBytes / 2, from + kCodeBytes - a_half * (kCodeBytes / 2));
        }
      };
#pragma unroll
      for (int k = 0; k < kDepth - 1; ++k) fetch(k);
      if (seq == 0 && p.wait == kWaitX) pdl_wait();
      int rows[2];
      {
        const int t = 64 * (lane >> 2 & 1) + 4 * warp + (lane & 3);
        const int64_t at = x.x_row + min(t, x.n - 1);
        const int mine = static_cast<int>(s.perm ? s.perm[at] / s.perm_div : at);
#pragma unroll
        for (int k = 0; k < 2; ++k) rows[k] = __shfl_sync(0xffffffffu, mine, 4 * k + (lane >> 3));
      }
      // chunk ch's b and scales of x, as soon as its stage is free
      auto ask = [&](int ch, int chunk) {
        if (!mbar_wait_bounded(bar(hd->empty[bslot]), bphase ^ 1, abort_flag, p.status)) return false;
        uint8_t* b = smem + bslot * kStageBytesC + kAtom;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int t = 64 * k + sub;
          if (t < x.n) {
            const int64_t from = static_cast<int64_t>(rows[k]) * x.chunks + ch;
            cp_async16(smem_u32(b) + t * 128 + ((piece ^ (t & 7)) << 4),
                       static_cast<const uint8_t*>(s.x) + from * kChunk + piece * 16);
            if (piece == 0)
              asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(
                               smem_u32(&hd->f[chunk & (kFactorsC - 1)][t])),
                           "l"(s.x_scale + from)
                           : "memory");
          }
        }
        if (++bslot == kStagesC) {
          bslot = 0;
          bphase ^= 1;
        }
        return true;
      };
      ok = ask(0, i);
      if (!ok) break;
      asm volatile("cp.async.commit_group;" ::: "memory");
      const int cols = x.n > 64 ? 32 : 16, t0 = (warp >> 2) * cols;  // tokens of the sums
      float weight = 1.0f;  // row weight of token t0 + lane
      if (!kSwiglu && s.row_w && t0 + lane < x.n) weight = s.row_w[s.row_perm[x.out_row + t0 + lane]];
      float acc[kTokens / 4];
#pragma unroll
      for (int j = 0; j < kTokens / 4; ++j) acc[j] = 0.0f;

      // one step more than chunks: step ch makes chunk ch and adds chunk ch - 1
      for (int ch = 0; ch <= x.chunks; ++ch) {
        if (ch < x.chunks) {
          const int fs = i & (kFactorsC - 1);
          // what was asked for a step ago (b of this chunk, half record
          // ch + kDepth - 2) has landed; then ask for the next
          if (ch + 1 < x.chunks && !ask(ch + 1, i + 1)) {
            ok = false;
            break;
          }
          fetch(ch + kDepth - 1);
          asm volatile("cp.async.commit_group;" ::: "memory");
          asm volatile("cp.async.wait_group 1;" ::: "memory");
          __syncwarp();
          if (has_a) {
            const uint8_t* rec = ring + (ch & (kDepth - 1)) * kHalf;
            const uint4 v = *reinterpret_cast<const uint4*>(rec + lane * 16);
            const uint32_t words[4] = {v.x, v.y, v.z, v.w};
            uint8_t* to = smem + slot * kStageBytesC + (16 * a_block + g) * 128 + (c & 1) * 8;
#pragma unroll
            for (int k = 0; k < 2; ++k) {  // parts of 32 columns
              uint32_t lo[2], hi[2];       // rows g and g + 8
#pragma unroll
              for (int j = 0; j < 2; ++j) {
                const uint32_t q = words[2 * k + j];  // columns in the order 0, 2, 1, 3
                lo[j] = __byte_perm(q & 0x0f0f0f0fu, 0, 0x3120);
                hi[j] = __byte_perm((q >> 4) & 0x0f0f0f0fu, 0, 0x3120);
              }
              const int at = ((4 * a_half + 2 * k + (c >> 1)) ^ g) << 4;
              *reinterpret_cast<uint2*>(to + at) = make_uint2(lo[0], lo[1]);
              *reinterpret_cast<uint2*>(to + 8 * 128 + at) = make_uint2(hi[0], hi[1]);
            }
            const uint8_t* sc = rec + kCodeBytes / 2;
            const int ar = 16 * a_block + g;
            if (kScales == 1 && a_half == 0 && c == 0) {  // rows g and g + 8
              const uint32_t v2 = *reinterpret_cast<const uint32_t*>(sc + g * 4);
              hd->r[fs][0][ar] = __uint_as_float(v2 << 16) * kSmall;
              hd->r[fs][0][ar + 8] = __uint_as_float(v2 & 0xffff0000u) * kSmall;
            }
            if (kScales == 4 && c < 2) {  // row g + 8 c, this half's two groups
              const uint32_t v2 = *reinterpret_cast<const uint32_t*>(sc + g * 16 + c * 8 + a_half * 4);
              hd->r[fs][(2 * a_half) % kScales][ar + 8 * c] = __uint_as_float(v2 << 16) * kSmall;
              hd->r[fs][(2 * a_half + 1) % kScales][ar + 8 * c] =
                  __uint_as_float(v2 & 0xffff0000u) * kSmall;
            }
          }
          fence_proxy_async_smem();  // the tensor cores read the operands next
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(hd->full[slot]));
          if (++slot == kStagesC) slot = 0;
          ++i;
        }
        if (ch > 0) {
          const int k = i - (ch < x.chunks ? 2 : 1), fs = k & (kFactorsC - 1);
          const int buf = k & (kBuffers - 1);
          // (the operands were full before; that wait is for f and r)
          if (!mbar_wait_bounded(bar(hd->tfull[buf]), k >> (kBuffers - 1) & 1, abort_flag, p.status) ||
              !mbar_wait_bounded(bar(hd->full[aslot]), aphase, abort_flag, p.status)) {
            ok = false;
            break;
          }
          if (++aslot == kStagesC) {
            aslot = 0;
            aphase ^= 1;
          }
          __syncwarp();
          tc_fence_after();
          const float4* f = reinterpret_cast<const float4*>(hd->f[fs] + t0);
          const uint32_t from =
              tmem + buf * kScales * kTokens + t0 + (static_cast<uint32_t>(32 * quarter) << 16);
          if constexpr (kScales == 1) {
            const float r = hd->r[fs][0][row];
#pragma unroll
            for (int b = 0; b < 2; ++b) {
              if (16 * b < cols) {
                uint32_t v[16];
                tmem_ld_x16(from + 16 * b, v);
                tmem_ld_wait(v);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                  add_scaled4(acc + 16 * b + 4 * j, f[4 * b + j], r, v + 4 * j);
              }
            }
          } else {
            float r[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) r[j] = hd->r[fs][j % kScales][row];
#pragma unroll
            for (int b = 0; b < 4; ++b) {
              if (8 * b < cols) {
                uint32_t x0[8], v0[8], v1[8];
                tmem_ld_two_x8(from + 8 * b, from + kTokens + 8 * b, x0, v1);
                join4(x0, r[0], v1, r[1]);
                join4(x0 + 4, r[0], v1 + 4, r[1]);
                tmem_ld_two_x8(from + 2 * kTokens + 8 * b, from + 3 * kTokens + 8 * b, v0, v1);
#pragma unroll
                for (int j = 0; j < 2; ++j)
                  add_joined4(acc + 8 * b + 4 * j, f[2 * b + j], x0 + 4 * j, r[2], v0 + 4 * j, r[3],
                              v1 + 4 * j);
              }
            }
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(hd->tempty[buf]));
        }
      }
      if (!ok) break;
#pragma unroll
      for (int j = 0; j < kTokens / 4; ++j) acc[j] *= kBack;
      write_unit<kSwiglu>(s, x, acc, weight, t0, cols, row, lane);
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
  } else {
    if (lane == 0) {
      int slot = 0, phase = 0, i = 0;
      bool ok = true;
      for (int u = u0; ok && u < plan.total; u = next_unit(u, rest)) {
        const Unit x = unit_at<kTokens>(p, lists, plan, u, pos, kRec);
        const uint32_t idesc = idesc_e4m3_f32(x.n > 64 ? 128 : 64);
        for (int ch = 0; ch < x.chunks; ++ch, ++i) {
          const int buf = i & (kBuffers - 1);
          if (!mbar_wait_bounded(bar(hd->tempty[buf]), (i >> (kBuffers - 1) & 1) ^ 1, abort_flag,
                                 p.status) ||
              !mbar_wait_bounded(bar(hd->full[slot]), phase, abort_flag, p.status)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t st = smem_u32(smem + slot * kStageBytesC);
          const uint64_t a = smem_desc_sw128(st), b = smem_desc_sw128(st + kAtom);
          const uint64_t minus = smem_desc_sw128(smem_u32(bias));
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) {  // 32 columns
            const uint32_t d = tmem + (buf * kScales + kk % kScales) * kTokens;
            tc_mma_e4m3(d, minus, b + 2u * kk, idesc, kk >= kScales);
            tc_mma_e4m3(d, a + 2u * kk, b + 2u * kk, idesc, 1);
          }
          tc_commit(bar(hd->empty[slot]));
          tc_commit(bar(hd->tfull[buf]));
          if (++slot == kStagesC) {
            slot = 0;
            phase ^= 1;
          }
        }
      }
      // nothing is in flight when the CTA gives its TMEM back
      tc_commit(bar(hd->drain));
      int own_abort = 0;
      if (!mbar_wait_bounded(bar(hd->drain), 0, &own_abort, p.status)) hd->abort = 1;
    }
    __syncwarp();
  }
  if (p.wait != kWaitWeights) pdl_wait();  // a kernel ends after the one before it has
  tc_fence_before();
  __syncthreads();
  if (threadIdx.x == 0 && hd->abort && !p.status) record_status(&library_status, MOE_ERR_TIMEOUT);
  if (warp == 0) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

template <typename Kernel>
cudaError_t launch_kernel(Kernel kernel, const Int4Launch& p, int threads, int num_sms,
                          cudaStream_t stream) {
  // every call: the attribute belongs to a device's context, and setting it
  // costs little beside a launch of many rows
  const cudaError_t err =
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, p.smem);
  if (err != cudaSuccess) return err;
  return launch_pdl(kernel, dim3(num_sms), dim3(threads), p.smem, stream, p);
}

// Rows of a group up to which it is read by gemv_int4.cu.  Among many groups a
// pass of eight rows costs 52 cycles a record and SM, HBM's rate, and making
// the operand here about 250, whatever the rows up to 128: 896 experts of 1 or
// 7 rows and two shared ones of 24 take 916 us, 947 with the limit at 16,
// which sends those two here.  One group alone crosses earlier: a map from 7168
// to 18432 columns, groups of 32, takes 59.6 us for 32 tokens and 76 to 78
// for 33 to 40 streamed, 57.6 for 41 here (E4M3 rows 57.8, 72 to 74, 69.7).
constexpr int kGemvRows = 40;

}  // namespace

cudaError_t launch_gemm_int4(const Int4Launch& p, bool swiglu, int group, int num_sms,
                             cudaStream_t stream) {
  Int4Launch l = p;
  int groups = 0;
  for (int i = 0; i < p.nseg; ++i) groups += p.seg[i].groups;
  if (p.seg[0].x_scale) {
    l.smem = group == 32 ? smem_bytes_c<32>(groups) : smem_bytes_c<128>(groups);
    return launch_kernel(swiglu ? group == 32 ? gemm_int4_bytes_kernel<true, 32>
                                              : gemm_int4_bytes_kernel<true, 128>
                         : group == 32 ? gemm_int4_bytes_kernel<false, 32>
                                       : gemm_int4_bytes_kernel<false, 128>,
                         l, kThreads, num_sms, stream);
  }
  bool small = true;
  for (int i = 0; i < p.nseg; ++i) small = small && p.seg[i].rows <= 64;
  l.smem = smem_bytes_b(small ? 64 : 128, groups, group);
  if (small)
    return launch_kernel(swiglu ? group == 32 ? gemm_int4_bf16_kernel<true, 32, 64>
                                              : gemm_int4_bf16_kernel<true, 128, 64>
                         : group == 32 ? gemm_int4_bf16_kernel<false, 32, 64>
                                       : gemm_int4_bf16_kernel<false, 128, 64>,
                         l, kThreadsB, num_sms, stream);
  return launch_kernel(swiglu ? group == 32 ? gemm_int4_bf16_kernel<true, 32, 128>
                                            : gemm_int4_bf16_kernel<true, 128, 128>
                       : group == 32 ? gemm_int4_bf16_kernel<false, 32, 128>
                                     : gemm_int4_bf16_kernel<false, 128, 128>,
                       l, kThreadsB, num_sms, stream);
}

cudaError_t library_status_word(int** word) {
  return cudaGetSymbolAddress(reinterpret_cast<void**>(word), library_status);
}

cudaError_t launch_int4(const Int4Params& q, int num_sms, cudaStream_t stream) {
  Int4Launch p;
  p.nseg = q.nseg;
  p.status = q.status;
  bool gemv = false, gemm = false;  // whether groups of either kind can occur
  for (int i = 0; i < q.nseg; ++i) {
    p.seg[i] = q.seg[i];
    gemv = gemv || q.seg[i].offsets || q.seg[i].rows <= kGemvRows;
    gemm = gemm || q.seg[i].rows > kGemvRows;
  }
  // `rows` bounds a group with explicit rows only while no token names an
  // expert twice, so without the second kernel the first takes any number
  p.most = gemm ? kGemvRows : 0x7fffffff;
  p.wait = q.early ? kWaitX : kWaitWeights;
  if (gemv) {
    const cudaError_t e = launch_gemv_int4(p, q.swiglu, q.group, num_sms, stream);
    if (e != cudaSuccess || !gemm) return e;
    // the pass's second launch reads nothing that its first wrote; after an
    // early one x is still only known to be there when that one has ended
    p.wait = q.early ? kWaitX : kWaitNone;
  }
  return launch_gemm_int4(p, q.swiglu, q.group, num_sms, stream);
}

}  // namespace fgs
