// Products of a few rows with 4-bit weights: the decode form of the expert
// passes and of a linear map (MOE_WEIGHTS_PACKED_INT4_*).
//
//   z[t, o] = sum_g s[o, g] sum_{k in group g} (c[o, k] - 8) x[t, k]
//
// c are 4-bit codes, s one bf16 scale per 32 or 128 columns of a row, x bf16
// or E4M3 with one fp32 scale per 128 columns.  The gate/up pass stores
// SiLU(z_gate) z_up, the other passes w_t z + add.
#include <cuda_fp16.h>

#include "common.cuh"
#include "internal.h"

namespace fgs {
namespace {

constexpr int kChunk = 128;       // columns of one packed record
constexpr int kBlockRows = 16;    // rows of one packed record
constexpr int kCodeBytes = kChunk * kBlockRows / 2;

__host__ __device__ constexpr int record_bytes(int group) {
  return kCodeBytes + kBlockRows * (kChunk / group) * 2;
}

// ------------------------------------------------------------------ packing
// One warp a record.  Lane l = 4 g + c holds, in word i, the A fragment that
// m16n8k16 takes for the columns 32 (i / 2) + 8 c + 4 (i % 2) + {0, 1, 2, 3}:
// nibble j and nibble j + 4 are the two values of fragment register j (rows
// g, g + 8, g, g + 8; the first column pair for j < 2, the second otherwise).
// The columns are dealt to lanes so that a lane's values of x for 32 columns
// are eight neighbours, one 16-byte load of a bf16 row.
__global__ void pack_int4_kernel(const uint8_t* __restrict__ codes,
                                 const __nv_bfloat16* __restrict__ scales,
                                 uint8_t* __restrict__ dst, int64_t records, int64_t rows,
                                 int64_t cols, int group, int gate_up) {
  const int64_t rec = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
  if (rec >= records) return;
  const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  const int64_t nch = cols / kChunk, nb = rows / kBlockRows;
  const int64_t chunk = rec % nch, block = rec / nch % nb, grp = rec / (nch * nb);
  const int64_t half = rows / 2;
  auto src_row = [&](int r) {  // row of the bank behind row r of the record
    if (!gate_up) return grp * rows + block * kBlockRows + r;
    return grp * rows + (r < 8 ? 0 : half) + block * 8 + (r & 7);
  };
  uint8_t* out = dst + rec * record_bytes(group);
  for (int i = 0; i < 8; ++i) {
    uint32_t w = 0;
    for (int j = 0; j < 4; ++j) {
      const int64_t row = src_row(g + 8 * (j & 1));
      const int64_t col = chunk * kChunk + 32 * (i >> 1) + 8 * c + 4 * (i & 1) + 2 * (j >> 1);
      const uint32_t b = codes[(row * cols + col) >> 1];
      w |= (b & 15u) << (4 * j) | (b >> 4) << (4 * j + 16);
    }
    *reinterpret_cast<uint32_t*>(out + (i >> 2) * 512 + lane * 16 + (i & 3) * 4) = w;
  }
  // scales: per g, the groups of row g and then those of row g + 8
  const int per = kChunk / group;
  __nv_bfloat16* so = reinterpret_cast<__nv_bfloat16*>(out + kCodeBytes);
  for (int i = lane; i < kBlockRows * per; i += 32) {
    const int gi = i / (2 * per), rest = i % (2 * per);
    const int64_t row = src_row(gi + 8 * (rest / per));
    so[i] = scales[row * (cols / group) + chunk * per + rest % per];
  }
}

// ------------------------------------------------------------- device parts
// The four fragment registers of one word of codes, as bf16 (or f16) c - 8:
// a nibble or'ed into the mantissa of 128 (1024) is 128 + c (1024 + c), and
// the subtraction of 136 (1032) is exact.
template <bool kHalf>
__device__ __forceinline__ void dequant(uint32_t w, uint32_t (&a)[4]) {
  const uint32_t magic = kHalf ? 0x64006400u : 0x43004300u;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t v = ((w >> (4 * j)) & 0x000f000fu) | magic;
    if (kHalf) {
      asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(a[j]) : "r"(v), "r"(0x64086408u));
    } else {
      asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(a[j]) : "r"(v), "r"(0x43084308u));
    }
  }
}

template <bool kHalf>
__device__ __forceinline__ void mma(float (&p)[4], const uint32_t (&a)[4], uint32_t b0,
                                    uint32_t b1) {
  if (kHalf)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(p[0]), "+f"(p[1]), "+f"(p[2]), "+f"(p[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(p[0]), "+f"(p[1]), "+f"(p[2]), "+f"(p[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
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

// Simple form: a warp a row block, eight tokens at a time, everything read
// from global memory.
template <bool kSwiglu, bool kX8, int kGroup>
__global__ void __launch_bounds__(256) gemv_int4_kernel(Int4Segment s) {
  pdl_wait();
  const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  const int block = blockIdx.x * (blockDim.x / 32) + (threadIdx.x >> 5);
  const int grp = blockIdx.y;
  if (block >= s.blocks) return;
  int64_t first = 0;
  int64_t n = s.rows;
  if (s.offsets) {
    first = s.offsets[grp];
    n = s.offsets[grp + 1] - first;
  }
  const uint8_t* W = s.W + (static_cast<int64_t>(grp) * s.blocks + block) * s.chunks *
                               record_bytes(kGroup);
  for (int64_t t0 = 0; t0 < n; t0 += 8) {
    const int64_t t = t0 + g;
    const bool live = t < n;
    int64_t src = 0;
    if (live) {
      src = s.offsets ? first + t : grp * s.x_group_rows + t;
      if (s.perm) src = s.perm[src] / s.perm_div;
    }
    float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int ch = 0; ch < s.chunks; ++ch) {
      const uint8_t* rec = W + static_cast<int64_t>(ch) * record_bytes(kGroup);
      const uint4 w0 = *reinterpret_cast<const uint4*>(rec + lane * 16);
      const uint4 w1 = *reinterpret_cast<const uint4*>(rec + 512 + lane * 16);
      const uint32_t words[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
      float q[4] = {0.0f, 0.0f, 0.0f, 0.0f};
      for (int kk = 0; kk < 4; ++kk) {
        uint4 x = make_uint4(0u, 0u, 0u, 0u);
        if (live) {
          const int64_t at = src * s.x_ld + ch * kChunk + kk * 32 + c * 8;
          if (kX8)
            x = e4m3x8_to_f16(*reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(s.x) + at));
          else
            x = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(s.x) + at);
        }
        float p[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        uint32_t a[4];
        dequant<kX8>(words[2 * kk], a);
        mma<kX8>(p, a, x.x, x.y);
        dequant<kX8>(words[2 * kk + 1], a);
        mma<kX8>(p, a, x.z, x.w);
        const __nv_bfloat16* sc = reinterpret_cast<const __nv_bfloat16*>(rec + kCodeBytes);
        constexpr int per = kChunk / kGroup;
        const float s0 = __bfloat162float(sc[g * 2 * per + (kGroup == 32 ? kk : 0)]);
        const float s1 = __bfloat162float(sc[g * 2 * per + per + (kGroup == 32 ? kk : 0)]);
        q[0] = fmaf(s0, p[0], q[0]);
        q[1] = fmaf(s0, p[1], q[1]);
        q[2] = fmaf(s1, p[2], q[2]);
        q[3] = fmaf(s1, p[3], q[3]);
      }
      for (int j = 0; j < 4; ++j) {
        float f = 1.0f;
        const int64_t tt = t0 + 2 * c + (j & 1);
        if (kX8 && tt < n) {
          int64_t r = s.offsets ? first + tt : grp * s.x_group_rows + tt;
          if (s.perm) r = s.perm[r] / s.perm_div;
          f = s.x_scale[r * s.chunks + ch];
        }
        acc[j] = fmaf(f, q[j], acc[j]);
      }
    }
    for (int j = 0; j < 2; ++j) {
      const int64_t tt = t0 + 2 * c + j;
      if (tt >= n) continue;
      const int64_t r = s.offsets ? first + tt : grp * s.out_group_rows + tt;
      if (kSwiglu) {
        s.out[r * s.out_ld + block * 8 + g] = __float2bfloat16_rn(silu_f(acc[j]) * acc[j + 2]);
      } else {
        const float w = s.row_w ? s.row_w[s.row_perm[r]] : 1.0f;
        for (int i = 0; i < 2; ++i) {
          const int64_t o = block * 16 + g + 8 * i;
          float v = w * acc[j + 2 * i];
          if (s.add) v += __bfloat162float(s.add[r * s.out_ld + o]);
          s.out[r * s.out_ld + o] = __float2bfloat16_rn(v);
        }
      }
    }
  }
}

template <bool kSwiglu, bool kX8>
cudaError_t launch_segment(const Int4Segment& s, int group, cudaStream_t stream) {
  const dim3 grid((s.blocks + 7) / 8, s.groups);
  if (group == 32) return launch_pdl(gemv_int4_kernel<kSwiglu, kX8, 32>, grid, dim3(256), 0, stream, s);
  return launch_pdl(gemv_int4_kernel<kSwiglu, kX8, 128>, grid, dim3(256), 0, stream, s);
}

}  // namespace

int64_t packed_int4_bytes(int64_t groups, int64_t rows, int64_t cols, int group) {
  return groups * (rows / kBlockRows) * (cols / kChunk) * record_bytes(group);
}

cudaError_t launch_pack_int4(int gate_up, int64_t groups, int64_t rows, int64_t cols, int group,
                             const void* codes, const void* scales, void* dst,
                             cudaStream_t stream) {
  const int64_t records = groups * (rows / kBlockRows) * (cols / kChunk);
  note_launch();
  pack_int4_kernel<<<static_cast<unsigned>((records + 7) / 8), 256, 0, stream>>>(
      static_cast<const uint8_t*>(codes), static_cast<const __nv_bfloat16*>(scales),
      static_cast<uint8_t*>(dst), records, rows, cols, group, gate_up);
  return cudaGetLastError();
}

cudaError_t launch_gemv_int4(const Int4Params& p, int, cudaStream_t stream) {
  for (int i = 0; i < p.nseg; ++i) {
    const Int4Segment& s = p.seg[i];
    cudaError_t e;
    if (p.swiglu)
      e = s.x_scale ? launch_segment<true, true>(s, p.group, stream)
                    : launch_segment<true, false>(s, p.group, stream);
    else
      e = s.x_scale ? launch_segment<false, true>(s, p.group, stream)
                    : launch_segment<false, false>(s, p.group, stream);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace fgs
