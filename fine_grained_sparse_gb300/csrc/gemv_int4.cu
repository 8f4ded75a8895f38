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
// The four fragment registers of one word of codes, as f16 pairs.  A nibble
// in the low four bits of an f16 is c 2^-24 (a subnormal), in the next four
// c 2^-20, and subtracting 8 of the same unit is exact: registers 0 and 2
// hold (c - 8) 2^-24, registers 1 and 3 (c - 8) 2^-20.  Those are rows g and
// g + 8, whose sums are scaled back when a block is done.  Nine operations
// for eight weights; through bf16 (whose seven mantissa bits take a nibble in
// one place only, beside 128) it is eleven, and the products of a full stream
// of records ran at 5.3 TB/s instead of 6.9.
__device__ __forceinline__ void dequant(uint32_t w, uint32_t (&a)[4]) {
  a[0] = w & 0x000f000fu;
  a[1] = w & 0x00f000f0u;
  w >>= 8;
  a[2] = w & 0x000f000fu;
  a[3] = w & 0x00f000f0u;
#pragma unroll
  for (int j = 0; j < 4; ++j)
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(a[j]) : "r"(a[j]), "r"(j & 1 ? 0x00800080u : 0x00080008u));
}

// D = A B and D += A B on 16 rows x 16 columns x 8 tokens.
__device__ __forceinline__ void mma_first(float (&p)[4], const uint32_t (&a)[4], uint32_t b0,
                                          uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%10, %10, %10, %10};"
      : "=f"(p[0]), "=f"(p[1]), "=f"(p[2]), "=f"(p[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.0f));
}
__device__ __forceinline__ void mma(float (&p)[4], const uint32_t (&a)[4], uint32_t b0,
                                    uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
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

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

// ------------------------------------------------------------------- kernel
constexpr int kWarps = 16;
constexpr int kThreads = 32 * kWarps;
constexpr int kDepth = 4;    // records of a warp's ring in shared memory
constexpr int kMaxTile = 32;  // tokens of one pass over the weights
constexpr int kSmem = 227 * 1024;
constexpr int kSlotBytes = kWarps * 32 * 16;  // partial sums, per eight tokens

// One tile of tokens of one group against the CTA's blocks of that group.
struct Tile {
  const uint8_t* W;   // first record of the range
  int64_t out_row;    // output row of token 0
  int64_t x_row;      // row of x (or of perm) of token 0
  int seg;            // segment, or -1: no tile left
  int blocks;         // 16-row blocks of the range
  int first_block;    // the range's first block within the group
  int n;              // tokens
};

// Shared memory: the header (the tile at hand, row weights, the scan's warp
// sums, group costs [groups + 1]), each warp's ring of records, partial sums,
// x (256-byte aligned) and the scales of x.
struct Header {
  Tile tile;
  int next_group, next_tile;
  float row_w[kMaxTile];
  int64_t warp_sum[kWarps];
  int64_t prefix[1];
};

__host__ __device__ inline int header_bytes(int groups) {
  return static_cast<int>(sizeof(Header) + 8 * groups + 255) / 256 * 256;
}

// A token's x as f16 and one fp32 scale per 128 columns.
__host__ __device__ inline int x_row_bytes(int chunks) { return chunks * kChunk * 2; }

// The most tokens of one tile: partial sums for them and their rows fit.
inline int tile_cap(int groups, int chunks, int group) {
  const int room = kSmem - header_bytes(groups) - kWarps * kDepth * record_bytes(group);
  int cap = 0;
  for (int j = 1; j <= kMaxTile / 8; ++j) {
    const int n = (room - j * kSlotBytes - 4 * 8 * j * chunks - 256) / x_row_bytes(chunks);
    const int m = n < 8 * j ? n : 8 * j;
    cap = m > cap ? m : cap;
  }
  return cap;
}

// Time of a record against 1 .. 4 times eight tokens, in quarters of the
// smallest.
__device__ __forceinline__ int64_t record_cost(int tile) {
  return tile <= 8 ? 4 : tile <= 16 ? 5 : tile <= 24 ? 6 : 8;
}

// acc += the record's 16 rows x 128 columns times 8 J tokens.  r: the record
// in shared memory at this lane's codes, rs: at its scales; x: this lane's
// bytes of the 128 columns of token g (token j's are jb bytes further); xs:
// the chunk's scales of tokens 2 c and 2 c + 1.  Tokens beyond the tile's are
// copies of its last one: their columns of the product are never stored.
template <int J, int kGroup>
__device__ __forceinline__ void multiply_record(float (&acc)[J][4], const uint8_t* smem,
                                                uint32_t r, uint32_t rs, const uint32_t (&x)[J],
                                                uint32_t xs) {
  const uint4 w0 = *reinterpret_cast<const uint4*>(smem + r);
  const uint4 w1 = *reinterpret_cast<const uint4*>(smem + r + 512);
  const uint32_t words[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
  uint4 sv = make_uint4(0u, 0u, 0u, 0u);
  if (kGroup == 32)
    sv = *reinterpret_cast<const uint4*>(smem + rs);
  else
    sv.x = *reinterpret_cast<const uint32_t*>(smem + rs);
  const uint32_t sc[4] = {sv.x, sv.y, sv.z, sv.w};
  float q[J][4];
#pragma unroll
  for (int kk = 0; kk < 4; ++kk) {
    uint32_t a0[4], a1[4];
    dequant(words[2 * kk], a0);
    dequant(words[2 * kk + 1], a1);
    // scales: words 0 and 1 hold row g's four groups, words 2 and 3 row
    // g + 8's; groups of 128: one word with both rows' scales
    const uint32_t lo = sc[kk >> 1], hi = sc[2 + (kk >> 1)];
    const float s0 = __uint_as_float(kk & 1 ? lo & 0xffff0000u : lo << 16);
    const float s1 = __uint_as_float(kk & 1 ? hi & 0xffff0000u : hi << 16);
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const uint4 v = *reinterpret_cast<const uint4*>(smem + (x[j] ^ (kk << 6)));
      if (kGroup == 128) {  // one sum over the record
        if (kk == 0)
          mma_first(q[j], a0, v.x, v.y);
        else
          mma(q[j], a0, v.x, v.y);
        mma(q[j], a1, v.z, v.w);
        continue;
      }
      float p[4];
      mma_first(p, a0, v.x, v.y);
      mma(p, a1, v.z, v.w);
      if (kk == 0) {
        q[j][0] = s0 * p[0];
        q[j][1] = s0 * p[1];
        q[j][2] = s1 * p[2];
        q[j][3] = s1 * p[3];
      } else {
        q[j][0] = fmaf(s0, p[0], q[j][0]);
        q[j][1] = fmaf(s0, p[1], q[j][1]);
        q[j][2] = fmaf(s1, p[2], q[j][2]);
        q[j][3] = fmaf(s1, p[3], q[j][3]);
      }
    }
  }
#pragma unroll
  for (int j = 0; j < J; ++j) {
    const float2 f = *reinterpret_cast<const float2*>(smem + xs + 32 * j);
    if (kGroup == 128) {
      const float s0 = __uint_as_float(sc[0] << 16), s1 = __uint_as_float(sc[0] & 0xffff0000u);
      q[j][0] *= s0;
      q[j][1] *= s0;
      q[j][2] *= s1;
      q[j][3] *= s1;
    }
    acc[j][0] = fmaf(f.x, q[j][0], acc[j][0]);
    acc[j][1] = fmaf(f.y, q[j][1], acc[j][1]);
    acc[j][2] = fmaf(f.x, q[j][2], acc[j][2]);
    acc[j][3] = fmaf(f.y, q[j][3], acc[j][3]);
  }
}

// What brings the sums of rows g and g + 8 back to units of 1: the codes are
// in units of 2^-24 and 2^-20, the scales of x 2^12 too large (half of the
// factor there and half here, so that neither small nor large values leave
// fp32's range).
constexpr float kUnitX = 4096.0f, kUnitLow = 4096.0f, kUnitHigh = 256.0f;

template <int J, bool kSwiglu>
__device__ __forceinline__ void store_block(const Int4Segment& s, const Header* hd,
                                            const float (&acc)[J][4], int block, int g, int c) {
  const int n = hd->tile.n;
#pragma unroll
  for (int j = 0; j < J; ++j) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int t = 8 * j + 2 * c + h;
      if (t >= n) continue;
      const int64_t r = (hd->tile.out_row + t) * s.out_ld;
      const float z[2] = {acc[j][h] * kUnitLow, acc[j][2 + h] * kUnitHigh};
      if (kSwiglu) {
        // H is rounded to bf16, the type of the layer's activations
        s.out[r + block * 8 + g] = __float2bfloat16_rn(silu_f(z[0]) * z[1]);
      } else {
        const float w = s.row_w ? hd->row_w[t] : 1.0f;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int64_t o = r + block * 16 + g + 8 * i;
          float v = w * z[i];
          if (s.add) v += __bfloat162float(s.add[o]);
          s.out[o] = __float2bfloat16_rn(v);
        }
      }
    }
  }
}

// The tile's rows of x into shared memory as f16 (row t at xo + t row_bytes)
// with one fp32 factor per 128 columns (at fo, [chunk][8 J tokens]), and its
// row weights.  A half warp takes 128 columns.  bf16 values are scaled by the
// power of two that brings the largest of them to [2^14, 2^15): exact for
// every value above 2^-29 of it, and within 2^-40 of it below.  E4M3 values
// are exact.  Pieces of a row are moved within 128 bytes by the row's number
// (16-byte piece q of a chunk to q ^ 4 (t & 1)), so that a fragment load of
// eight tokens meets every bank once.
template <bool kX8>
__device__ __forceinline__ void load_x(const Int4Segment& s, uint8_t* smem, uint32_t xo,
                                       uint32_t fo, int j8) {
  Header* hd = reinterpret_cast<Header*>(smem);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int n = hd->tile.n, chunks = s.chunks, piece = lane & 15;
  int64_t src = 0;
  if (lane < n) {
    src = hd->tile.x_row + lane;
    if (warp == 0 && s.row_w) hd->row_w[lane] = s.row_w[s.row_perm[hd->tile.out_row + lane]];
    if (s.perm) src = s.perm[src] / s.perm_div;
  }
  constexpr int kAhead = 4;  // loads in flight
  const int tasks = n * chunks;
  for (int base = 2 * warp; base < tasks; base += 2 * kWarps * kAhead) {
    uint4 v[kAhead];
    float f[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int task = min(base + 2 * kWarps * u + (lane >> 4), tasks - 1);
      const int row = task / chunks, ch = task - row * chunks;
      const int64_t from = __shfl_sync(0xffffffffu, src, row);
      if (kX8) {
        const uint2 b = *reinterpret_cast<const uint2*>(
            static_cast<const uint8_t*>(s.x) + (from * chunks + ch) * kChunk + piece * 8);
        v[u].x = b.x;
        v[u].y = b.y;
        f[u] = s.x_scale[from * chunks + ch];
      } else {
        v[u] = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(s.x) +
                                               (from * chunks + ch) * kChunk + piece * 8);
      }
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int task = base + 2 * kWarps * u + (lane >> 4);
      if (base + 2 * kWarps * u >= tasks) break;
      const int row = task / chunks, ch = task - row * chunks;
      if (kX8) {
        v[u] = e4m3x8_to_f16(make_uint2(v[u].x, v[u].y));
        f[u] *= kUnitX;
      } else {
        uint32_t w[4] = {v[u].x, v[u].y, v[u].z, v[u].w}, m = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) m = __vmaxu2(m, w[i] & 0x7fff7fffu);
#pragma unroll
        for (int o = 8; o; o >>= 1) m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, o));
        m = max(m & 0xffffu, m >> 16);
        // the exponent of the largest value; an infinity or NaN counts as the
        // largest finite one, and tiny maxima are left small
        const uint32_t e = min(max(m >> 7, 15u), 254u);
        const float up = __uint_as_float((268u - e) << 23);  // 2^(141 - e)
        f[u] = __uint_as_float((e - 2u) << 23);              // 2^(e - 141) 2^12
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float lo = __uint_as_float(w[i] << 16) * up;
          const float hi = __uint_as_float(w[i] & 0xffff0000u) * up;
          asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(hi), "f"(lo));
        }
        v[u] = make_uint4(w[0], w[1], w[2], w[3]);
      }
      if (task < tasks) {
        *reinterpret_cast<uint4*>(smem + xo + (row * chunks + ch) * (2 * kChunk) +
                                  ((piece ^ ((row & 1) << 2)) << 4)) = v[u];
        if (piece == 0) *reinterpret_cast<float*>(smem + fo + (ch * j8 + row) * 4) = f[u];
      }
    }
  }
}

// The tile's blocks x chunks records, dealt evenly to the warps as one
// sequence; a block cut by a warp boundary is summed from its pieces, in
// warp order, by the first warp that starts inside it.
template <int J, bool kSwiglu, bool kX8, int kGroup>
__device__ __forceinline__ void run_tile(const Int4Segment& s, uint8_t* smem, int header) {
  constexpr int kRec = record_bytes(kGroup);
  Header* hd = reinterpret_cast<Header*>(smem);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, c = lane & 3;
  const int nch = s.chunks;
  const uint32_t ring = header + warp * kDepth * kRec;
  const uint32_t so = header + kWarps * kDepth * kRec;
  const uint32_t fo = so + J * kSlotBytes;
  const uint32_t xo = (fo + 32 * J * nch + 255u) & ~255u;
  const int64_t total = static_cast<int64_t>(hd->tile.blocks) * nch;
  const int64_t a = total * warp / kWarps;
  const int count = static_cast<int>(total * (warp + 1) / kWarps - a);
  // The ring is filled kDepth - 1 records ahead; past the end the last
  // record is read again, so that every step waits for the same number.
  const uint8_t* w = hd->tile.W + a * kRec + lane * 16;
  const int last = max(count - 1, 0) * kRec;
  auto fetch = [&](uint32_t slot, int at) {
    const uint32_t to = smem_u32(smem + slot) + lane * 16;
    cp_async16(to, w + at);
    cp_async16(to + 512, w + at + 512);
    if (lane < (kRec - kCodeBytes) / 16) cp_async16(to + kCodeBytes, w + at + kCodeBytes);
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  if (count > 0) {
#pragma unroll
    for (int u = 0; u < kDepth - 1; ++u) fetch(ring + u * kRec, min(u * kRec, last));
  }
  load_x<kX8>(s, smem, xo, fo, 8 * J);
  __syncthreads();

  int block = static_cast<int>(a / nch), ch = static_cast<int>(a - static_cast<int64_t>(block) * nch);
  bool mid = ch != 0;  // the piece at hand began inside its block
  uint32_t x[J], xs = fo + ch * 32 * J + c * 8;
#pragma unroll
  for (int j = 0; j < J; ++j) {
    const int t = min(8 * j + g, hd->tile.n - 1);
    x[j] = xo + (t * nch + ch) * (2 * kChunk) + ((t & 1) << 6) + c * 16;
  }
  float acc[J][4];
#pragma unroll
  for (int j = 0; j < J; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[j][i] = 0.0f;
  auto put = [&](uint32_t at) {
    float* o = reinterpret_cast<float*>(smem + at) + lane;
#pragma unroll
    for (int j = 0; j < J; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) o[(4 * j + i) * 32] = acc[j][i];
  };
  const uint32_t first_slot = so + warp * J * 512;  // a piece that began inside its block
  uint32_t rd = ring, wr = ring + (kDepth - 1) * kRec;
  int ahead = (kDepth - 1) * kRec;
#pragma unroll 1
  for (int i = 0; i < count; ++i) {
    asm volatile("cp.async.wait_group %0;" ::"n"(kDepth - 2) : "memory");
    __syncwarp();  // the record is there, and the one before it was read by all
    fetch(wr, min(ahead, last));
    ahead += kRec;
    multiply_record<J, kGroup>(acc, smem, rd + lane * 16,
                               rd + kCodeBytes + g * (kGroup == 32 ? 16 : 4), x, xs);
    wr = rd;
    rd += kRec;
    if (rd == ring + kDepth * kRec) rd = ring;
    xs += 32 * J;
#pragma unroll
    for (int j = 0; j < J; ++j) x[j] += 2 * kChunk;
    if (++ch == nch) {
      if (mid)
        put(first_slot);
      else
        store_block<J, kSwiglu>(s, hd, acc, hd->tile.first_block + block, g, c);
      mid = false;
      ch = 0;
      ++block;
      xs -= 32 * J * nch;
#pragma unroll
      for (int j = 0; j < J; ++j) {
        x[j] -= 2 * kChunk * nch;
#pragma unroll
        for (int k = 0; k < 4; ++k) acc[j][k] = 0.0f;
      }
    }
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  __syncwarp();
  // a piece that ends inside its block: its sums go where the ring was,
  // unless it also began there
  if (ch != 0 && count > 0) put(mid ? first_slot : ring);
  __syncthreads();
  if (warp > 0 && a % nch != 0) {
    const int64_t r = a / nch;
    if (total * (warp - 1) / kWarps <= r * nch) {
      auto slot = [&](uint32_t at) { return reinterpret_cast<const float*>(smem + at) + lane; };
      const float* p = slot(ring - kDepth * kRec);
#pragma unroll
      for (int j = 0; j < J; ++j)
#pragma unroll
        for (int k = 0; k < 4; ++k) acc[j][k] = p[(4 * j + k) * 32];
      for (int v = warp; v < kWarps; ++v) {
        const int64_t lo = total * v / kWarps, hi = total * (v + 1) / kWarps;
        if (lo >= (r + 1) * nch) break;
        if (lo == hi) continue;
        const float* o = slot(so + v * J * 512);
#pragma unroll
        for (int j = 0; j < J; ++j)
#pragma unroll
          for (int k = 0; k < 4; ++k) acc[j][k] += o[(4 * j + k) * 32];
      }
      store_block<J, kSwiglu>(s, hd, acc, hd->tile.first_block + static_cast<int>(r), g, c);
    }
  }
}

// The same out of line, so that each J keeps its registers to itself.
template <int J, bool kSwiglu, bool kX8, int kGroup>
__device__ __noinline__ void run_tile_call(const Int4Segment& s, uint8_t* smem, int header) {
  run_tile<J, kSwiglu, kX8, kGroup>(s, smem, header);
}

struct Int4Launch {
  Int4Segment seg[2];
  int nseg;
  int cap[2];  // tokens of a tile
};

// Rows of group k (groups of the second segment after the first's) and where
// they begin.
__device__ __forceinline__ int64_t rows_of(const Int4Launch& p, int k, int64_t& first) {
  const Int4Segment& s = p.seg[k >= p.seg[0].groups];
  first = 0;
  if (!s.offsets) return s.rows;
  first = s.offsets[k];
  return s.offsets[k + 1] - first;
}

// Tiles of a group of n rows of segment i, and what one block of a tile costs.
__device__ __forceinline__ int tiles_of(const Int4Launch& p, int i, int64_t n, int64_t& cost) {
  const int tiles = static_cast<int>((n + p.cap[i] - 1) / p.cap[i]);
  cost = n > 0 ? record_cost(static_cast<int>((n + tiles - 1) / tiles)) * p.seg[i].chunks : 0;
  return tiles;
}

// One thread: the CTA's next tile into the header.  Blocks (of every tile of
// every group, in order) are dealt to the CTAs by cost: a block belongs to
// the CTA in whose share [lo, hi) of the total it begins.
__device__ __noinline__ void next_tile(const Int4Launch& p, Header* hd, int groups, int rec) {
  const int64_t total = hd->prefix[groups];
  const int64_t lo = total * blockIdx.x / gridDim.x, hi = total * (blockIdx.x + 1) / gridDim.x;
  int k = hd->next_group, t = hd->next_tile;
  if (k < 0) {  // first call: the last group that begins at or before lo
    int k1 = groups;
    k = 0;
    while (k1 - k > 1) {
      const int m = (k + k1) / 2;
      if (hd->prefix[m] <= lo)
        k = m;
      else
        k1 = m;
    }
  }
  hd->tile.seg = -1;
  for (; k < groups && hd->prefix[k] < hi; ++k, t = -1) {
    if (hd->prefix[k + 1] <= lo || hd->prefix[k + 1] == hd->prefix[k]) continue;
    const int i = k >= p.seg[0].groups;
    const Int4Segment& s = p.seg[i];
    const int grp = i ? k - p.seg[0].groups : k;
    int64_t first, w;
    const int64_t n = rows_of(p, k, first);
    const int tiles = tiles_of(p, i, n, w);
    const int64_t tile_cost = w * s.blocks;
    if (t < 0) t = lo > hd->prefix[k] ? static_cast<int>((lo - hd->prefix[k]) / tile_cost) : 0;
    for (; t < tiles; ++t) {
      const int64_t base = hd->prefix[k] + t * tile_cost;
      if (base >= hi) break;
      const int64_t r0 = lo > base ? (lo - base + w - 1) / w : 0;
      int64_t r1 = (hi - base + w - 1) / w;
      if (r1 > s.blocks) r1 = s.blocks;
      if (r0 >= r1) continue;
      const int64_t row0 = n * t / tiles;
      Tile& T = hd->tile;
      T.seg = i;
      T.W = s.W + (static_cast<int64_t>(grp) * s.blocks + r0) * s.chunks * rec;
      T.blocks = static_cast<int>(r1 - r0);
      T.first_block = static_cast<int>(r0);
      T.n = static_cast<int>(n * (t + 1) / tiles - row0);
      T.out_row = row0 + (s.offsets ? first : grp * s.out_group_rows);
      T.x_row = row0 + (s.offsets ? first : grp * s.x_group_rows);
      hd->next_group = k;
      hd->next_tile = t + 1;
      return;
    }
  }
}

// kSmall: no tile has more than eight tokens.
template <bool kSwiglu, bool kX8, int kGroup, bool kSmall>
__global__ void __launch_bounds__(kThreads, 1) gemv_int4_kernel(const __grid_constant__ Int4Launch p) {
  extern __shared__ __align__(1024) uint8_t smem[];
  Header* hd = reinterpret_cast<Header*>(smem);
  const int groups = p.seg[0].groups + (p.nseg > 1 ? p.seg[1].groups : 0);
  const int header = header_bytes(groups);
  pdl_wait();
  {  // prefix[k] = cost of the groups before k
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = (groups + kThreads - 1) / kThreads;
    auto cost = [&](int k) {
      const int i = k >= p.seg[0].groups;
      int64_t first, w;
      const int tiles = tiles_of(p, i, rows_of(p, k, first), w);
      return w * tiles * p.seg[i].blocks;
    };
    int64_t mine = 0;
    for (int k = tid * per; k < (tid + 1) * per && k < groups; ++k) mine += cost(k);
    int64_t incl = mine;
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    if (lane == 31) hd->warp_sum[warp] = incl;
    __syncthreads();
    int64_t at = incl - mine;
    for (int v = 0; v < warp; ++v) at += hd->warp_sum[v];
    for (int k = tid * per; k < (tid + 1) * per && k < groups; ++k) {
      hd->prefix[k] = at;
      at += cost(k);
      if (k == groups - 1) hd->prefix[groups] = at;
    }
    if (tid == 0) hd->next_group = hd->next_tile = -1;
  }
  for (;;) {
    __syncthreads();  // the tile before this one is done with shared memory
    if (threadIdx.x == 0) next_tile(p, hd, groups, record_bytes(kGroup));
    __syncthreads();
    if (hd->tile.seg < 0) break;
    const Int4Segment& s = p.seg[hd->tile.seg];
    if (kSmall) {
      run_tile<1, kSwiglu, kX8, kGroup>(s, smem, header);
      continue;
    }
    switch ((hd->tile.n + 7) / 8) {
      case 1: run_tile_call<1, kSwiglu, kX8, kGroup>(s, smem, header); break;
      case 2: run_tile_call<2, kSwiglu, kX8, kGroup>(s, smem, header); break;
      case 3: run_tile_call<3, kSwiglu, kX8, kGroup>(s, smem, header); break;
      default: run_tile_call<4, kSwiglu, kX8, kGroup>(s, smem, header); break;
    }
  }
}

template <bool kSwiglu, bool kX8, int kGroup, bool kSmall>
cudaError_t launch_kernel(const Int4Launch& p, int num_sms, cudaStream_t stream) {
  static int configured[64] = {0};
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  if (dev >= 64 || !configured[dev]) {
    err = cudaFuncSetAttribute(gemv_int4_kernel<kSwiglu, kX8, kGroup, kSmall>,
                               cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (err != cudaSuccess) return err;
    if (dev < 64) configured[dev] = 1;
  }
  return launch_pdl(gemv_int4_kernel<kSwiglu, kX8, kGroup, kSmall>, dim3(num_sms), dim3(kThreads), kSmem,
                    stream, p);
}

template <bool kSwiglu, bool kX8>
cudaError_t launch_group(Int4Launch& p, int group, int num_sms, cudaStream_t stream) {
  bool small = true;
  for (int i = 0; i < p.nseg; ++i) small = small && (p.seg[i].rows <= 8 || p.cap[i] <= 8);
  if (small)  // a group with more rows than the bound says is still cut into tiles of eight
    for (int i = 0; i < p.nseg; ++i) p.cap[i] = p.cap[i] < 8 ? p.cap[i] : 8;
  if (small)
    return group == 32 ? launch_kernel<kSwiglu, kX8, 32, true>(p, num_sms, stream)
                       : launch_kernel<kSwiglu, kX8, 128, true>(p, num_sms, stream);
  return group == 32 ? launch_kernel<kSwiglu, kX8, 32, false>(p, num_sms, stream)
                     : launch_kernel<kSwiglu, kX8, 128, false>(p, num_sms, stream);
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

cudaError_t launch_gemv_int4(const Int4Params& p, int num_sms, cudaStream_t stream) {
  Int4Launch l;
  l.nseg = p.nseg;
  int groups = 0;
  for (int i = 0; i < p.nseg; ++i) groups += p.seg[i].groups;
  const bool x8 = p.seg[0].x_scale != nullptr;
  for (int i = 0; i < p.nseg; ++i) {
    l.seg[i] = p.seg[i];
    l.cap[i] = tile_cap(groups, p.seg[i].chunks, p.group);
    if (l.cap[i] < 1) return cudaErrorInvalidValue;  // the callers' limit on the width
  }
  if (p.swiglu)
    return x8 ? launch_group<true, true>(l, p.group, num_sms, stream)
              : launch_group<true, false>(l, p.group, num_sms, stream);
  return x8 ? launch_group<false, true>(l, p.group, num_sms, stream)
            : launch_group<false, false>(l, p.group, num_sms, stream);
}

}  // namespace fgs
