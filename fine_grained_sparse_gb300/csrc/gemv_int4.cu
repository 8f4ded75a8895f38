// Products of a few rows with 4-bit weights: the decode form of the expert
// passes and of a linear map (MOE_WEIGHTS_PACKED_INT4_*).
//
//   z[t, o] = sum_g s[o, g] sum_{k in group g} (c[o, k] - 8) x[t, k]
//
// c are 4-bit codes, s one bf16 scale per 32 or 128 columns of a row, x bf16
// or E4M3 with one fp32 scale per 128 columns.  The gate/up pass stores
// SiLU(z_gate) z_up, the other passes w_t z + add.
#include "int4.cuh"

namespace fgs {
namespace {

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
  uint32_t words[8];
#pragma unroll
  for (int kk = 0; kk < 4; ++kk) {  // 32 columns, eight of them a lane's
    const int64_t at = chunk * kChunk + 32 * kk + 8 * c;
    const uint32_t v0 = *reinterpret_cast<const uint32_t*>(codes + (src_row(g) * cols + at) / 2);
    const uint32_t v1 = *reinterpret_cast<const uint32_t*>(codes + (src_row(g + 8) * cols + at) / 2);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      // four codes of a row from 16 bits to bits 0, 16, 8 and 24
      const uint32_t a = v0 >> (16 * h), b = v1 >> (16 * h);
      words[2 * kk + h] = (a & 0x0f0fu) | (a & 0xf0f0u) << 12 |
                          ((b & 0x0f0fu) | (b & 0xf0f0u) << 12) << 4;
    }
  }
  *reinterpret_cast<uint4*>(out + lane * 16) = make_uint4(words[0], words[1], words[2], words[3]);
  *reinterpret_cast<uint4*>(out + 512 + lane * 16) =
      make_uint4(words[4], words[5], words[6], words[7]);
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

// ------------------------------------------------------------------- kernel
constexpr int kWarps = 16;
constexpr int kThreads = 32 * kWarps;
constexpr int kDepth = 4;  // records of a warp's ring in shared memory
constexpr int kTile = 8;   // most tokens of one pass over the weights
constexpr int kSmem = 227 * 1024;
constexpr int kSlotBytes = 512;   // a block's sums for kTile tokens
constexpr int kTileCost = 128;    // what beginning a tile costs, in records

// Shared memory: the header (row weights of the tile, the scan's warp sums,
// the CTA's first group, the group lists), each warp's ring of records,
// partial sums, the scales of x and (256-byte aligned) x.
struct Header {
  float row_w[kTile];
  int64_t warp_sum[kWarps];
  int at_first, pad;
  int64_t lists[1];
};

__host__ __device__ inline int header_bytes(int groups) {
  return static_cast<int>(sizeof(Header) + group_list_bytes(groups) + 255) / 256 * 256;
}

// A token's x as f16, and fp32 scales of kTile tokens per 128 columns.
__host__ __device__ inline int x_row_bytes(int chunks) { return chunks * kChunk * 2; }
__host__ __device__ inline int x_scale_bytes(int chunks) { return chunks * kTile * 4; }

// Shared memory beside the tile's rows of x, and the most tokens of a tile.
inline int fixed_smem(int groups, int chunks, int group) {
  return header_bytes(groups) + kWarps * (kDepth * record_bytes(group) + kSlotBytes) +
         x_scale_bytes(chunks) + 256;
}
inline int tile_cap(int groups, int chunks, int group) {
  const int n = (kSmem - fixed_smem(groups, chunks, group)) / x_row_bytes(chunks);
  return n < kTile ? n : kTile;
}

// acc += the record's 16 rows x 128 columns times eight tokens.  r: the
// record in shared memory at this lane's codes, rs: at its scales; x: this
// lane's bytes of the 128 columns of token g; xs: the chunk's scales of
// tokens 2 c and 2 c + 1.  Tokens beyond the tile's are copies of its last
// one: their columns of the product are never stored.
template <int kGroup>
__device__ __forceinline__ void multiply_record(float (&acc)[4], const uint8_t* smem, uint32_t r,
                                                uint32_t rs, uint32_t x, uint32_t xs) {
  const uint4 w0 = *reinterpret_cast<const uint4*>(smem + r);
  const uint4 w1 = *reinterpret_cast<const uint4*>(smem + r + 512);
  const uint32_t words[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
  uint4 sv = make_uint4(0u, 0u, 0u, 0u);
  if (kGroup == 32)
    sv = *reinterpret_cast<const uint4*>(smem + rs);
  else
    sv.x = *reinterpret_cast<const uint32_t*>(smem + rs);
  const uint32_t sc[4] = {sv.x, sv.y, sv.z, sv.w};
  float q[4];
#pragma unroll
  for (int kk = 0; kk < 4; ++kk) {
    uint32_t a0[4], a1[4];
    dequant(words[2 * kk], a0);
    dequant(words[2 * kk + 1], a1);
    const uint4 v = *reinterpret_cast<const uint4*>(smem + (x ^ (kk << 6)));
    if (kGroup == 128) {  // one sum over the record
      if (kk == 0)
        mma_first(q, a0, v.x, v.y);
      else
        mma(q, a0, v.x, v.y);
      mma(q, a1, v.z, v.w);
      continue;
    }
    // scales: words 0 and 1 hold row g's four groups, words 2 and 3 row g + 8's
    const uint32_t lo = sc[kk >> 1], hi = sc[2 + (kk >> 1)];
    const float s0 = __uint_as_float(kk & 1 ? lo & 0xffff0000u : lo << 16);
    const float s1 = __uint_as_float(kk & 1 ? hi & 0xffff0000u : hi << 16);
    float p[4];
    mma_first(p, a0, v.x, v.y);
    mma(p, a1, v.z, v.w);
    if (kk == 0) {
      q[0] = s0 * p[0];
      q[1] = s0 * p[1];
      q[2] = s1 * p[2];
      q[3] = s1 * p[3];
    } else {
      q[0] = fmaf(s0, p[0], q[0]);
      q[1] = fmaf(s0, p[1], q[1]);
      q[2] = fmaf(s1, p[2], q[2]);
      q[3] = fmaf(s1, p[3], q[3]);
    }
  }
  const float2 f = *reinterpret_cast<const float2*>(smem + xs);
  if (kGroup == 128) {  // one word: row g's scale, then row g + 8's
    const float s0 = __uint_as_float(sc[0] << 16), s1 = __uint_as_float(sc[0] & 0xffff0000u);
    q[0] *= s0;
    q[1] *= s0;
    q[2] *= s1;
    q[3] *= s1;
  }
  acc[0] = fmaf(f.x, q[0], acc[0]);
  acc[1] = fmaf(f.y, q[1], acc[1]);
  acc[2] = fmaf(f.x, q[2], acc[2]);
  acc[3] = fmaf(f.y, q[3], acc[3]);
}

// What brings the sums of rows g and g + 8 back to units of 1: the codes are
// in units of 2^-24 and 2^-20, and part of that is in the factors of x, so
// that neither small nor large values leave fp32's range.  The factors of bf16
// rows are 2^12 too large, the scales of E4M3 rows 2^6 (a group of finite rows
// has a scale below 2^120).
template <bool kX8>
__device__ constexpr float unit_x() { return kX8 ? 0x1p6f : 0x1p12f; }
template <bool kX8>
__device__ constexpr float unit_low() { return 0x1p24f / unit_x<kX8>(); }
template <bool kX8>
__device__ constexpr float unit_high() { return 0x1p20f / unit_x<kX8>(); }

// One tile of tokens of one group against the CTA's blocks of that group.
struct Tile {
  const uint8_t* W;  // first record of the range
  int blocks;        // 16-row blocks of the range
  int first_block;   // the range's first block within the group
  int n;             // tokens
  int64_t out_row;   // output row of token 0
  int64_t x_row;     // row of x (or of perm) of token 0
};

template <bool kSwiglu, bool kX8>
__device__ __forceinline__ void store_block(const Int4Segment& s, const Tile& T, const float* row_w,
                                            const float (&acc)[4], int block, int g, int c) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int t = 2 * c + h;
    if (t >= T.n) continue;
    const int64_t r = (T.out_row + t) * s.out_ld;
    const float z[2] = {acc[h] * unit_low<kX8>(), acc[2 + h] * unit_high<kX8>()};
    if (kSwiglu) {
      // H is rounded to bf16, the type of the layer's activations
      s.out[r + block * 8 + g] = __float2bfloat16_rn(silu_f(z[0]) * z[1]);
    } else {
      const float w = s.row_w ? row_w[t] : 1.0f;
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

// The tile's rows of x into shared memory as f16 (row t at xo + t row bytes)
// with one fp32 factor per 128 columns (at fo, [chunk][kTile]), and its row
// weights.  A half warp takes 128 columns.  bf16 values are scaled by the
// power of two that brings the largest of them to [2^14, 2^15): exact for
// every value above 2^-31 of it, and within 2^-39 of it below.  That is the
// price of f16 fragments (bf16 ones hold every value, at 5.3 instead of 6.9
// TB/s), and 2^-15 of what an fp32 sum loses beside the largest value.  E4M3
// values are exact.  Pieces of a row are moved within 128 bytes by the row's
// number (16-byte piece q of a chunk to q ^ 4 (t & 1)), so that a fragment
// load of eight tokens meets every bank once.
// between() runs after the first loads have been asked for.
template <bool kX8, typename Between>
__device__ __forceinline__ void load_x(const Int4Segment& s, const Tile& T, uint8_t* smem,
                                       uint32_t xo, uint32_t fo, float* row_w, Between between) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int n = T.n, chunks = s.chunks, piece = lane & 15;
  int64_t src = 0;
  int pair = 0;
  const bool weigher = warp == kWarps - 1 && lane < n && s.row_w;
  if (lane < n) {
    src = T.x_row + lane;
    if (weigher) pair = s.row_perm[T.out_row + lane];
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
    if (base == 2 * warp) between();
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int task = base + 2 * kWarps * u + (lane >> 4);
      if (base + 2 * kWarps * u >= tasks) break;
      const int row = task / chunks, ch = task - row * chunks;
      if (kX8) {
        v[u] = e4m3x8_to_f16(make_uint2(v[u].x, v[u].y));
        f[u] *= unit_x<true>();
      } else {
        uint32_t e;
        v[u] = bf16x8_to_f16(v[u], e);
        f[u] = __uint_as_float((e - 2u) << 23);  // 2^(e - 141) 2^12
      }
      if (task < tasks) {
        *reinterpret_cast<uint4*>(smem + xo + (row * chunks + ch) * (2 * kChunk) +
                                  ((piece ^ ((row & 1) << 2)) << 4)) = v[u];
        if (piece == 0) *reinterpret_cast<float*>(smem + fo + (ch * kTile + row) * 4) = f[u];
      }
    }
  }
  if (2 * warp >= tasks) between();
  if (weigher) row_w[lane] = s.row_w[pair];
}

// The tile's blocks x chunks records, dealt evenly to the warps as one
// sequence; a block cut by a warp boundary is summed from its pieces, in
// warp order, by the first warp that starts inside it.
template <bool kSwiglu, bool kX8, int kGroup>
__device__ __forceinline__ void run_tile(const Int4Segment& s, const Divisor& by_chunks,
                                         const Tile& T, uint8_t* smem, int header, int wait) {
  constexpr int kRec = record_bytes(kGroup);
  Header* hd = reinterpret_cast<Header*>(smem);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, c = lane & 3;
  const int nch = s.chunks;
  const uint32_t ring = header + warp * kDepth * kRec;
  const uint32_t so = header + kWarps * kDepth * kRec;
  const uint32_t fo = so + kWarps * kSlotBytes;
  const uint32_t xo = (fo + x_scale_bytes(nch) + 255u) & ~255u;
  const int64_t total = static_cast<int64_t>(T.blocks) * nch;
  const int64_t a = total * warp / kWarps;
  const int count = static_cast<int>(total * (warp + 1) / kWarps - a);
  // The ring is filled kDepth - 1 records ahead; past the end the last
  // record is read again, so that every step waits for the same number.
  const uint8_t* w = T.W + a * kRec + lane * 16;
  const int last = max(count - 1, 0) * kRec;
  auto fetch = [&](uint32_t slot, int at) {
    const uint32_t to = smem_u32(smem + slot) + lane * 16;
    cp_async16(to, w + at);
    cp_async16(to + 512, w + at + 512);
    if (lane < (kRec - kCodeBytes) / 16) cp_async16(to + kCodeBytes, w + at + kCodeBytes);
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  auto begin = [&]() {
    if (count > 0) {
#pragma unroll
      for (int u = 0; u < kDepth - 1; ++u) fetch(ring + u * kRec, min(u * kRec, last));
    }
  };
  // the weights first if x is still to come, else the first loads of x
  if (wait == kWaitX) begin();
  if (wait != kWaitNone) pdl_wait();
  load_x<kX8>(s, T, smem, xo, fo, hd->row_w, [&]() {
    if (wait != kWaitX) begin();
  });
  __syncthreads();

  int block = a < (1ll << 31) ? static_cast<int>(divide(static_cast<uint32_t>(a), by_chunks))
                              : static_cast<int>(a / nch);
  int ch = static_cast<int>(a - static_cast<int64_t>(block) * nch);
  const int inside = ch, begun = block;  // where in its block the warp starts
  bool mid = ch != 0;                    // the piece at hand began inside its block
  const int token = min(g, T.n - 1);
  uint32_t x = xo + (token * nch + ch) * (2 * kChunk) + ((token & 1) << 6) + c * 16;
  uint32_t xs = fo + ch * (4 * kTile) + c * 8;
  float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  auto put = [&](uint32_t at) {
    float* o = reinterpret_cast<float*>(smem + at) + lane;
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i * 32] = acc[i];
  };
  const uint32_t first_slot = so + warp * kSlotBytes;  // a piece that began inside its block
  uint32_t rd = ring, wr = ring + (kDepth - 1) * kRec;
  int ahead = (kDepth - 1) * kRec;
#pragma unroll 2
  for (int i = 0; i < count; ++i) {
    asm volatile("cp.async.wait_group %0;" ::"n"(kDepth - 2) : "memory");
    __syncwarp();  // the record is there, and the one before it was read by all
    fetch(wr, min(ahead, last));
    ahead += kRec;
    multiply_record<kGroup>(acc, smem, rd + lane * 16,
                            rd + kCodeBytes + g * (kGroup == 32 ? 16 : 4), x, xs);
    wr = rd;
    rd += kRec;
    if (rd == ring + kDepth * kRec) rd = ring;
    xs += 4 * kTile;
    x += 2 * kChunk;
    if (++ch == nch) {
      if (mid)
        put(first_slot);
      else
        store_block<kSwiglu, kX8>(s, T, hd->row_w, acc, T.first_block + block, g, c);
      mid = false;
      ch = 0;
      ++block;
      xs -= 4 * kTile * nch;
      x -= 2 * kChunk * nch;
#pragma unroll
      for (int k = 0; k < 4; ++k) acc[k] = 0.0f;
    }
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  __syncwarp();
  // a piece that ends inside its block: its sums go where the ring was,
  // unless it also began there
  if (ch != 0 && count > 0) put(mid ? first_slot : ring);
  __syncthreads();
  if (warp > 0 && inside != 0 &&
      total * (warp - 1) / kWarps <= static_cast<int64_t>(begun) * nch) {
    auto add = [&](uint32_t at) {
      const float* o = reinterpret_cast<const float*>(smem + at) + lane;
#pragma unroll
      for (int k = 0; k < 4; ++k) acc[k] += o[k * 32];
    };
#pragma unroll
    for (int k = 0; k < 4; ++k) acc[k] = 0.0f;
    add(ring - kDepth * kRec);
    for (int v = warp; v < kWarps; ++v) {
      const int64_t lo = total * v / kWarps;
      if (lo >= (begun + 1ll) * nch) break;
      if (lo < total * (v + 1) / kWarps) add(so + v * kSlotBytes);
    }
    store_block<kSwiglu, kX8>(s, T, hd->row_w, acc, T.first_block + begun, g, c);
  }
}

// ceil(x / d) within [0, most]
__device__ __forceinline__ int blocks_before(int64_t x, const Divisor& d, int most) {
  if (x <= 0) return 0;
  if (x >= static_cast<int64_t>(d.d) * most) return most;
  if (x < (1ll << 31)) return static_cast<int>(divide(static_cast<uint32_t>(x) + d.d - 1, d));
  return static_cast<int>((x + d.d - 1) / d.d);
}

// Bound by HBM: each weight is read once per eight rows of its group, through
// private rings that need no barrier between warps.  896 latent experts with
// 300 present, 24 tokens: 908 us for 5.65 GB, 6.2 TB/s over both launches; a
// single token of 384 experts (223 MB) 47.1 us, where the launches' beginnings
// weigh.  One CTA of 16 warps an SM: two of 64 registers a thread took 260 us
// for eight tokens, this 235.  Tiles of eight tokens: sixteen a pass took 11.1
// us for 13 tokens of a 3584-7168 map, two passes of these 10.1.
//
// Blocks (of every tile of every group, in order) are dealt to the CTAs by
// cost, a record costing one: a block belongs to the CTA in whose share
// [lo, hi) of the total it begins.  Beginning a tile costs kTileCost, so a
// CTA whose share holds the end of one group and the start of another has
// fewer records.
template <bool kSwiglu, bool kX8, int kGroup>
__global__ void __launch_bounds__(kThreads, 1) gemv_int4_kernel(const __grid_constant__ Int4Launch p) {
  extern __shared__ __align__(1024) uint8_t smem[];
  Header* hd = reinterpret_cast<Header*>(smem);
  const int n0 = p.seg[0].groups, groups = n0 + (p.nseg > 1 ? p.seg[1].groups : 0);
  const int header = header_bytes(groups);
  // Routing needs the kernels before this one, unless the launch says so;
  // a launch without it plans its work while the kernel before it drains.
  int wait = p.wait == kWaitWeights && p.seg[0].offsets ? kWaitNone : p.wait;
  if (wait != p.wait) pdl_wait();
  pdl_release();

  const GroupLists lists = group_lists(hd->lists, groups);
  int64_t lo = 0, hi = 0;
  const GroupPlan plan = plan_groups<kThreads>(
      p, lists, hd->warp_sum,
      [&](int si, int n) -> int64_t {
        if (n <= 0 || n > p.most) return 0;
        const int64_t tile = static_cast<int64_t>(p.seg[si].blocks) * p.seg[si].chunks + kTileCost;
        return n <= p.cap[si] ? tile : tile * ((n + p.cap[si] - 1u) / p.cap[si]);
      },
      [&](int64_t total) {
        const int64_t share = total < (1ll << 32) ? divide(static_cast<uint32_t>(total), p.ctas)
                                                  : total / gridDim.x;
        const int rest = static_cast<int>(total - share * gridDim.x), cta = blockIdx.x;
        lo = share * cta + min(cta, rest);
        hi = lo + share + (cta < rest);
      },
      [&](int pos, int64_t before, int64_t cost) {
        if (before <= lo && lo < before + cost) hd->at_first = pos;
      });

  for (int pos = lo < hi ? hd->at_first : plan.present; pos < plan.present; ++pos) {
    const int64_t before = lists.before[pos];
    if (before >= hi) break;
    const int k = lists.number[pos], si = k >= n0;
    const Int4Segment& s = p.seg[si];
    const int grp = si ? k - n0 : k;
    const int row = s.offsets ? lists.first[k] : 0;
    const int n = s.offsets ? lists.first[k + 1] - row : static_cast<int>(s.rows);
    const int tiles = n <= p.cap[si] ? 1 : (n + p.cap[si] - 1u) / p.cap[si];
    const int64_t tile_cost = static_cast<int64_t>(s.blocks) * s.chunks + kTileCost;
    int t = tiles > 1 && lo > before ? static_cast<int>((lo - before) / tile_cost) : 0;
    for (; t < tiles; ++t) {
      const int64_t base = before + t * tile_cost + kTileCost;
      const int r0 = blocks_before(lo - base, p.chunks[si], s.blocks);
      const int r1 = blocks_before(hi - base, p.chunks[si], s.blocks);
      if (r1 == 0) break;
      if (r0 >= r1) continue;
      const int row0 = tiles > 1 ? static_cast<int>(static_cast<int64_t>(n) * t / tiles) : 0;
      Tile T;
      T.W = s.W + (static_cast<int64_t>(grp) * s.blocks + r0) * s.chunks * record_bytes(kGroup);
      T.blocks = r1 - r0;
      T.first_block = r0;
      T.n = (tiles > 1 ? static_cast<int>(static_cast<int64_t>(n) * (t + 1) / tiles) : n) - row0;
      T.out_row = row0 + (s.offsets ? row : grp * s.out_group_rows);
      T.x_row = row0 + (s.offsets ? row : grp * s.x_group_rows);
      run_tile<kSwiglu, kX8, kGroup>(s, p.chunks[si], T, smem, header, wait);
      wait = kWaitNone;
      __syncthreads();  // shared memory is free for the next tile
    }
  }
  if (wait != kWaitNone) pdl_wait();  // a kernel ends after the one before it has
}

template <bool kSwiglu, bool kX8, int kGroup>
cudaError_t launch_kernel(const Int4Launch& p, int num_sms, cudaStream_t stream) {
  static int configured[64] = {0};
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  if (dev >= 64 || !configured[dev]) {
    err = cudaFuncSetAttribute(gemv_int4_kernel<kSwiglu, kX8, kGroup>,
                               cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (err != cudaSuccess) return err;
    if (dev < 64) configured[dev] = 1;
  }
  return launch_pdl(gemv_int4_kernel<kSwiglu, kX8, kGroup>, dim3(num_sms), dim3(kThreads),
                    p.smem, stream, p);
}

template <bool kSwiglu, bool kX8>
cudaError_t launch_group(const Int4Launch& p, int group, int num_sms, cudaStream_t stream) {
  return group == 32 ? launch_kernel<kSwiglu, kX8, 32>(p, num_sms, stream)
                     : launch_kernel<kSwiglu, kX8, 128>(p, num_sms, stream);
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

cudaError_t launch_gemv_int4(const Int4Launch& p, bool swiglu, int group, int num_sms,
                             cudaStream_t stream) {
  Int4Launch l = p;
  int groups = 0;
  for (int i = 0; i < p.nseg; ++i) groups += p.seg[i].groups;
  l.smem = 0;
  l.ctas = divisor(num_sms);
  for (int i = 0; i < p.nseg; ++i) {
    const Int4Segment& s = p.seg[i];
    l.chunks[i] = divisor(s.chunks);
    l.cap[i] = tile_cap(groups, s.chunks, group);
    if (l.cap[i] < 1) return cudaErrorInvalidValue;  // the callers' limit on the width
    if (s.rows < l.cap[i]) l.cap[i] = static_cast<int>(s.rows);
    const int need = fixed_smem(groups, s.chunks, group) + l.cap[i] * x_row_bytes(s.chunks);
    l.smem = l.smem > need ? l.smem : need;
  }
  const bool x8 = p.seg[0].x_scale != nullptr;
  if (swiglu)
    return x8 ? launch_group<true, true>(l, group, num_sms, stream)
              : launch_group<true, false>(l, group, num_sms, stream);
  return x8 ? launch_group<false, true>(l, group, num_sms, stream)
            : launch_group<false, false>(l, group, num_sms, stream);
}

}  // namespace fgs
