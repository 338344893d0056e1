// w4_quant.cuh -- weights held in 4 bits with a 16-bit scale for each group of G
// = 32, 64 or 128 consecutive columns: quantisation, packing of codes that exist,
// and the inverse.
//
//   value = scale (code - zero), code 0 .. 15, zero 8 or a byte for each group
//   without zeros: scale = rn16(max|w| / 7), code = clamp(rint(w / scale), -8, 7) + 8
//   with zeros:    lo = min(w, 0), hi = max(w, 0), scale = rn16((hi - lo) / 15),
//                  zero = clamp(rint(-lo / scale), 0, 15), code = clamp(rint(w / scale) + zero, 0, 15)
// (rint: ties to even; a scale that rounds to 0 gives codes that are the zero.)
//
// Layout: tiles of 32 features x 128 columns, tile (i, j) of a matrix at 2048 (i kt +
// j) bytes. Feature f, 32-column block b, 8-column word w of a tile are the 4 bytes at 512 b + 16 f + 4 w:
// a warp of the product reads 512 contiguous bytes, 16 a lane, 32 columns of the
// lane's own feature. In a word, column 2 m is in bits 4m .. 4m+3 and column 2 m + 1 in
// bits 4m+16 .. 4m+19, so that a shift and a mask leave two neighbouring columns in
// a register's halves. Scales (and zeros) of a tile: [128 / G groups][f]. Rows
// and columns past the matrix are code 0 with scale 0.
//
// A weight of 11008 x 4096 is 90 MB to read and 23.2 to write, 17 us at the rate of a copy.
// Quantising it takes 27.7 us with zeros, 26.1 without: 60 % of that rate, the quotients and conversions
// take the rest. The inverse is bound by memory: 22.0 us to 16-bit values, 31.9 to fp32 ones (180 MB). (A lane with 8 columns, 16 of them sharing a group's
// scale and its divisions, took 85.)
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "tile_kernel.cuh"

namespace ge {

struct W4Params {
  int64_t tiles;         // of all matrices
  int32_t rows, cols;    // of one matrix
  int32_t rt, kt;        // tiles along the rows (32) and the columns (128) of one matrix
  int32_t group;
  const void* src;       // quantise: the 16-bit matrix; pack: the codes, two a byte, the lower column in the low 4 bits
  const void* src_scales;
  const uint8_t* src_zeros;
  uint8_t* q;
  void* scales;
  uint8_t* zeros;        // null: zero = 8
  void* out;             // dequantise
};

constexpr int kW4Rows = 32, kW4TileBytes = 2048;
constexpr uint16_t kW4Nan = 0x7fff;  // a NaN of either 16-bit type

// byte of the word of feature f (0..31) and 8-column unit u (0..15) in a tile
__device__ __forceinline__ uint32_t w4_word(uint32_t f, uint32_t u) { return 512 * (u >> 2) + 16 * f + 4 * (u & 3u); }

template <bool BF16>
__device__ __forceinline__ float w4_float(uint16_t h) {
  if constexpr (BF16)
    return __uint_as_float(static_cast<uint32_t>(h) << 16);
  else
    return __half2float(__ushort_as_half(h));
}
template <bool BF16>
__device__ __forceinline__ uint16_t w4_round16(float f) {
  return static_cast<uint16_t>(pack2<BF16>(f, 0.f) & 0xffffu);
}

// (No read-only loads in these kernels: they may start before the kernel ahead of them, which
// writes their operands, has ended.)
__device__ __forceinline__ uint4 w4_load_once(const void* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

// The tile's words as staged by its warp, out to the packed weight.
__device__ __forceinline__ void w4_store_tile(uint8_t* q, const uint32_t* stage) {
  const uint32_t lane = lane_id();
  __syncwarp();
#pragma unroll
  for (int i = 0; i < 4; ++i)
    reinterpret_cast<uint4*>(q)[32 * i + lane] = reinterpret_cast<const uint4*>(stage)[32 * i + lane];
  __syncwarp();
}

// w / s with the error that the codes' rounding allows: a quotient corrected by one exact
// remainder (P. W. Markstein, Computation of elementary functions on the IBM RISC System/6000
// processor, IBM J. Res. Dev. 34, 1990). w and s are integers a, b < 2^11 times powers of two, |w / s| < 32.
//   Ties, w / s = m + 1/2: a number of few bits. r = 1 / s rounded, so q0 = w r is off by a few units of its last
//   place; w - q0 s is a few such units times s, which fp32 holds (s >= 1e-30: no underflow), and the step
//   w / s - q0 is off by 2^-23 of itself: the result rounds to m + 1/2 exactly.
//   Others are (2 w - (2 m + 1) s) / (2 s) from a tie, whose numerator is a multiple of the smaller of s / b
//   and 2 w / a: at least 1 / (2 b) >= 2^-12, or (w / s) / a >= 2^-13 where |w / s| >= 1/4 (below it no tie is
//   nearer than 1/4). The result is off by 32 x 2^-23 at most and stays on its side.
__device__ __forceinline__ float w4_divide(float w, float s, float r) {
  const float q0 = w * r;
  return fmaf(fmaf(-q0, s, w), r, q0);
}

// the larger (smaller) of two pairs; NaN stays
template <bool BF16>
__device__ __forceinline__ uint32_t w4_max2(uint32_t a, uint32_t b) {
  uint32_t d;
  if constexpr (BF16)
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  else
    asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
template <bool BF16>
__device__ __forceinline__ uint32_t w4_min2(uint32_t a, uint32_t b) {
  uint32_t d;
  if constexpr (BF16)
    asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  else
    asm("min.NaN.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// A lane has 32 columns of one feature: a whole group or a half or a quarter of one, whose
// extremes it finds two values at a time, and the 16 bytes of its codes. A warp takes 8
// features of a tile, a CTA two tiles side by side.
template <bool BF16, bool ZEROS>
__global__ void __launch_bounds__(256) w4_quantize_kernel(const W4Params p) {
  wait_for_inputs();
  const uint32_t lane = lane_id(), warp = threadIdx.x >> 5, b = lane & 3u, f = 8 * (warp & 3u) + (lane >> 2);
  const uint32_t pairs = (static_cast<uint32_t>(p.kt) + 1) / 2;
  const uint32_t row_tile = blockIdx.x / pairs, j = 2 * (blockIdx.x - row_tile * pairs) + (warp >> 2);
  if (j >= static_cast<uint32_t>(p.kt)) return;
  const uint32_t m = row_tile / static_cast<uint32_t>(p.rt), row = (row_tile - m * p.rt) * kW4Rows + f, col = j * 128 + 32 * b;
  const int64_t tile = static_cast<int64_t>(row_tile) * p.kt + j;
  const bool in = row < static_cast<uint32_t>(p.rows) && col < static_cast<uint32_t>(p.cols);
  uint32_t w[16];
  {
    const uint16_t* from = reinterpret_cast<const uint16_t*>(p.src) + (static_cast<int64_t>(m) * p.rows + row) * p.cols + col;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint4 v = in ? reinterpret_cast<const uint4*>(from)[i] : make_uint4(0, 0, 0, 0);
      w[4 * i] = v.x, w[4 * i + 1] = v.y, w[4 * i + 2] = v.z, w[4 * i + 3] = v.w;
    }
  }
  uint32_t hi2 = 0, lo2 = 0;
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    hi2 = w4_max2<BF16>(hi2, ZEROS ? w[e] : w[e] & 0x7fff7fffu);
    if constexpr (ZEROS) lo2 = w4_min2<BF16>(lo2, w[e]);
  }
  hi2 = w4_max2<BF16>(hi2, __funnelshift_l(hi2, hi2, 16));
  lo2 = w4_min2<BF16>(lo2, __funnelshift_l(lo2, lo2, 16));
  for (int off = 1; off < p.group / 32; off <<= 1) {
    hi2 = w4_max2<BF16>(hi2, __shfl_xor_sync(0xffffffffu, hi2, off));
    if constexpr (ZEROS) lo2 = w4_min2<BF16>(lo2, __shfl_xor_sync(0xffffffffu, lo2, off));
  }
  const float hi = w4_float<BF16>(static_cast<uint16_t>(hi2)), lo = w4_float<BF16>(static_cast<uint16_t>(lo2));
  float top = ZEROS ? __fdiv_rn(hi - lo, 15.f) : __fdiv_rn(hi, 7.f);
  if (!(top <= 3.4e38f)) top = __uint_as_float(0x7fc00000u);  // an infinity or NaN: the group stands for NaN
  const uint16_t s16 = w4_round16<BF16>(top);
  const float s = w4_float<BF16>(s16);
  float zero = 8.f;
  if constexpr (ZEROS) zero = s > 0.f ? fminf(fmaxf(rintf(__fdiv_rn(-lo, s)), 0.f), 15.f) : 0.f;
  const uint32_t z = static_cast<uint32_t>(zero), z2 = z * 0x00010001u;
  const auto value = [&](int e, int i) {
    return w4_float<BF16>(static_cast<uint16_t>(i ? w[e] >> 16 : w[e] & 0xffffu));
  };
  uint32_t word[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) word[k] = z * 0x11111111u;
  if (s >= 1e-30f) {
    // |w / s| < 32 (an s that was rounded to few bits included), so that the integer is
    // the low 16 bits of the quotient + 1.5 2^23, whose addition rounds it; two at a time from there
    const float r = __frcp_rn(s);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      word[k] = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int e = 4 * k + i;
        const uint32_t c0 = __float_as_uint(w4_divide(value(e, 0), s, r) + 12582912.f);
        const uint32_t c1 = __float_as_uint(w4_divide(value(e, 1), s, r) + 12582912.f);
        const uint32_t code = __viaddmin_s16x2_relu(__byte_perm(c0, c1, 0x5410), z2, 0x000f000fu);
        word[k] += code << (4 * i);
      }
    }
  } else if (s > 0.f) {  // the reciprocal would leave fp32
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      word[k] = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float c = rintf(__fdiv_rn(value(4 * k + i / 2, i & 1), s)) + zero;
        word[k] |= static_cast<uint32_t>(fminf(fmaxf(c, 0.f), 15.f)) << (4 * (i / 2) + 16 * (i & 1));
      }
    }
  }
  reinterpret_cast<uint4*>(p.q + tile * kW4TileBytes)[32 * b + f] =
      in ? make_uint4(word[0], word[1], word[2], word[3]) : make_uint4(0, 0, 0, 0);
  const uint32_t per = static_cast<uint32_t>(p.group) / 32;  // 1, 2 or 4 lanes
  if ((b & (per - 1)) == 0) {
    const int64_t at = (tile * (4 / per) + b / per) * kW4Rows + f;
    reinterpret_cast<uint16_t*>(p.scales)[at] = in ? s16 : 0;
    if constexpr (ZEROS) p.zeros[at] = in ? static_cast<uint8_t>(z) : 0;
  }
}

// Codes as a checkpoint has them (rows x cols / 2 bytes), scales and zeros rows x
// cols / G, to the layout. Copies, but for a zero point of 128 or more, which the product's operands have
// no room for: the group gets a NaN scale.
static __global__ void __launch_bounds__(256) w4_pack_kernel(const W4Params p) {
  __shared__ __align__(16) uint32_t stage[8][kW4TileBytes / 4];
  wait_for_inputs();
  const uint32_t lane = lane_id(), warp = threadIdx.x >> 5, u = lane & 15u, ng = 128u / p.group;
  const int groups = p.cols / p.group;
  for (int64_t tile = static_cast<int64_t>(blockIdx.x) * 8 + warp; tile < p.tiles; tile += static_cast<int64_t>(gridDim.x) * 8) {
    const int j = static_cast<int>(tile % p.kt);
    const int64_t row_tile = tile / p.kt;
    const int i = static_cast<int>(row_tile % p.rt);
    const int64_t m = row_tile / p.rt;
    const int col = j * 128 + 8 * static_cast<int>(u);
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      const uint32_t f = 2 * k + (lane >> 4);
      const int row = i * kW4Rows + static_cast<int>(f);
      uint32_t src = 0;
      if (row < p.rows && col < p.cols)
        src = *reinterpret_cast<const uint32_t*>(reinterpret_cast<const uint8_t*>(p.src) +
                                                 (m * p.rows + row) * (p.cols / 2) + col / 2);
      const auto gather = [](uint32_t x) {  // the low 4 bits of each byte, side by side
        x &= 0x0f0f0f0fu;
        x = (x | (x >> 4)) & 0x00ff00ffu;
        return (x | (x >> 8)) & 0xffffu;
      };
      stage[warp][w4_word(f, u) / 4] = gather(src) | (gather(src >> 4) << 16);
    }
    for (uint32_t k = 0; k < ng; ++k) {  // a lane its feature
      const int row = i * kW4Rows + static_cast<int>(lane), g = j * static_cast<int>(ng) + static_cast<int>(k);
      const bool in = row < p.rows && g < groups;
      const int64_t from = in ? (m * p.rows + row) * groups + g : 0, at = (tile * ng + k) * kW4Rows + lane;
      const uint32_t zero = in && p.zeros ? p.src_zeros[from] : 0u;
      reinterpret_cast<uint16_t*>(p.scales)[at] =
          zero > 127u ? kW4Nan : in ? reinterpret_cast<const uint16_t*>(p.src_scales)[from] : 0;
      if (p.zeros) p.zeros[at] = static_cast<uint8_t>(zero & 127u);
    }
    w4_store_tile(p.q + tile * kW4TileBytes, stage[warp]);
  }
}

// The values: a warp has 8 features of a tile, a CTA two tiles side by side; a row of
// the tile at a time, four columns a lane (fp32, exact: 8 or 11 bits times 8), or two rows, eight
// columns a lane (16-bit, rounded once).
template <bool BF16, bool F32>
__global__ void __launch_bounds__(256) w4_dequantize_kernel(const W4Params p) {
  __shared__ __align__(16) uint32_t stage[8][128];
  wait_for_inputs();
  const uint32_t lane = lane_id(), warp = threadIdx.x >> 5, ng = 128u / static_cast<uint32_t>(p.group);
  const uint32_t pairs = (static_cast<uint32_t>(p.kt) + 1) / 2;
  const uint32_t row_tile = blockIdx.x / pairs, j = 2 * (blockIdx.x - row_tile * pairs) + (warp >> 2);
  if (j >= static_cast<uint32_t>(p.kt)) return;
  const uint32_t m = row_tile / static_cast<uint32_t>(p.rt), f0 = 8 * (warp & 3u), row0 = (row_tile - m * p.rt) * kW4Rows + f0;
  const int64_t tile = static_cast<int64_t>(row_tile) * p.kt + j;
  // [block of 32 columns][feature]: 16 bytes
  reinterpret_cast<uint4*>(stage[warp])[lane] =
      w4_load_once(reinterpret_cast<const uint4*>(p.q + tile * kW4TileBytes) + 32 * (lane >> 3) + f0 + (lane & 7u));
  __syncwarp();
  constexpr int V = F32 ? 4 : 8;  // columns a lane
  const uint32_t c0 = F32 ? lane * 4 : (lane & 15u) * 8, col = j * 128 + c0;
  if (col >= static_cast<uint32_t>(p.cols)) return;
#pragma unroll
  for (int k = 0; k < (F32 ? 8 : 4); ++k) {
    const uint32_t f = F32 ? k : 2 * k + (lane >> 4), row = row0 + f;
    if (row >= static_cast<uint32_t>(p.rows)) break;
    const int64_t at = (tile * ng + c0 / static_cast<uint32_t>(p.group)) * kW4Rows + f0 + f;
    const float s = w4_float<BF16>(reinterpret_cast<const uint16_t*>(p.scales)[at]);
    float z = p.zeros ? static_cast<float>(p.zeros[at]) : 8.f;
    if (z > 127.f) z = __uint_as_float(0x7fc00000u);  // not a zero point (w4_pack leaves none)
    const uint32_t word = stage[warp][(c0 / 32) * 32 + f * 4 + (c0 / 8 & 3u)];
    float v[V];
#pragma unroll
    for (int e = 0; e < V; ++e) {
      const uint32_t c = F32 ? (lane & 1u) * 4 + e : e;
      v[e] = s * (static_cast<float>((word >> (4 * (c >> 1) + 16 * (c & 1u))) & 15u) - z);
    }
    const int64_t o = (static_cast<int64_t>(m) * p.rows + row) * p.cols + col;
    if constexpr (F32)
      __stcs(reinterpret_cast<float4*>(reinterpret_cast<float*>(p.out) + o), make_float4(v[0], v[1], v[2], v[3]));
    else
      *reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(p.out) + o) =
          make_uint4(pack2<BF16>(v[0], v[1]), pack2<BF16>(v[2], v[3]), pack2<BF16>(v[4], v[5]), pack2<BF16>(v[6], v[7]));
  }
}

}  // namespace ge
