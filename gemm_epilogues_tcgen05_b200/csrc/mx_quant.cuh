// mx_quant.cuh -- microscaled 4-bit values: quantisation and its inverse.
//
// A block is 32 consecutive elements along a row. Its scale is the power of
// two 2^(floor(log2 max|x|) - 2) (2 is the exponent of the largest e2m1
// power of two, 4), at least 2^-127, held as the biased exponent (e8m0); an
// element is x / scale -- exact, since the scale is a power of two -- rounded
// to the nearest e2m1 value 0, .5, 1, 1.5, 2, 3, 4, 6, ties to the even code,
// larger magnitudes to 6. A block of zeros has scale 2^-127; one with an
// infinity or NaN has scale byte 255 (NaN) and stands for NaN throughout.
//
// Two values share a byte, the lower column in the low four bits. Scales are
// laid out as the tensor cores' scale loads want them: tiles of 128 rows x 4
// blocks (128 columns), 512 bytes each, row tile by row tile, k tile by k
// tile inside; row r, block b of a tile at byte 16 (r % 32) + 4 (r / 32) + b.
// Blocks past the last column are scale byte 0, so that the product's padding
// (zero values) stays zero. With row groups, every group starts a new row
// tile, so a tile of the grouped product always starts at a tile of scales.
//
// The kernels are bound by memory: 2 bytes read and 17/32 written an element
// (the inverse the other way round). What is read once (the source) and what is
// large and not read back soon (fp32 values) passes L2 with an evict-first
// hint, which leaves the packed values there for the kernel that reads them
// next: 4096 x 11008, transposed source, quantised and back to fp32, 72 us
// without and 60.6 us with (294 MB; 45 us at the copy rate). Alone: 1000 x 4096
// 3.7 us and 4.4 us (launch-bound), 4096 x 4096 9.0 us (4.7 TB/s), 11008 x 4096
// transposed 20 us (5.7 TB/s), to fp32 29.9 us (6.8 TB/s).
#pragma once

#include <cuda_fp4.h>

#include "grouped_kernel.cuh"

namespace ge {

struct MxQuantParams {
  int64_t batch, rows;   // matrices; rows of each (the values' rows)
  int32_t cols;          // elements of a row, a multiple of 32
  int32_t kt;            // scale tiles along a row: ceil(cols / 128)
  int32_t rt;            // scale tiles along the rows of one matrix (no groups)
  int32_t groups;        // row groups (0: none)
  int32_t flat;          // a row's place among the scales is its index (one matrix, or whole scale tiles)
  const int32_t* offsets;
  const void* src;
  uint8_t* q;
  uint8_t* scales;
  void* out;             // dequantisation
  int32_t out_f32;
};

// Scale byte of a block from its largest magnitude, given by the bits of the
// 16-bit values with their signs off: as unsigned integers these are ordered
// as the magnitudes are, infinity above every number and NaN above infinity.
template <bool BF16>
__device__ __forceinline__ uint32_t mx_scale_byte(uint32_t top) {
  float f;
  if constexpr (BF16)
    f = __uint_as_float(top << 16);
  else
    f = __half2float(__ushort_as_half(static_cast<unsigned short>(top)));
  const int e = static_cast<int>(__float_as_uint(f) >> 23);
  return e == 255 ? 255u : static_cast<uint32_t>(max(e - 2, 0));
}
__device__ __forceinline__ uint32_t mx_abs2(uint32_t u) { return u & 0x7fff7fffu; }
// 2^(127 - byte), exact for bytes up to 253 (255 stands for NaN; its values are not read)
__device__ __forceinline__ float mx_inverse_scale(uint32_t byte) { return __uint_as_float((254u - min(byte, 253u)) << 23); }
// 2^(byte - 127)
__device__ __forceinline__ float mx_scale_value(uint32_t byte) {
  return byte == 255u ? __uint_as_float(0x7fc00000u) : byte == 0u ? __uint_as_float(0x00400000u) : __uint_as_float(byte << 23);
}
// eight values to e2m1, the first in the lowest four bits
__device__ __forceinline__ uint32_t mx_pack8(float a, float b, float c, float d, float e, float f, float g, float h) {
  uint32_t r;
  asm("{\n\t.reg .b8 p, q, s, t;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 p, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 q, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 s, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 t, %8, %7;\n\t"
      "mov.b32 %0, {p, q, s, t};\n\t}"
      : "=r"(r)
      : "f"(a), "f"(b), "f"(c), "f"(d), "f"(e), "f"(f), "f"(g), "f"(h));
  return r;
}
// two packed values
__device__ __forceinline__ float2 mx_unpack2(uint32_t byte) {
  const __half2_raw h = __nv_cvt_fp4x2_to_halfraw2(static_cast<__nv_fp4x2_storage_t>(byte), __NV_E2M1);
  return __half22float2(__half2(h));
}

template <bool BF16>
__device__ __forceinline__ float2 unpack2(uint32_t u) {
  if constexpr (BF16) {
    return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&u));
  } else {
    return __half22float2(*reinterpret_cast<const __half2*>(&u));
  }
}

// The row's place among the scale tiles (rows counted with the padding of
// whole tiles), or -1 for a row of no group.
__device__ __forceinline__ int64_t mx_scale_row(const MxQuantParams& p, const int* offs, const int* start, int64_t row) {
  if (p.groups == 0) {
    if (p.flat) return row;
    const int64_t b = row / p.rows;
    return b * (static_cast<int64_t>(p.rt) * 128) + (row - b * p.rows);
  }
  const int r = static_cast<int>(row);
  if (r < offs[0] || r >= offs[p.groups]) return -1;
  int lo = 0, hi = p.groups;  // offs[lo] <= r < offs[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (offs[mid] <= r)
      lo = mid;
    else
      hi = mid;
  }
  return static_cast<int64_t>(start[lo]) * 128 + (r - offs[lo]);
}

__device__ __forceinline__ int64_t mx_scale_at(const MxQuantParams& p, int64_t srow, int ktile) {
  return ((srow >> 7) * p.kt + ktile) * 512 + (srow & 31) * 16 + ((srow >> 5) & 3) * 4;
}

__device__ __forceinline__ void mx_table(const MxQuantParams& p, int* offs, int* start) {
  if (p.groups > 0 && threadIdx.x < 32) {
    GroupedParams g{};
    g.T = static_cast<int32_t>(p.rows);
    g.E = p.groups;
    g.offsets = p.offsets;
    grouped_table<128>(g, offs, start, 1);
  }
  if (p.groups > 0) __syncthreads();
}

// Rows contiguous. A warp takes 1024 columns of one row in four loads of 16
// bytes a lane (8 elements; four lanes make a block), all in flight together.
template <bool BF16>
__global__ void __launch_bounds__(256) mx_quantize_kernel(const MxQuantParams p) {
  wait_for_inputs();
  extern __shared__ int table[];
  int* offs = table;
  int* start = table + p.groups + 1;
  mx_table(p, offs, start);
  const int lane = static_cast<int>(lane_id());
  const int c0 = static_cast<int>(blockIdx.y) * 1024 + lane * 8;
  for (int64_t row = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5); row < p.batch * p.rows;
       row += static_cast<int64_t>(gridDim.x) * 8) {
    const int64_t srow = mx_scale_row(p, offs, start, row);
    if (srow < 0) continue;
    const uint16_t* src = reinterpret_cast<const uint16_t*>(p.src) + row * p.cols;
    uint4 x[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      x[i] = c0 + i * 256 < p.cols ? __ldcs(reinterpret_cast<const uint4*>(src + c0 + i * 256)) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int c = c0 + i * 256;
      uint32_t top = __vmaxu2(__vmaxu2(mx_abs2(x[i].x), mx_abs2(x[i].y)), __vmaxu2(mx_abs2(x[i].z), mx_abs2(x[i].w)));
      top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const uint32_t byte = mx_scale_byte<BF16>(max(top & 0xffffu, top >> 16));
      const float s = mx_inverse_scale(byte);
      const float2 a = unpack2<BF16>(x[i].x), b = unpack2<BF16>(x[i].y), d = unpack2<BF16>(x[i].z),
                   e = unpack2<BF16>(x[i].w);
      const uint32_t w = mx_pack8(a.x * s, a.y * s, b.x * s, b.y * s, d.x * s, d.y * s, e.x * s, e.y * s);
      // four blocks' bytes make the word of this row in a scale tile
      uint32_t word = byte << ((lane >> 2 & 3) * 8);
      if (c >= p.cols) word = 0u;
      word |= __shfl_xor_sync(0xffffffffu, word, 4);
      word |= __shfl_xor_sync(0xffffffffu, word, 8);
      if (c < p.cols) *reinterpret_cast<uint32_t*>(p.q + (row * p.cols + c) / 2) = w;
      if ((lane & 15) == 0 && c < p.cols)
        *reinterpret_cast<uint32_t*>(p.scales + mx_scale_at(p, srow, c >> 7)) = word;
    }
  }
}

// Rows strided (the source is cols x rows, as a K x N weight whose blocks run
// along K): a lane takes two neighbouring rows and 128 columns, 4 bytes a
// load, so a warp reads 128 contiguous bytes of every source row.
template <bool BF16>
__global__ void __launch_bounds__(128) mx_quantize_t_kernel(const MxQuantParams p) {
  wait_for_inputs();
  const int lane = static_cast<int>(lane_id());
  const int kt = static_cast<int>(blockIdx.y);
  const int64_t rchunks = (p.rows + 63) / 64;
  for (int64_t it = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5); it < p.batch * rchunks;
       it += static_cast<int64_t>(gridDim.x) * 4) {
    const int64_t b = p.batch == 1 ? 0 : it / rchunks;
    const int64_t r = (it - b * rchunks) * 64 + lane * 2;
    if (r >= p.rows) continue;  // no exchange between lanes below
    const uint16_t* src = reinterpret_cast<const uint16_t*>(p.src) + b * p.rows * p.cols + r;
    uint32_t word0 = 0u, word1 = 0u;
#pragma unroll 1
    for (int blk = 0; blk < 4; ++blk) {
      const int c = kt * 128 + blk * 32;
      if (c >= p.cols) break;
      uint32_t x[32];
#pragma unroll
      for (int j = 0; j < 32; ++j) x[j] = __ldcs(reinterpret_cast<const uint32_t*>(src + (static_cast<int64_t>(c) + j) * p.rows));
      uint32_t top = 0u;  // both rows' largest magnitudes
#pragma unroll
      for (int j = 0; j < 32; ++j) top = __vmaxu2(top, mx_abs2(x[j]));
      const uint32_t b0 = mx_scale_byte<BF16>(top & 0xffffu), b1 = mx_scale_byte<BF16>(top >> 16);
      const float s0 = mx_inverse_scale(b0), s1 = mx_inverse_scale(b1);
      uint32_t q0[4], q1[4];
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        float2 v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = unpack2<BF16>(x[g * 8 + j]);
        q0[g] = mx_pack8(v[0].x * s0, v[1].x * s0, v[2].x * s0, v[3].x * s0, v[4].x * s0, v[5].x * s0, v[6].x * s0,
                         v[7].x * s0);
        q1[g] = mx_pack8(v[0].y * s1, v[1].y * s1, v[2].y * s1, v[3].y * s1, v[4].y * s1, v[5].y * s1, v[6].y * s1,
                         v[7].y * s1);
      }
      uint8_t* dst = p.q + ((b * p.rows + r) * p.cols + c) / 2;
      *reinterpret_cast<uint4*>(dst) = make_uint4(q0[0], q0[1], q0[2], q0[3]);
      *reinterpret_cast<uint4*>(dst + p.cols / 2) = make_uint4(q1[0], q1[1], q1[2], q1[3]);
      word0 |= b0 << (8 * blk);
      word1 |= b1 << (8 * blk);
    }
    const int64_t srow = b * (static_cast<int64_t>(p.rt) * 128) + r;
    *reinterpret_cast<uint32_t*>(p.scales + mx_scale_at(p, srow, kt)) = word0;
    *reinterpret_cast<uint32_t*>(p.scales + mx_scale_at(p, srow + 1, kt)) = word1;
  }
}

// The inverse: 8 elements a lane and step, 256 columns of a row a warp, four
// steps in flight.
template <bool BF16>
__global__ void __launch_bounds__(256) mx_dequantize_kernel(const MxQuantParams p) {
  wait_for_inputs();
  extern __shared__ int table[];
  int* offs = table;
  int* start = table + p.groups + 1;
  mx_table(p, offs, start);
  const int lane = static_cast<int>(lane_id());
  const int c0 = static_cast<int>(blockIdx.y) * 1024 + lane * 8;
  for (int64_t row = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5); row < p.batch * p.rows;
       row += static_cast<int64_t>(gridDim.x) * 8) {
    const int64_t srow = mx_scale_row(p, offs, start, row);
    if (srow < 0) continue;
    uint32_t x[4], sb[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int c = c0 + i * 256;
      x[i] = c < p.cols ? *reinterpret_cast<const uint32_t*>(p.q + (row * p.cols + c) / 2) : 0u;
      sb[i] = c < p.cols ? p.scales[mx_scale_at(p, srow, c >> 7) + (c >> 5 & 3)] : 0u;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int c = c0 + i * 256;
      if (p.out_f32) {
        // neighbouring lanes (one block's, so one scale) share both words, so
        // that each store instruction covers 512 contiguous bytes
        const uint32_t even = __shfl_sync(0xffffffffu, x[i], lane & ~1), odd = __shfl_sync(0xffffffffu, x[i], lane | 1);
        if (c >= p.cols) continue;
        const float s = mx_scale_value(sb[i]);
        const int h = (lane & 1) * 16;
        const float2 a = mx_unpack2(even >> h & 0xffu), b = mx_unpack2(even >> (h + 8) & 0xffu);
        const float2 d = mx_unpack2(odd >> h & 0xffu), e = mx_unpack2(odd >> (h + 8) & 0xffu);
        float* dst = reinterpret_cast<float*>(p.out) + row * p.cols + (c & ~15) + (lane & 1) * 4;
        __stcs(reinterpret_cast<float4*>(dst), make_float4(a.x * s, a.y * s, b.x * s, b.y * s));
        __stcs(reinterpret_cast<float4*>(dst + 8), make_float4(d.x * s, d.y * s, e.x * s, e.y * s));
      } else if (c < p.cols) {
        const float s = mx_scale_value(sb[i]);
        float2 v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = mx_unpack2(x[i] >> (8 * j) & 0xffu);
        *reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(p.out) + row * p.cols + c) =
            make_uint4(pack2<BF16>(v[0].x * s, v[0].y * s), pack2<BF16>(v[1].x * s, v[1].y * s),
                       pack2<BF16>(v[2].x * s, v[2].y * s), pack2<BF16>(v[3].x * s, v[3].y * s));
      }
    }
  }
}

}  // namespace ge
