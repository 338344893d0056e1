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
// Both kernels are bound by memory: 2 bytes read and 17/32 written an element
// (the inverse the other way round).
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
  const int32_t* offsets;
  const void* src;
  uint8_t* q;
  uint8_t* scales;
  void* out;             // dequantisation
  int32_t out_f32;
};

// scale byte of a block whose largest magnitude is `top`
__device__ __forceinline__ uint32_t mx_scale_byte(float top) {
  const int e = static_cast<int>(__float_as_uint(top) >> 23);  // top >= 0, or NaN
  return top != top || e == 255 ? 255u : static_cast<uint32_t>(max(e - 2, 0));
}
// 2^(127 - byte), exact for bytes up to 253 (255 stands for NaN; its values are not read)
__device__ __forceinline__ float mx_inverse_scale(uint32_t byte) { return __uint_as_float((254u - min(byte, 253u)) << 23); }
// 2^(byte - 127)
__device__ __forceinline__ float mx_scale_value(uint32_t byte) {
  return byte == 255u ? __uint_as_float(0x7fc00000u) : byte == 0u ? __uint_as_float(0x00400000u) : __uint_as_float(byte << 23);
}
// |a| or |b|, whichever is larger; NaN if either is
__device__ __forceinline__ float max_abs_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(fabsf(a)), "f"(fabsf(b)));
  return r;
}
__device__ __forceinline__ uint32_t mx_pack2(float lo, float hi) {
  return __nv_cvt_float2_to_fp4x2(make_float2(lo, hi), __NV_E2M1, cudaRoundNearest);
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
  if (p.groups == 0) return (row / p.rows) * (static_cast<int64_t>(p.rt) * 128) + row % p.rows;
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
  extern __shared__ int table[];
  int* offs = table;
  int* start = table + p.groups + 1;
  mx_table(p, offs, start);
  const int lane = static_cast<int>(lane_id());
  const int chunks = (p.cols + 1023) / 1024;
  const int64_t items = p.batch * p.rows * chunks;
  for (int64_t it = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5); it < items;
       it += static_cast<int64_t>(gridDim.x) * 8) {
    const int64_t row = it / chunks;
    const int c0 = static_cast<int>(it - row * chunks) * 1024 + lane * 8;
    const int64_t srow = mx_scale_row(p, offs, start, row);
    if (srow < 0) continue;
    const uint16_t* src = reinterpret_cast<const uint16_t*>(p.src) + row * p.cols;
    uint4 x[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      x[i] = c0 + i * 256 < p.cols ? *reinterpret_cast<const uint4*>(src + c0 + i * 256) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int c = c0 + i * 256;
      const float2 a = unpack2<BF16>(x[i].x), b = unpack2<BF16>(x[i].y), d = unpack2<BF16>(x[i].z),
                   e = unpack2<BF16>(x[i].w);
      float top = max_abs_nan(max_abs_nan(max_abs_nan(a.x, a.y), max_abs_nan(b.x, b.y)),
                              max_abs_nan(max_abs_nan(d.x, d.y), max_abs_nan(e.x, e.y)));
      top = max_abs_nan(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = max_abs_nan(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const uint32_t byte = mx_scale_byte(top);
      const float s = mx_inverse_scale(byte);
      const uint32_t w = mx_pack2(a.x * s, a.y * s) | mx_pack2(b.x * s, b.y * s) << 8 | mx_pack2(d.x * s, d.y * s) << 16 |
                         mx_pack2(e.x * s, e.y * s) << 24;
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
  const int lane = static_cast<int>(lane_id());
  const int64_t rchunks = (p.rows + 63) / 64;
  const int64_t items = p.batch * rchunks * p.kt;
  for (int64_t it = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5); it < items;
       it += static_cast<int64_t>(gridDim.x) * 4) {
    const int64_t b = it / (rchunks * p.kt);
    const int64_t in = it - b * rchunks * p.kt;
    const int kt = static_cast<int>(in / rchunks);
    const int64_t r = (in - kt * rchunks) * 64 + lane * 2;
    if (r >= p.rows) continue;  // no exchange between lanes below
    const uint16_t* src = reinterpret_cast<const uint16_t*>(p.src) + b * p.rows * p.cols + r;
    uint32_t word0 = 0u, word1 = 0u;
#pragma unroll 1
    for (int blk = 0; blk < 4; ++blk) {
      const int c = kt * 128 + blk * 32;
      if (c >= p.cols) break;
      uint32_t x[32];
#pragma unroll
      for (int j = 0; j < 32; ++j) x[j] = *reinterpret_cast<const uint32_t*>(src + (static_cast<int64_t>(c) + j) * p.rows);
      float t0 = 0.f, t1 = 0.f;
#pragma unroll
      for (int j = 0; j < 32; ++j) {
        const float2 v = unpack2<BF16>(x[j]);
        t0 = max_abs_nan(t0, v.x);
        t1 = max_abs_nan(t1, v.y);
      }
      const uint32_t b0 = mx_scale_byte(t0), b1 = mx_scale_byte(t1);
      const float s0 = mx_inverse_scale(b0), s1 = mx_inverse_scale(b1);
      uint32_t q0[4], q1[4];
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        q0[g] = q1[g] = 0u;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 u = unpack2<BF16>(x[g * 8 + 2 * j]), v = unpack2<BF16>(x[g * 8 + 2 * j + 1]);
          q0[g] |= mx_pack2(u.x * s0, v.x * s0) << (8 * j);
          q1[g] |= mx_pack2(u.y * s1, v.y * s1) << (8 * j);
        }
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
  extern __shared__ int table[];
  int* offs = table;
  int* start = table + p.groups + 1;
  mx_table(p, offs, start);
  const int lane = static_cast<int>(lane_id());
  const int chunks = (p.cols + 1023) / 1024;
  const int64_t items = p.batch * p.rows * chunks;
  for (int64_t it = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5); it < items;
       it += static_cast<int64_t>(gridDim.x) * 8) {
    const int64_t row = it / chunks;
    const int c0 = static_cast<int>(it - row * chunks) * 1024 + lane * 8;
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
      if (c >= p.cols) break;
      const float s = mx_scale_value(sb[i]);
      float v[8];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const __half2_raw h = __nv_cvt_fp4x2_to_halfraw2(static_cast<__nv_fp4x2_storage_t>(x[i] >> (8 * j)), __NV_E2M1);
        const float2 f = __half22float2(__half2(h));
        v[2 * j] = f.x * s;
        v[2 * j + 1] = f.y * s;
      }
      if (p.out_f32) {
        float4* dst = reinterpret_cast<float4*>(reinterpret_cast<float*>(p.out) + row * p.cols + c);
        dst[0] = make_float4(v[0], v[1], v[2], v[3]);
        dst[1] = make_float4(v[4], v[5], v[6], v[7]);
      } else {
        *reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(p.out) + row * p.cols + c) =
            make_uint4(pack2<BF16>(v[0], v[1]), pack2<BF16>(v[2], v[3]), pack2<BF16>(v[4], v[5]), pack2<BF16>(v[6], v[7]));
      }
    }
  }
}

}  // namespace ge
