// w4_kernel.cuh -- few rows times a weight held in 4 bits with group scales (layout:
// w4_quant.cuh): Y[t][n] = epilog(sum_k X[t][k] s_g (q[n][k] - z_g)), and as a gated
// layer (two matrices).
//
// The weight is streamed once, 32 bytes a lane and instruction, and is the bound:
// N K / 2 bytes and the scales. q - z is a small integer, exact in the 16-bit type:
// a shift, a mask, an or with 128's (1024's) bits and one subtraction make two of them, with no
// rounding of weights anywhere. A warp multiplies 16 features (the M slot) x 32
// columns with 8 NT rows of X (the N slot) by m16n8k16 tensor-core instructions,
// adds up a group in fp32, then adds the group's sum times its scale to the
// feature's sum. (The tensor memory path wants its operand in shared or tensor
// memory and 128 features at a time, and could scale the sums only per tile
// read; with few rows the instructions per weight, not the MMA rate, count.)
//
// A CTA takes a run of feature tiles; its warps share each tile's columns, 128 at a
// time in turn, across tile ends, DEPTH tiles of loads ahead, and join their
// fp32 sums through shared memory in a fixed order. X (its columns of the
// slice) stays in shared memory. Where X of all columns does not fit, the columns
// are cut into slices for different CTAs, which leave fp32 sums in the workspace for
// w4_finish_kernel.
#pragma once

#include "activation.cuh"
#include "tile_kernel.cuh"
#include "w4_quant.cuh"

namespace ge {

struct W4MulParams {
  int32_t T, N, K;
  int32_t rt, kt;        // 16-feature tiles of a matrix; 128-column blocks
  int32_t items;         // feature tiles (MATS = 2, not gated: pairs of them)
  int32_t slices, slice_kt;  // column slices, blocks of each (the last may have fewer)
  int32_t epi, act;      // EpiKind; gated: an ActKind
  int32_t bias_f32, out_f32;
  const void* X;
  const uint8_t* q;
  const void* scales;
  const uint8_t* zeros;
  const void* bias;
  void* out;
  float* sums;           // slices > 1: [slices][matrices][T][16 rt]
};

template <int NT>
struct W4Shape {
  static constexpr int WARPS = NT <= 2 ? 16 : 8;
  static constexpr int BUFS = NT <= 2 ? 2 : 1;       // of the join
  static constexpr int COL = 20;                      // floats of a row's 16 features in it (no bank conflicts)
  static constexpr int PART = 8 * NT * COL;           // floats of a warp and matrix
};

// bytes of a row of X in shared memory: 64 past a multiple of 128, so that rows are on other banks
__host__ __device__ constexpr int w4_row_bytes(int blocks) { return blocks * 256 + 64; }

struct W4Tile {
  uint32_t w[8];   // [4 blocks of 32 columns][r]
  uint32_t s[4];   // [groups]: the scales of both rows
  uint32_t z[2];   // [groups][r] bytes
};

template <int NG>
__device__ __forceinline__ void w4_load_tile(W4Tile& t, const W4MulParams& p, int64_t tile) {
  const uint32_t lane = lane_id();
  asm volatile("ld.global.nc.L1::no_allocate.L2::evict_first.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(t.w[0]), "=r"(t.w[1]), "=r"(t.w[2]), "=r"(t.w[3]), "=r"(t.w[4]), "=r"(t.w[5]), "=r"(t.w[6]), "=r"(t.w[7])
               : "l"(p.q + tile * 1024 + lane * 32));
  const uint32_t* s = reinterpret_cast<const uint32_t*>(p.scales) + (tile * 8 + (lane >> 2)) * NG;
  if constexpr (NG == 4) {
    const uint4 v = __ldg(reinterpret_cast<const uint4*>(s));
    t.s[0] = v.x, t.s[1] = v.y, t.s[2] = v.z, t.s[3] = v.w;
  } else if constexpr (NG == 2) {
    const uint2 v = __ldg(reinterpret_cast<const uint2*>(s));
    t.s[0] = v.x, t.s[1] = v.y;
  } else {
    t.s[0] = __ldg(s);
  }
  if (p.zeros) {
    const uint8_t* z = p.zeros + (tile * 8 + (lane >> 2)) * (2 * NG);
    if constexpr (NG == 4) {
      const uint2 v = __ldg(reinterpret_cast<const uint2*>(z));
      t.z[0] = v.x, t.z[1] = v.y;
    } else if constexpr (NG == 2) {
      t.z[0] = __ldg(reinterpret_cast<const uint32_t*>(z));
    } else {
      t.z[0] = __ldg(reinterpret_cast<const uint16_t*>(z));
    }
  } else {
    t.z[0] = t.z[1] = 0x08080808u;
  }
}

template <bool BF16>
__device__ __forceinline__ uint32_t w4_sub(uint32_t a, uint32_t b) {
  if constexpr (BF16) {
    const __nv_bfloat162 r = __hsub2(*reinterpret_cast<__nv_bfloat162*>(&a), *reinterpret_cast<__nv_bfloat162*>(&b));
    return *reinterpret_cast<const uint32_t*>(&r);
  } else {
    const __half2 r = __hsub2(*reinterpret_cast<__half2*>(&a), *reinterpret_cast<__half2*>(&b));
    return *reinterpret_cast<const uint32_t*>(&r);
  }
}

// zero point z (0 .. 127) as two halves of 128 + z (1024 + z), exact in the type
template <bool BF16>
__device__ __forceinline__ uint32_t w4_zero2(uint32_t z) {
  if constexpr (BF16) {
    // 128 + z: the exponent of 128, z in the 7 bits below
    return 0x43004300u + z * 0x00010001u;
  } else {
    return 0x64006400u + z * 0x00010001u;
  }
}

// q - z of two neighbouring columns, exactly
template <bool BF16>
__device__ __forceinline__ uint32_t w4_pair(uint32_t word, int m, uint32_t zero2) {
  constexpr uint32_t kOne = BF16 ? 0x43004300u : 0x64006400u;
  return w4_sub<BF16>(((word >> (4 * m)) & 0x000f000fu) | kOne, zero2);
}

template <bool BF16>
__device__ __forceinline__ void w4_mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                       uint32_t b1) {
  if constexpr (BF16)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// One output from its sums (gated: gate and up projection), feature n of row t.
template <bool BF16>
__device__ __forceinline__ void w4_output(const W4MulParams& p, float a, float b, int t, int n) {
  const bool gated = p.epi == EPI_GATED;
  if (p.bias && p.epi != EPI_STORE) {
    a += load_bias<BF16>(p.bias, p.bias_f32, n);
    if (gated) b += load_bias<BF16>(p.bias, p.bias_f32, p.N + n);
  }
  if (gated || p.epi == EPI_GELU_BIAS) {
    float z[2] = {a, a}, v[2], none[2];
    act_values<2, false>(gated ? p.act : ACT_GELU, z, v, none);
    a = gated ? v[0] * b : v[0];
  } else if (p.epi == EPI_RELU_BIAS) {
    a = a > 0.f ? a : 0.f;
  }
  const int64_t o = static_cast<int64_t>(t) * p.N + n;
  if (p.out_f32)
    reinterpret_cast<float*>(p.out)[o] = a;
  else
    reinterpret_cast<uint16_t*>(p.out)[o] = w4_round16<BF16>(a);
}

// MATS streams of tiles share the fragments of X: the gate's and the up
// projection's tile (GATED), or two neighbouring tiles of one matrix.
template <int NT, int MATS, bool GATED, int NG, bool BF16>
__global__ void __launch_bounds__(32 * W4Shape<NT>::WARPS, 1) w4_kernel(const W4MulParams p) {
  using S = W4Shape<NT>;
  constexpr int W = S::WARPS, THREADS = 32 * W;
  constexpr int DEPTH = MATS == 1 ? 4 : 2;  // tiles of each stream whose loads are under way
  static_assert(MATS == 2 || !GATED, "a gated layer has two streams");
  extern __shared__ __align__(16) uint8_t w4_smem[];
  float* join = reinterpret_cast<float*>(w4_smem);  // [BUFS][W][MATS][PART]
  uint8_t* xs = w4_smem + S::BUFS * W * MATS * S::PART * 4;

  const uint32_t lane = lane_id(), warp = threadIdx.x >> 5, g = lane >> 2, c = lane & 3u;
  const int row0 = blockIdx.z * 8 * NT, rows = min(p.T - row0, 8 * NT);
  const int kb0 = blockIdx.y * p.slice_kt, nkb = min(p.kt - kb0, p.slice_kt);
  const int lo = static_cast<int>(static_cast<int64_t>(blockIdx.x) * p.items / gridDim.x);
  const int hi = static_cast<int>(static_cast<int64_t>(blockIdx.x + 1) * p.items / gridDim.x);
  wait_for_inputs();

  const auto tile_of = [&](int item, int m, int b) {
    const int i = GATED ? m * p.rt + item : MATS == 2 ? min(2 * item + m, p.rt - 1) : item;
    return static_cast<int64_t>(i) * p.kt + kb0 + b;
  };
  // this warp's sequence: blocks warp, warp + W, ... of the run of tiles, (item, b)
  W4Tile ring[DEPTH][MATS];
  int li = lo, lb = static_cast<int>(warp);  // the next to be loaded
  while (lb >= nkb) {
    lb -= nkb;
    ++li;
  }
  const auto load = [&](W4Tile (&t)[MATS]) {
    if (li < hi) {
#pragma unroll
      for (int m = 0; m < MATS; ++m) w4_load_tile<NG>(t[m], p, tile_of(li, m, lb));
      lb += W;
      while (lb >= nkb) {
        lb -= nkb;
        ++li;
      }
    }
  };
  int item = lo, b = static_cast<int>(warp);
  while (b >= nkb) {
    b -= nkb;
    ++item;
  }
#pragma unroll
  for (int d = 0; d < DEPTH; ++d) load(ring[d]);

  // X: this slice's columns of this CTA's rows, zeros past K
  const int xb = w4_row_bytes(p.slice_kt);
  const int units = nkb * 16;  // of 8 columns
  for (int e = threadIdx.x; e < rows * units; e += THREADS) {
    const int r = e / units, u = e - r * units, col = kb0 * 128 + u * 8;
    const uint4 v = col < p.K ? __ldg(reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(p.X) +
                                                                     static_cast<int64_t>(row0 + r) * p.K + col))
                              : make_uint4(0, 0, 0, 0);
    *reinterpret_cast<uint4*>(xs + r * xb + u * 16) = v;
  }
  __syncthreads();

  float acc[MATS][NT][4];
  const auto clear = [&]() {
#pragma unroll
    for (int m = 0; m < MATS; ++m)
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[m][t][e] = 0.f;
  };
  clear();
  const uint32_t x0 = smem_u32(xs) + g * xb + c * 16;

  // the sums of item `at` are complete: join the warps' and finish
  int turn = 0;
  const auto finish = [&](int at) {
    float* buf = join + (S::BUFS == 2 ? (turn & 1) * (W * MATS * S::PART) : 0);
    float* mine = buf + warp * (MATS * S::PART);
    if (S::BUFS == 1 && turn > 0) __syncthreads();  // the last one has been read
    ++turn;
#pragma unroll
    for (int m = 0; m < MATS; ++m)
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          mine[m * S::PART + (t * 8 + 2 * c + (e & 1)) * S::COL + g + 8 * (e >> 1)] = acc[m][t][e];
    clear();
    __syncthreads();
    const int n_out = rows * 16 * (GATED ? 1 : MATS);
    for (int o = threadIdx.x; o < n_out; o += THREADS) {
      const int f = o & 15, m = GATED ? 0 : (o >> 4) % MATS, t = GATED ? o >> 4 : (o >> 4) / MATS;
      const float* from = buf + m * S::PART + t * S::COL + f;
      float a = 0.f, u = 0.f;
#pragma unroll
      for (int w = 0; w < W; ++w) {
        a += from[w * (MATS * S::PART)];
        if constexpr (GATED) u += from[w * (MATS * S::PART) + S::PART];
      }
      const int n = (GATED ? at : MATS * at + m) * 16 + f;
      if (n >= p.N) continue;
      if (p.slices == 1) {
        w4_output<BF16>(p, a, u, row0 + t, n);
      } else {
        const int64_t ld = static_cast<int64_t>(p.rt) * 16;
        float* to = p.sums + (static_cast<int64_t>(blockIdx.y) * (GATED ? 2 : 1) * p.T + row0 + t) * ld + n;
        to[0] = a;
        if constexpr (GATED) to[p.T * ld] = u;
      }
    }
  };

  const auto work = [&](const W4Tile (&tile)[MATS], int block) {
    const uint32_t xk = x0 + block * 256;
    float part[MATS][NT][4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {  // 32 columns
      constexpr int PER = 4 / NG;  // of them in a group
      if (k % PER == 0) {
#pragma unroll
        for (int m = 0; m < MATS; ++m)
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) part[m][t][e] = 0.f;
      }
      uint4 x[NT];
#pragma unroll
      for (int t = 0; t < NT; ++t)
        x[t] = t * 8 + static_cast<int>(g) < rows ? ld_shared_v4(xk + t * 8 * xb + k * 64) : make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int m = 0; m < MATS; ++m) {
        const uint32_t zz = tile[m].z[(k / PER) >> 1] >> (16 * ((k / PER) & 1));
        const uint32_t z0 = w4_zero2<BF16>(zz & 127u), z1 = w4_zero2<BF16>((zz >> 8) & 127u);
        const uint32_t w0 = tile[m].w[2 * k], w1 = tile[m].w[2 * k + 1];
        uint32_t a[4], bq[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          a[e] = w4_pair<BF16>(w0, e, z0);
          bq[e] = w4_pair<BF16>(w1, e, z1);
        }
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          w4_mma<BF16>(part[m][t], a[0], bq[0], a[1], bq[1], x[t].x, x[t].y);
          w4_mma<BF16>(part[m][t], a[2], bq[2], a[3], bq[3], x[t].z, x[t].w);
        }
        if (k % PER == PER - 1) {
          const uint32_t s2 = tile[m].s[k / PER];
          const float s0 = w4_float<BF16>(static_cast<uint16_t>(s2 & 0xffffu));
          const float s1 = w4_float<BF16>(static_cast<uint16_t>(s2 >> 16));
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            acc[m][t][0] = fmaf(s0, part[m][t][0], acc[m][t][0]);
            acc[m][t][1] = fmaf(s0, part[m][t][1], acc[m][t][1]);
            acc[m][t][2] = fmaf(s1, part[m][t][2], acc[m][t][2]);
            acc[m][t][3] = fmaf(s1, part[m][t][3], acc[m][t][3]);
          }
        }
      }
    }
  };

  int at = lo;  // the item that acc holds
  while (at < hi) {
#pragma unroll
    for (int d = 0; d < DEPTH; ++d) {
      // (every warp finishes every item once, also one that had none of its blocks)
      while (at < item && at < hi) finish(at++);
      if (at < hi) {
        work(ring[d], b);
        load(ring[d]);
        b += W;
        while (b >= nkb) {
          b -= nkb;
          ++item;
        }
      }
    }
  }
}

// Column slices' sums added in order, then the epilog.
template <bool BF16>
__global__ void __launch_bounds__(256) w4_finish_kernel(const W4MulParams p) {
  wait_for_inputs();
  const int64_t ld = static_cast<int64_t>(p.rt) * 16, mat = static_cast<int64_t>(p.T) * ld;
  const int mats = p.epi == EPI_GATED ? 2 : 1;
  for (int64_t o = blockIdx.x * 256ll + threadIdx.x; o < static_cast<int64_t>(p.T) * p.N; o += gridDim.x * 256ll) {
    const int t = static_cast<int>(o / p.N), n = static_cast<int>(o - static_cast<int64_t>(t) * p.N);
    const float* from = p.sums + t * ld + n;
    float a = 0.f, u = 0.f;
    for (int s = 0; s < p.slices; ++s) {
      a += __ldcg(from + s * mats * mat);
      if (mats == 2) u += __ldcg(from + (s * mats + 1) * mat);
    }
    w4_output<BF16>(p, a, u, t, n);
  }
}

}  // namespace ge
