// quant_q8.cu -- quantisation to 8 bits with a power-of-two scale per group of
// 128 values: along the rows (q), along the columns (qt, the transposed
// tensor), or both from one read of the input.
//
// q[i,k] = rn(x[i,k] 2^-s), s the group's exponent (q8.cuh).  Bound by memory:
// the input once and one byte per element and output.
//
// A CTA takes a 128 x 128 tile, in which every group of either direction (and
// a 128 x 128 block) is whole.  Thread (g, c) of 16 x 16 holds the 8 x 8 block
// of rows 8g.. and columns 8c.. in registers: a row's maximum is then four
// shuffles over 16 lanes, a column's one shuffle and a sum over eight warps
// in shared memory, and the bytes of a column's eight rows form one 8-byte
// word of the transposed tile.  That tile goes through shared memory (word g
// of column k at slot g ^ (k / 8), so that neither side meets a bank conflict)
// and leaves in 128-byte lines.
#include "common.cuh"
#include "launch.h"
#include "q8.cuh"

namespace spf {

namespace {

constexpr int kQuantThreads = 256;

enum class Src { kF32, kBf16, kQ8 };

template <Src S>
struct SrcBytes {
  static constexpr int v = S == Src::kF32 ? 4 : S == Src::kBf16 ? 2 : 1;
};

// Eight consecutive elements of a row from column `col` on, zero past K.
template <Src S>
__device__ __forceinline__ void load8(const QuantArgs& a, int64_t row, int64_t col, float scale, float (&v)[8]) {
  const char* p = static_cast<const char*>(a.x) + (row * a.ldx + col) * SrcBytes<S>::v;
  uint32_t w[8] = {};
  if (a.vec && col + 8 <= a.K) {
    if constexpr (S == Src::kQ8) {
      const uint2 u = __ldcs(reinterpret_cast<const uint2*>(p));
      w[0] = u.x;
      w[1] = u.y;
    } else {
#pragma unroll
      for (int i = 0; i < SrcBytes<S>::v / 2; ++i) {
        const uint4 u = ld_stream(p + 16 * i);
        w[4 * i] = u.x;
        w[4 * i + 1] = u.y;
        w[4 * i + 2] = u.z;
        w[4 * i + 3] = u.w;
      }
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      if (col + e >= a.K) continue;
      if constexpr (S == Src::kF32)
        w[e] = *(reinterpret_cast<const uint32_t*>(p) + e);
      else if constexpr (S == Src::kBf16)
        w[e / 2] |= (uint32_t) * (reinterpret_cast<const uint16_t*>(p) + e) << (16 * (e & 1));
      else
        w[e / 4] |= (uint32_t) * (reinterpret_cast<const uint8_t*>(p) + e) << (8 * (e & 3));
    }
  }
  if constexpr (S == Src::kF32) {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = __uint_as_float(w[e]);
  } else if constexpr (S == Src::kBf16) {
#pragma unroll
    for (int i = 0; i < 4; ++i) Act16<__nv_bfloat16>::unpack_word(w[i], v[2 * i], v[2 * i + 1]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      q8_unpack2(w[i / 2] >> (16 * (i & 1)), a.x_e5m2 != 0, v[2 * i], v[2 * i + 1]);
      v[2 * i] *= scale;
      v[2 * i + 1] *= scale;
    }
  }
}

// Up to eight bytes to p, `n` of them inside the tensor.
__device__ __forceinline__ void store8(uint8_t* p, uint2 w, int64_t n) {
  if (n >= 8) {
    *reinterpret_cast<uint2*>(p) = w;
    return;
  }
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (e < n) p[e] = (uint8_t)((e < 4 ? w.x : w.y) >> (8 * (e & 3)));
}

template <Src S, bool E5M2, bool BLOCK>
__global__ void __launch_bounds__(kQuantThreads) sp_quant_q8_kernel(const QuantArgs a) {
  __shared__ uint32_t wmax[kQuantThreads / 32][kQ8Group];  // column maxima of each warp
  __shared__ uint8_t cscale[kQ8Group];
  __shared__ __align__(16) uint2 tile[kQ8Group * 16];      // transposed bytes

  const int c = threadIdx.x & 15, g = threadIdx.x >> 4, warp = threadIdx.x >> 5;
  const int64_t tm = blockIdx.x / a.ktiles, tk = blockIdx.x - tm * a.ktiles;
  const int64_t row0 = tm * kQ8Group + 8 * g, col0 = tk * kQ8Group + 8 * c;

  grid_dep_wait();
  grid_dep_launch_dependents();

  float v[8][8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float scale = 1.f;
    if (row0 + i < a.M) {
      if constexpr (S == Src::kQ8)
        scale = q8_scale(a.x_scale[(row0 + i) / a.x_scale_rows * a.ldx_scale + tk]);
      load8<S>(a, row0 + i, col0, scale, v[i]);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[i][e] = 0.f;
    }
  }

  uint32_t rsb[8];  // scale byte of each of this thread's rows
  uint32_t bsb = 0;
  if constexpr (BLOCK) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) m = max(m, abs_bits(v[i][e]));
    m = lanes_max<32>(m);
    if ((threadIdx.x & 31) == 0) wmax[warp][0] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kQuantThreads / 32; ++w) m = max(m, wmax[w][0]);
    bsb = q8_scale_byte<E5M2>(m);
#pragma unroll
    for (int i = 0; i < 8; ++i) rsb[i] = bsb;
    if (threadIdx.x == 0) {
      if (a.q) a.q_scale[tm * a.ldq_scale + tk] = (uint8_t)bsb;
      if (a.qt) a.qt_scale[tk * a.ldqt_scale + tm] = (uint8_t)bsb;
    }
  } else if (a.q) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      uint32_t m = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) m = max(m, abs_bits(v[i][e]));
      rsb[i] = q8_scale_byte<E5M2>(lanes_max<16>(m));
      if (c == 0 && row0 + i < a.M) a.q_scale[(row0 + i) * a.ldq_scale + tk] = (uint8_t)rsb[i];
    }
  }
  if (a.q) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (row0 + i >= a.M) continue;
      const float inv = q8_inv_scale(rsb[i]);
      store8(a.q + (row0 + i) * a.ldq + col0,
             make_uint2(q8_pack4<E5M2>(v[i][0] * inv, v[i][1] * inv, v[i][2] * inv, v[i][3] * inv),
                        q8_pack4<E5M2>(v[i][4] * inv, v[i][5] * inv, v[i][6] * inv, v[i][7] * inv)),
             a.K - col0);
    }
  }
  if (!a.qt) return;

  if constexpr (!BLOCK) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) m = max(m, abs_bits(v[i][e]));
      m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 16));  // the warp's other row group
      if ((threadIdx.x & 16) == 0) wmax[warp][8 * c + e] = m;
    }
    __syncthreads();
    if (threadIdx.x < kQ8Group) {
      uint32_t m = 0;
#pragma unroll
      for (int w = 0; w < kQuantThreads / 32; ++w) m = max(m, wmax[w][threadIdx.x]);
      const uint32_t sb = q8_scale_byte<E5M2>(m);
      cscale[threadIdx.x] = (uint8_t)sb;
      const int64_t col = tk * kQ8Group + threadIdx.x;
      if (col < a.K) a.qt_scale[col * a.ldqt_scale + tm] = (uint8_t)sb;
    }
    __syncthreads();
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float inv = q8_inv_scale(BLOCK ? bsb : (uint32_t)cscale[8 * c + e]);
    tile[(8 * c + e) * 16 + (g ^ c)] =
        make_uint2(q8_pack4<E5M2>(v[0][e] * inv, v[1][e] * inv, v[2][e] * inv, v[3][e] * inv),
                   q8_pack4<E5M2>(v[4][e] * inv, v[5][e] * inv, v[6][e] * inv, v[7][e] * inv));
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int k = g + 16 * i;  // column of the tile; lane c takes its rows 8c..
    const int64_t col = tk * kQ8Group + k, row = tm * kQ8Group + 8 * c;
    if (col < a.K && row < a.M)
      store8(a.qt + col * a.ldqt + row, tile[k * 16 + (c ^ (k >> 3))], a.M - row);
  }
}

template <Src S>
cudaError_t launch_src(const QuantArgs& a, bool e5m2, bool block, unsigned grid, cudaStream_t st) {
  void (*k)(const QuantArgs) =
      e5m2 ? (block ? sp_quant_q8_kernel<S, true, true> : sp_quant_q8_kernel<S, true, false>)
           : (block ? sp_quant_q8_kernel<S, false, true> : sp_quant_q8_kernel<S, false, false>);
  return pdl_launch(k, dim3(grid), dim3(kQuantThreads), 0, st, a);
}

}  // namespace

cudaError_t launch_quant_q8(const QuantArgs& a, int x_dtype, bool e5m2, bool block, cudaStream_t st) {
  const unsigned grid = (unsigned)((a.M + kQ8Group - 1) / kQ8Group * a.ktiles);
  switch (x_dtype) {
    case SP_ELEM_F32: return launch_src<Src::kF32>(a, e5m2, block, grid, st);
    case SP_ELEM_BF16: return launch_src<Src::kBf16>(a, e5m2, block, grid, st);
    default: return launch_src<Src::kQ8>(a, e5m2, block, grid, st);
  }
}

}  // namespace spf
