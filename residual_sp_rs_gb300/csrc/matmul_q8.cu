// matmul_q8.cu -- C = A B^T of 8-bit tensors with a power-of-two scale per 128
// values along K.
//
//   C[i,j] = sum_k (2^sa[i,k/128] qa[i,k]) (2^sb[j,k/128] qb[j,k]),
//
// both factors exact in fp32, sums in fp32, one rounding to C's type.  64 x 64
// tiles of C, 16 columns of K a step through shared memory, 4 x 4 sums a
// thread.
#include "common.cuh"
#include "launch.h"
#include "q8.cuh"

namespace spf {

namespace {

constexpr int kTile = 64, kStep = 16;

__device__ __forceinline__ float element(const uint8_t* p, const uint8_t* scale, int64_t ld, int64_t lds, int srows,
                                         bool e5m2, int64_t row, int64_t rows, int64_t k, int64_t K) {
  if (row >= rows || k >= K) return 0.f;
  float lo, hi;
  q8_unpack2(p[row * ld + k], e5m2, lo, hi);
  return lo * q8_scale(scale[row / srows * lds + (k >> 7)]);
}

__global__ void __launch_bounds__(256) sp_matmul_q8_kernel(const MatmulArgs a) {
  __shared__ float sa[kStep][kTile + 1], sb[kStep][kTile + 1];
  const int64_t ntiles = (a.N + kTile - 1) / kTile;
  const int64_t m0 = blockIdx.x / ntiles * kTile, n0 = blockIdx.x % ntiles * kTile;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  grid_dep_wait();
  grid_dep_launch_dependents();
  float acc[4][4] = {};
  for (int64_t k0 = 0; k0 < a.K; k0 += kStep) {
    for (int i = threadIdx.x; i < kTile * kStep; i += 256) {
      const int r = i / kStep, k = i % kStep;
      sa[k][r] = element(a.a, a.a_scale, a.lda, a.lda_scale, a.a_scale_rows, a.a_e5m2, m0 + r, a.M, k0 + k, a.K);
      sb[k][r] = element(a.b, a.b_scale, a.ldb, a.ldb_scale, a.b_scale_rows, a.b_e5m2, n0 + r, a.N, k0 + k, a.K);
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kStep; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] += sa[k][ty + 16 * i] * sb[k][tx + 16 * j];
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t m = m0 + ty + 16 * i, n = n0 + tx + 16 * j;
      if (m >= a.M || n >= a.N) continue;
      if (a.c_f32) {
        float* p = static_cast<float*>(a.c) + m * a.ldc + n;
        *p = a.accumulate ? *p + acc[i][j] : acc[i][j];
      } else {
        static_cast<__nv_bfloat16*>(a.c)[m * a.ldc + n] = __float2bfloat16_rn(acc[i][j]);
      }
    }
}

}  // namespace

cudaError_t launch_matmul_q8(const MatmulArgs& a, cudaStream_t st) {
  const int64_t tiles = ((a.M + kTile - 1) / kTile) * ((a.N + kTile - 1) / kTile);
  return pdl_launch(sp_matmul_q8_kernel, dim3((unsigned)tiles), dim3(256), 0, st, a);
}

}  // namespace spf
