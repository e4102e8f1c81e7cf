// quant_q8.cu -- quantisation to 8 bits with a power-of-two scale per group of
// 128 values: along the rows (q), along the columns (qt, the transposed
// tensor), or both from one read of the input.
//
// q[i,k] = rn(x[i,k] 2^-s), s the group's exponent (q8.cuh).  Bound by memory:
// the input once and one byte per element and output.
//
// A CTA takes a 128 x 128 tile, in which every group of either direction (and
// a 128 x 128 block) is whole.  A thread holds the block of its kRows rows and
// 8 columns in registers: bf16 as packed words, 8 rows; fp32 and 8-bit input as
// fp32 values, 4 rows, so that 64 registers do and 32 warps fit on an SM.  The
// rows' maxima are then taken over 16 lanes, a column's by one shuffle and
// over the warps in shared memory, and the bytes of a column's rows
// form one word of the transposed tile.  That tile goes through shared memory
// (8-byte word r of column k at slot r ^ (k / 8), so that neither side meets a
// bank conflict) and leaves 128 bytes of a column at a time.
//
// An 8-bit tile is 16 KB, too little for the resident CTAs to keep the memory
// busy between their barriers.  So two CTAs stay on each SM, and tiled bulk
// copies bring the next kRing tiles of each while one is worked on.  Waits for
// them are bounded; a CTA whose wait runs out takes its tiles by plain loads
// from there on, so that only time is lost.
//
// 66 M values: bf16 along the rows 32.5 us (90% of the copy bandwidth), along
// the columns 35 (83%), both 47 (82%); 8-bit along the rows 29 us (67%), along
// the columns 35 (55%); 33.5 M fp32 values in blocks, both ways, 35 us (85%).
// The 8-bit columns fill no pipe (issue 56%, shared memory 48%): 13 instructions
// a value between four barriers a tile, whose warps stall at the barriers, on
// shared memory and on their own last instruction in equal parts.
#include "common.cuh"
#include "launch.h"
#include "q8.cuh"
#include "umma.cuh"

namespace spf {

namespace {

constexpr int kRing = 3;                    // 8-bit input: tiles in flight per CTA
constexpr uint32_t kTileBytes = 128 * 128;

enum class Src { kF32, kBf16, kQ8 };

template <Src S>
struct Shape {
  static constexpr int kRows = S == Src::kBf16 ? 8 : 4;      // rows per thread
  static constexpr int kThreads = 16 * kQ8Group / kRows;
  static constexpr int kWords = S == Src::kBf16 ? 4 : 8;     // registers per row
};

// Maxima of R (4 or 8) rows over 16 lanes: at each step a lane hands over the
// half of the rows that its partner keeps, so R + log2(16 / R) shuffles do
// instead of 4 R, and what follows is worked out once per row instead of in 16
// lanes.  The lane c of 16 ends up with row held_row(c), lane lane_of(r) has row r.
template <int R>
__device__ __forceinline__ uint32_t rows_max(uint32_t (&m)[R], int c) {
#pragma unroll
  for (int n = R / 2, off = 8; off > 0; n /= 2, off /= 2) {
    if (n >= 1) {
      const bool upper = c & off;
#pragma unroll
      for (int j = 0; j < n; ++j) {
        const uint32_t keep = upper ? m[n + j] : m[j], send = upper ? m[j] : m[n + j];
        m[j] = max(keep, __shfl_xor_sync(0xFFFFFFFFu, send, off));
      }
    } else {
      m[0] = max(m[0], __shfl_xor_sync(0xFFFFFFFFu, m[0], off));
    }
  }
  return m[0];
}
template <int R>
__device__ __forceinline__ constexpr int held_row(int c) {
  return c / (16 / R);
}
template <int R>
__device__ __forceinline__ constexpr int lane_of(int r) {
  return r * (16 / R);
}

// Eight consecutive elements of a row from column `col` on, zero past K.
template <Src S>
__device__ __forceinline__ void load8(const QuantArgs& a, int32_t row, int32_t col, uint32_t (&w)[Shape<S>::kWords]) {
  const char* p = static_cast<const char*>(a.x) + ((int64_t)row * a.ldx + col) * (S == Src::kF32 ? 4 : 2);
  if (a.vec && a.K - col >= 8) {
#pragma unroll
    for (int i = 0; i < (S == Src::kF32 ? 4 : 2) / 2; ++i) {
      const uint4 u = ld_stream(p + 16 * i);
      w[4 * i] = u.x;
      w[4 * i + 1] = u.y;
      w[4 * i + 2] = u.z;
      w[4 * i + 3] = u.w;
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < Shape<S>::kWords; ++i) w[i] = 0u;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    if (e >= a.K - col) continue;
    if constexpr (S == Src::kF32)
      w[e] = *(reinterpret_cast<const uint32_t*>(p) + e);
    else
      w[e / 2] |= (uint32_t) * (reinterpret_cast<const uint16_t*>(p) + e) << (16 * (e & 1));
  }
}

// Eight consecutive bytes of a row of an 8-bit x, zero past K.
__device__ __forceinline__ uint2 load8_q8(const QuantArgs& a, int32_t row, int32_t col) {
  const uint8_t* p = static_cast<const uint8_t*>(a.x) + (int64_t)row * a.ldx + col;
  if (a.K - col >= 8) return *reinterpret_cast<const uint2*>(p);
  uint32_t w[2] = {};
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (e < a.K - col) w[e / 4] |= (uint32_t)p[e] << (8 * (e & 3));
  return make_uint2(w[0], w[1]);
}

// Up to N (8 or 16) bytes to p, `n` of them inside the tensor.
__device__ __forceinline__ void store8(uint8_t* p, uint2 w, int32_t n) {
  if (n >= 8) {
    *reinterpret_cast<uint2*>(p) = w;
    return;
  }
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (e < n) p[e] = (uint8_t)((e < 4 ? w.x : w.y) >> (8 * (e & 3)));
}
__device__ __forceinline__ void store16(uint8_t* p, uint4 w, int32_t n) {
  if (n >= 16) {
    *reinterpret_cast<uint4*>(p) = w;
    return;
  }
  store8(p, make_uint2(w.x, w.y), n);
  store8(p + 8, make_uint2(w.z, w.w), n - 8);
}

template <Src S, bool E5M2, bool BLOCK, bool XE5M2>
__global__ void __launch_bounds__(Shape<S>::kThreads, 1024 / Shape<S>::kThreads) sp_quant_q8_kernel(const QuantArgs a, const __grid_constant__ CUtensorMap map) {
  constexpr int kRows = Shape<S>::kRows, kThreads = Shape<S>::kThreads, kWarps = kThreads / 32;
  // column 8c + e: maxima of each warp at 17e + c, 2^-s at 2c + (e & 1) of pair e / 2
  __shared__ uint32_t wmax[kWarps][8 * 17];
  __shared__ float cinv[4][32];
  __shared__ __align__(16) uint2 tile[kQ8Group * 16];  // transposed bytes

  const int c = threadIdx.x & 15, g = threadIdx.x >> 4, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  extern __shared__ __align__(128) unsigned char ring_raw[];
  unsigned char* const ring = ring_raw + ((128u - (smem_addr(ring_raw) & 127u)) & 127u);
  __shared__ uint64_t landed[kRing];
  __shared__ uint32_t open_tile, open_stage, open_phase;  // thread 0's: where a wait ran out
  if constexpr (S == Src::kQ8) {
    if (threadIdx.x == 0) {
      prefetch_tensor_map(&map);
      for (int s = 0; s < kRing; ++s) mbar_init(&landed[s], 1);
      fence_mbar_init();
    }
    __syncthreads();
  }
  grid_dep_wait();
  grid_dep_launch_dependents();

  // 8-bit x: tile `t` to stage `s` of the ring
  auto fetch = [&](uint32_t t, int s) {
    if (t >= (uint32_t)a.tiles) return;
    if (blockIdx.x == 0 && a.drop_stage >= 0 && t == (uint32_t)a.drop_stage * gridDim.x) return;  // test hook: never lands
    const uint32_t tm = t / (uint32_t)a.ktiles, tk = t - tm * (uint32_t)a.ktiles;
    mbar_arrive_expect_tx(&landed[s], kTileBytes);
    tma_load_2d<1>(smem_addr(ring) + s * kTileBytes, &map, (int32_t)(tk * kQ8Group), (int32_t)(tm * kQ8Group),
                   smem_addr(&landed[s]));
  };
  if constexpr (S == Src::kQ8)
    if (threadIdx.x == 0)
      for (int s = 0; s < kRing; ++s) fetch(blockIdx.x + s * gridDim.x, s);
  int stage = 0;
  uint32_t phase = 0;
  bool copies = true;  // no wait of this CTA has run out

  // tiles, rows and columns stay below 2^31; a.tiles + kRing * gridDim.x below 2^32
  for (uint32_t t = blockIdx.x; t < (uint32_t)a.tiles; t += gridDim.x) {
    const uint32_t tm = t / (uint32_t)a.ktiles, tk = t - tm * (uint32_t)a.ktiles;
    const int32_t row0 = (int32_t)tm * kQ8Group + kRows * g, col0 = (int32_t)tk * kQ8Group + 8 * c;
    const int32_t rows = a.M - row0;  // of this thread's inside the tensor (may be more, or negative)
    uint32_t w[kRows][Shape<S>::kWords] = {};
    uint32_t xs = 127u;  // 8-bit x: lane i of the 16 that share rows holds row i's scale byte
    if constexpr (S == Src::kQ8)
      if (c < kRows && c < rows)
        xs = a.x_scale[(int64_t)((row0 + c) >> a.x_scale_shift) * a.ldx_scale + tk];
    if constexpr (S == Src::kQ8) {
      const bool was = copies, ok = was && mbar_wait(&landed[stage], phase, a.wait_ns);
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        const uint2 u = *reinterpret_cast<const uint2*>(ring + stage * kTileBytes + (kRows * g + i) * 128 + 8 * c);
        w[i][0] = u.x;
        w[i][1] = u.y;
      }
      copies = __syncthreads_and(ok);  // and the stage, and the last tile's words and maxima, have been read
      if (copies) {
        if (threadIdx.x == 0) fetch(t + kRing * gridDim.x, stage);
        if (++stage == kRing) {
          stage = 0;
          phase ^= 1u;
        }
      } else {
        // no copy is started any more, least of all on the barriers whose phases are open
        if (was && threadIdx.x == 0) {
          open_tile = t;
          open_stage = stage;
          open_phase = phase;
        }
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
          const uint2 u = i < rows ? load8_q8(a, row0 + i, col0) : make_uint2(0u, 0u);
          w[i][0] = u.x;
          w[i][1] = u.y;
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < kRows; ++i)
        if (i < rows) load8<S>(a, row0 + i, col0, w[i]);
    }
    if constexpr (S == Src::kQ8) {
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        const float scale = q8_scale(__shfl_sync(0xFFFFFFFFu, xs, (lane & 16) + i));
        const uint32_t lo = w[i][0], hi = w[i][1];
        float v[8];
#pragma unroll
        for (int p = 0; p < 4; ++p)
          q8_unpack2((p < 2 ? lo : hi) >> (16 * (p & 1)), XE5M2, v[2 * p], v[2 * p + 1]);
#pragma unroll
        for (int e = 0; e < 8; ++e) w[i][e] = __float_as_uint(v[e] * scale);
      }
    }
    // elements 2p and 2p + 1 of row i
    auto pair = [&](int i, int p) -> f2_t {
      if constexpr (S == Src::kBf16)
        return bf2_to_f2(w[i][p]);
      else
        return f2(__uint_as_float(w[i][2 * p]), __uint_as_float(w[i][2 * p + 1]));
    };
    // bit pattern of the largest magnitude of row i
    auto row_max = [&](int i) -> uint32_t {
      if constexpr (S == Src::kBf16) {
        uint32_t m = __vmaxu2(__vmaxu2(w[i][0] & 0x7FFF7FFFu, w[i][1] & 0x7FFF7FFFu),
                              __vmaxu2(w[i][2] & 0x7FFF7FFFu, w[i][3] & 0x7FFF7FFFu));
        return max(m & 0xFFFF0000u, m << 16);
      } else {
        float m = 0.f;
#pragma unroll
        for (int e = 0; e < 8; e += 2) m = max3_abs(m, __uint_as_float(w[i][e]), __uint_as_float(w[i][e + 1]));
        return __float_as_uint(m);
      }
    };

    uint32_t bsb = 0;
    if constexpr (BLOCK) {
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < kRows; ++i) m = max(m, row_max(i));
      m = lanes_max<32>(m);
      if (lane == 0) wmax[warp][0] = m;
      __syncthreads();
#pragma unroll
      for (int k = 0; k < kWarps; ++k) m = max(m, wmax[k][0]);
      bsb = q8_scale_byte<E5M2>(m);
      if (threadIdx.x == 0) {
        if (a.q) a.q_scale[tm * a.ldq_scale + tk] = (uint8_t)bsb;
        if (a.qt) a.qt_scale[tk * a.ldqt_scale + tm] = (uint8_t)bsb;
      }
    }
    if (a.q) {
      float inv = q8_inv_scale(bsb);  // without BLOCK that of row held_row(c)
      if constexpr (!BLOCK) {
        uint32_t m[kRows];
#pragma unroll
        for (int i = 0; i < kRows; ++i) m[i] = row_max(i);
        const uint32_t sb = q8_scale_byte<E5M2>(rows_max<kRows>(m, c));
        inv = q8_inv_scale(sb);
        const int r = held_row<kRows>(c);
        if (lane_of<kRows>(r) == c && r < rows) a.q_scale[(int64_t)(row0 + r) * a.ldq_scale + tk] = (uint8_t)sb;
      }
      uint8_t* out = a.q + (int64_t)row0 * a.ldq + col0;
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        const float f = BLOCK ? inv : __shfl_sync(0xFFFFFFFFu, inv, (lane & 16) + lane_of<kRows>(i));
        const f2_t inv2 = f2(f, f);
        float e[8];
#pragma unroll
        for (int p = 0; p < 4; ++p) f2_split(f2_mul(pair(i, p), inv2), e[2 * p], e[2 * p + 1]);
        if (i < rows)
          store8(out, make_uint2(q8_pack4<E5M2>(e[0], e[1], e[2], e[3]), q8_pack4<E5M2>(e[4], e[5], e[6], e[7])),
                 a.K - col0);
        out += a.ldq;
      }
    }
    if (!a.qt) continue;

    if constexpr (!BLOCK) {
      // column maxima: this thread's rows, the warp's other row group, the warps
      if constexpr (S == Src::kBf16) {
#pragma unroll
        for (int p = 0; p < 4; ++p) {
          uint32_t m = w[0][p] & 0x7FFF7FFFu;
#pragma unroll
          for (int i = 1; i < kRows; ++i) m = __vmaxu2(m, w[i][p] & 0x7FFF7FFFu);
          m = __vmaxu2(m, __shfl_xor_sync(0xFFFFFFFFu, m, 16));
          if (lane < 16) {
            wmax[warp][17 * (2 * p) + c] = m << 16;
            wmax[warp][17 * (2 * p + 1) + c] = m & 0xFFFF0000u;
          }
        }
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          float f = 0.f;
#pragma unroll
          for (int i = 0; i < kRows; i += 2) f = max3_abs(f, __uint_as_float(w[i][e]), __uint_as_float(w[i + 1][e]));
          uint32_t m = __float_as_uint(f);
          m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 16));
          if (lane < 16) wmax[warp][17 * e + c] = m;
        }
      }
      __syncthreads();
      if (threadIdx.x < kQ8Group) {
        const int e = threadIdx.x & 7, cc = threadIdx.x >> 3;
        uint32_t m = 0;
#pragma unroll
        for (int k = 0; k < kWarps; ++k) m = max(m, wmax[k][17 * e + cc]);
        const uint32_t sb = q8_scale_byte<E5M2>(m);
        cinv[e >> 1][2 * cc + (e & 1)] = q8_inv_scale(sb);
        const int32_t col = (int32_t)tk * kQ8Group + threadIdx.x;
        if (col < a.K) a.qt_scale[(int64_t)col * a.ldqt_scale + tm] = (uint8_t)sb;
      }
      __syncthreads();
    }
    const float binv = q8_inv_scale(bsb);
    uint32_t* words = reinterpret_cast<uint32_t*>(tile);
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      const float2 ci = BLOCK ? make_float2(binv, binv) : *reinterpret_cast<const float2*>(&cinv[p][2 * c]);
      const f2_t inv2 = f2(ci.x, ci.y);
      float lo[kRows], hi[kRows];
#pragma unroll
      for (int i = 0; i < kRows; ++i) f2_split(f2_mul(pair(i, p), inv2), lo[i], hi[i]);
      // 8-byte word r of column k (rows 8r..) at slot r ^ (k / 8)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float* f = h ? hi : lo;
        const int k = 8 * c + 2 * p + h;
        if constexpr (kRows == 8)
          tile[k * 16 + (g ^ c)] = make_uint2(q8_pack4<E5M2>(f[0], f[1], f[2], f[3]), q8_pack4<E5M2>(f[4], f[5], f[6], f[7]));
        else
          words[(k * 16 + ((g >> 1) ^ c)) * 2 + (g & 1)] = q8_pack4<E5M2>(f[0], f[1], f[2], f[3]);
      }
    }
    __syncthreads();
    // 16 bytes a lane: words 2j and 2j + 1 of column k, swapped where k / 8 is odd
    // (for all of a thread's columns or none: they are 32 or 64 apart)
    const int j = threadIdx.x & 7, k0 = threadIdx.x >> 3;
    const int32_t row = (int32_t)tm * kQ8Group + 16 * j, cols = a.K - ((int32_t)tk * kQ8Group + k0);
    const int32_t inside = a.M - row;  // bytes of the lane's 16 inside the tensor
    uint8_t* out = a.qt + ((int64_t)tk * kQ8Group + k0) * a.ldqt + row;
    const bool swapped = (k0 >> 3) & 1;
#pragma unroll
    for (int k = 0; k < kQ8Group; k += kThreads / 8) {
      uint4 u = reinterpret_cast<const uint4*>(tile)[(k0 + k) * 8 + (j ^ ((k0 + k) >> 4))];
      if (swapped) u = make_uint4(u.z, u.w, u.x, u.y);
      if (k < cols && inside > 0) store16(out, u, inside);
      out += (int64_t)(kThreads / 8) * a.ldqt;
    }
  }
  // None of the copies under way may land when the CTA has left.  (After the
  // loop: this second wait inside it cost the loop 5%.)
  if constexpr (S == Src::kQ8)
    if (!copies && threadIdx.x == 0) {
      uint32_t s = open_stage, p = open_phase;
      for (uint32_t t = open_tile, n = 0; n < kRing && t < (uint32_t)a.tiles; ++n, t += gridDim.x) {
        mbar_wait(&landed[s], p, a.wait_ns);
        if (++s == kRing) {
          s = 0;
          p ^= 1u;
        }
      }
    }
}

template <Src S, bool XE5M2 = false>
cudaError_t launch_src(const QuantArgs& a, bool e5m2, bool block, cudaStream_t st) {
  void (*k)(const QuantArgs, const CUtensorMap) =
      e5m2 ? (block ? sp_quant_q8_kernel<S, true, true, XE5M2> : sp_quant_q8_kernel<S, true, false, XE5M2>)
           : (block ? sp_quant_q8_kernel<S, false, true, XE5M2> : sp_quant_q8_kernel<S, false, false, XE5M2>);
  CUtensorMap map = {};
  int64_t grid = a.tiles;
  size_t smem = 0;
  if constexpr (S == Src::kQ8) {
    cudaError_t e = byte_map(a.x, a.M, a.K, a.ldx, kQ8Group, false, &map);
    int dev = 0, sms = 0;
    if (e == cudaSuccess) e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    smem = 128 + kRing * kTileBytes;  // 128: the alignment of the copies' targets
    if (e == cudaSuccess) e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    if (grid > 2 * sms) grid = 2 * sms;
  }
  return pdl_launch(k, dim3((unsigned)grid), dim3(Shape<S>::kThreads), smem, st, a, map);
}

}  // namespace

cudaError_t launch_quant_q8(const QuantArgs& a, int x_dtype, bool e5m2, bool block, cudaStream_t st) {
  switch (x_dtype) {
    case SP_ELEM_F32: return launch_src<Src::kF32>(a, e5m2, block, st);
    case SP_ELEM_BF16: return launch_src<Src::kBf16>(a, e5m2, block, st);
    case SP_ELEM_E5M2: return launch_src<Src::kQ8, true>(a, e5m2, block, st);
    default: return launch_src<Src::kQ8>(a, e5m2, block, st);
  }
}

}  // namespace spf
