// matmul_q8.cu -- C = A B^T of 8-bit tensors with a power-of-two scale per 128
// values along K, on the 5th-generation tensor cores.
//
//   C[i,j] = sum_k (2^sa[i,k/128] qa[i,k]) (2^sb[j,k/128] qb[j,k])
//
// The tensor core applies the scales itself (kind mxf8f6f4: a ue8m0 byte per
// row and 32 values of K; the four 32-value steps of a 128-value block use
// the same byte) and keeps the whole sum over K in fp32 in tensor memory, so
// nothing is rounded before C's own type.
//
// A CTA (CG = 1) or a pair of CTAs (CG = 2) works on one tile: 128 rows of
// the X operand per CTA against BN rows of the Y operand.  X is A and Y is B,
// or the other way round (SWAP) when A has few rows: then the weights fill
// the tensor core's 128 rows and the tokens its short side.
//   warp 0     producer: one 128-byte wide tile of X and of Y per stage, by
//              tiled bulk copies into a ring of stages (128-byte swizzle)
//   warp 1     issues the tensor core instructions (and owns tensor memory)
//   warps 2-3  bring the scale bytes: per 4 blocks of K one 32-bit word per
//              row, into the 32 x 16 byte layout that goes to tensor memory
//   warps 4-   epilogue: tensor memory to C
// Tiles are dealt to the resident CTAs in turn; the two accumulators in tensor
// memory let the epilogue of one tile run under the products of the next.
// Few tiles (decoding): `ks` CTAs of a cluster split K and add their fp32
// sums through distributed shared memory in rank order, so the result does not
// depend on timing.
//
// Bounds and what was measured (back to back): a large product by the tensor
// core's power (16384 x 4096 x 8192: 316-325 us, 3.4 PFLOP/s; 291 us on zeros) and
// by the 64 KB a pair and block of K that come from L2 (the same loop without
// loads: 259 us); few tokens by the weights' bytes from memory (1 x 32768 x 8192:
// 42 us, 95% of the copy bandwidth; 1 x 8192 x 8192: 14 us, 71%, of which 3.4 us
// start and join); small products by starting, the first copies' latency and the
// last epilogue (4096 x 1536 x 768: 8.7 us).
//
// Every wait is bounded (tma.cuh); a role that gives up reports it in the
// status word, the tiles that were not finished are written as NaN, and tensor
// memory is freed after the instructions and copies in flight are done.
#include <cuda.h>

#include <cmath>

#include "common.cuh"
#include "launch.h"
#include "q8.cuh"
#include "umma.cuh"

namespace spf {

namespace {

// Two epilogue warps per quarter of the lanes where a tile of C is wide; a short
// side has one, and two CTAs of it fit on an SM.
__host__ __device__ constexpr int epilogue_warps(bool swap) { return swap ? 4 : 8; }
__host__ __device__ constexpr int threads(bool swap) { return 128 + 32 * epilogue_warps(swap); }
constexpr int kXRows = 128;                   // rows of X per CTA
constexpr uint32_t kXBytes = kXRows * 128;    // one stage of X
constexpr int kMaxStages = 12;
constexpr int kScaleSlots = 4;                // ring of scale words, 4 blocks of K each
constexpr uint32_t kScaleAtom = 512;          // 128 rows x 4 scale bytes
constexpr uint32_t kStoreBytes = 4096;        // each epilogue warp's 32 x 32 piece of C

struct MatmulPlan {
  int32_t BN;            // rows of Y per tile, a multiple of 16 (32 for CG = 2), at most 256
  int32_t stages;
  int32_t ks;            // CTAs that split K (CG = 1)
  int32_t xtiles, ytiles;
  int32_t width;         // X tiles side by side in the order of the tiles
  int32_t nkb;           // 128-value blocks of K
  uint32_t tmem_cols;    // power of two
  uint32_t acc1;         // column of the second accumulator
  int32_t overlap;       // the accumulators share columns
  uint32_t sf_col;       // first column of the scales
  uint32_t smem;
};

struct Shared {
  uint64_t full[kMaxStages], empty[kMaxStages];
  uint64_t sf_full[kScaleSlots], sf_empty[kScaleSlots];
  uint64_t acc_full[2], acc_free[2], drain;  // of each accumulator
  uint32_t tmem;
};

__host__ __device__ constexpr uint32_t scale_atoms_y(int BN) { return (uint32_t)(BN + 127) / 128; }

// Tile t of the list: `width` tiles of X, along Y, then the next ones, so that
// the tiles in flight share their operands in L2.
// (32-bit: the two 64-bit divisions took 0.7 us a tile of every role's time.)
__device__ __forceinline__ void tile_at(const MatmulPlan& p, uint32_t t, int32_t& tx, int32_t& ty) {
  const uint32_t per = (uint32_t)p.width * (uint32_t)p.ytiles, g = t / per, in = t - g * per;
  const uint32_t width = min((uint32_t)p.width, (uint32_t)p.xtiles - g * (uint32_t)p.width), row = in / width;
  tx = (int32_t)(g * (uint32_t)p.width + (in - row * width));
  ty = (int32_t)row;
}

__device__ __forceinline__ void store_one(const MatmulArgs& a, int64_t o, float v) {
  if (a.c_f32) {
    float* c = static_cast<float*>(a.c) + o;
    *c = v + (a.accumulate ? *c : 0.f);
  } else {
    static_cast<__nv_bfloat16*>(a.c)[o] = __float2bfloat16_rn(v);
  }
}

// C goes out through 4 KB of shared memory per epilogue warp: 32 rows of 128
// bytes (32 fp32 or 64 bf16 columns), the 16-byte pieces of a row exclusive-
// or'ed with the row so that neither side meets a bank conflict, and from there
// in whole 128-byte lines.
__device__ __forceinline__ void stage_piece(unsigned char* buf, int lane, int q, uint4 v) {
  *reinterpret_cast<uint4*>(buf + lane * 128 + ((q ^ (lane & 7)) << 4)) = v;
}

// Rows x.. of the staged piece to columns y.. of C, ny of them inside C.
template <typename T>
__device__ __forceinline__ void store_piece(const MatmulArgs& a, const unsigned char* buf, int64_t x, int64_t XR,
                                            int64_t y, int ny, int lane) {
  constexpr int kPer = 16 / sizeof(T);  // elements in 16 bytes
  T* c = static_cast<T*>(a.c) + x * a.ldc + y;
  const int rows = (int)min((int64_t)32, XR - x);
  if (a.c_vec && ny % kPer == 0) {
    const int q = lane & 7, r0 = lane >> 3;
    if (q * kPer >= ny) return;
    uint4 o[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      o[i] = *reinterpret_cast<const uint4*>(buf + (4 * i + r0) * 128 + ((q ^ ((4 * i + r0) & 7)) << 4));
    T* p = c + r0 * a.ldc + kPer * q;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (4 * i + r0 < rows) {
        if constexpr (sizeof(T) == 4) {
          if (a.accumulate) {
            const float4 b = *reinterpret_cast<const float4*>(p);
            o[i] = make_uint4(__float_as_uint(__uint_as_float(o[i].x) + b.x), __float_as_uint(__uint_as_float(o[i].y) + b.y),
                              __float_as_uint(__uint_as_float(o[i].z) + b.z), __float_as_uint(__uint_as_float(o[i].w) + b.w));
          }
        }
        *reinterpret_cast<uint4*>(p) = o[i];
      }
      p += 4 * a.ldc;
    }
  } else {
    for (int j = lane; j < ny; j += 32) {
#pragma unroll 8
      for (int r = 0; r < 32; ++r) {
        if (r >= rows) continue;
        T o = *reinterpret_cast<const T*>(buf + r * 128 + (((j / kPer) ^ (r & 7)) << 4) + sizeof(T) * (j % kPer));
        T* p = c + r * a.ldc + j;
        if constexpr (sizeof(T) == 4)
          if (a.accumulate) o += *p;
        *p = o;
      }
    }
  }
}

template <int CG, bool SWAP>
__global__ void __launch_bounds__(threads(SWAP), SWAP ? 2 : 1)
    sp_matmul_q8_kernel(const MatmulArgs a, const MatmulPlan p, const __grid_constant__ CUtensorMap mapx,
                        const __grid_constant__ CUtensorMap mapy) {
  extern __shared__ __align__(1024) unsigned char dsm_raw[];
  __shared__ Shared sh;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = CG == 2 || p.ks > 1 ? cluster_rank() : 0;
  const bool leader = CG == 1 || rank == 0;  // of the CTA pair
  const uint32_t base = (smem_addr(dsm_raw) + 1023u) & ~1023u;
  unsigned char* dsm = dsm_raw + (base - smem_addr(dsm_raw));
  const uint32_t ybytes = (uint32_t)(p.BN / CG) * 128u, stage_bytes = kXBytes + ybytes;
  const uint32_t sf_bytes = kScaleAtom * (1 + scale_atoms_y(p.BN));
  const uint32_t sf_base = base + (uint32_t)p.stages * stage_bytes;

  // X is the operand whose rows fill the tensor core's 128 lanes
  const int64_t XR = SWAP ? a.N : a.M, YR = SWAP ? a.M : a.N;
  const uint32_t tiles = (uint32_t)p.xtiles * (uint32_t)p.ytiles;  // below 2^31
  const uint32_t group = CG * p.ks;                                // CTAs per tile
  const uint32_t first = blockIdx.x / group, step = gridDim.x / group;
  const int split = CG == 1 ? (int)rank : 0;
  const int kb0 = (int)((int64_t)p.nkb * split / p.ks), kb1 = (int)((int64_t)p.nkb * (split + 1) / p.ks);

  if (warp == 0 && lane == 0) {
    if (p.nkb > 0) {
      prefetch_tensor_map(&mapx);
      prefetch_tensor_map(&mapy);
    }
    for (int s = 0; s < p.stages; ++s) {
      mbar_init(&sh.full[s], 1);
      mbar_init(&sh.empty[s], 1);
    }
    for (int s = 0; s < kScaleSlots; ++s) {
      mbar_init(&sh.sf_full[s], 2 * CG);
      mbar_init(&sh.sf_empty[s], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.acc_full[i], 1);
      mbar_init(&sh.acc_free[i], epilogue_warps(SWAP) * CG);
    }
    mbar_init(&sh.drain, 1);
    fence_mbar_init();
  }
  // An allocation waits while the SM's columns are taken, and a cluster's CTAs
  // then wait for each other.  That ends: those of two clusters that fit on an SM
  // together (by shared memory) want at most its 512 columns between them.
  if (warp == 1) tmem_alloc<CG>(&sh.tmem, p.tmem_cols);
  tmem_fence_before();
  if (CG == 2 || p.ks > 1)
    cluster_sync();
  else
    __syncthreads();
  tmem_fence_after();
  const uint32_t tmem = sh.tmem;
  grid_dep_wait();
  grid_dep_launch_dependents();

  const uint64_t limit = a.wait_ns;
  if (warp == 0) {
    // ---- producer -------------------------------------------------------------
    if (lane == 0) {
      int s = 0, issued = 0;
      uint32_t ph = 0;
      bool ok = true;
      for (uint32_t t = first; t < tiles && ok; t += step) {
        int32_t tx, ty;
        tile_at(p, t, tx, ty);
        const int32_t x0 = (tx * CG + (CG == 2 ? (int32_t)rank : 0)) * kXRows;
        const int32_t y0 = ty * p.BN + (CG == 2 ? (int32_t)rank * (p.BN / 2) : 0);
        for (int kb = kb0; kb < kb1; ++kb) {
          if (!mbar_wait(&sh.empty[s], ph ^ 1u, limit)) {
            ok = false;
            break;
          }
          if (!(issued == a.drop_stage && blockIdx.x == 0)) {  // test hook: this stage never lands
            const uint32_t st = base + (uint32_t)s * stage_bytes;
            uint32_t bar = smem_addr(&sh.full[s]);
            if (leader) mbar_arrive_expect_tx(&sh.full[s], stage_bytes * CG);
            if (CG == 2) bar = map_cta(bar, 0);
            tma_load_2d<CG>(st, &mapx, kb * 128, x0, bar);
            tma_load_2d<CG>(st + kXBytes, &mapy, kb * 128, y0, bar);
          }
          ++issued;
          if (++s == p.stages) {
            s = 0;
            ph ^= 1u;
          }
        }
      }
      if (!ok) report_status(a.status, kStatusMatmulWaitTimeout);
      // nothing may still be landing in shared memory when the CTA exits; the
      // leader's barriers count the pair's copies
      if (leader)
        for (int j = max(0, issued - p.stages); j < issued; ++j)
          mbar_wait(&sh.full[j % p.stages], (uint32_t)(j / p.stages) & 1u, limit);
    }
  } else if (warp == 1) {
    // ---- tensor core instructions ------------------------------------------------
    if (leader) {
      const uint32_t one = elect_one();
      const uint32_t idesc = idesc_mxf8(SWAP ? a.b_e5m2 : a.a_e5m2, SWAP ? a.a_e5m2 : a.b_e5m2, kXRows * CG, p.BN);
      const uint32_t sfx = tmem + p.sf_col, sfy = sfx + 4;
      // every lane waits, so that the warp stays together and agrees
      auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
        const bool ok = __all_sync(0xFFFFFFFFu, mbar_wait_cluster(bar, parity, limit));
        tmem_fence_after();
        return ok;
      };
      int s = 0, q = 0;
      uint32_t ph = 0, qph = 0;
      uint32_t n = 0;  // tiles of this CTA so far
      bool ok = true;
      for (uint32_t t = first; t < tiles && ok; t += step, ++n) {
        const uint32_t d = tmem + (n & 1u ? p.acc1 : 0u);
        // The accumulators of a wide tile overlap in the columns that the
        // epilogue of the tile before reads first; else this one is free once
        // the tile before that has been read.
        const uint32_t back = p.overlap ? 1u : 2u;
        if (n >= back && !(ok = wait(&sh.acc_free[(n - back) & 1u], ((n - back) >> 1) & 1u))) break;
        // this stage's data and the next scales, tested for while the products
        // before them were issued
        bool landed = false, scales = false;
        for (int kb = kb0; kb < kb1; ++kb) {
          if (kb == kb0 || (kb & 3) == 0) {
            if (!__all_sync(0xFFFFFFFFu, scales) && !(ok = wait(&sh.sf_full[q], qph))) break;
            const uint32_t src = sf_base + (uint32_t)q * sf_bytes;
            tmem_cp_scales<CG>(sfx, desc_rows16(src), one);
            tmem_cp_scales<CG>(sfy, desc_rows16(src + kScaleAtom), one);
            if (p.BN > 128) tmem_cp_scales<CG>(sfy + 4, desc_rows16(src + 2 * kScaleAtom), one);
            umma_commit<CG>(&sh.sf_empty[q], one);
            if (++q == kScaleSlots) {
              q = 0;
              qph ^= 1u;
            }
          }
          if (!__all_sync(0xFFFFFFFFu, landed) &&
              !(ok = __all_sync(0xFFFFFFFFu, mbar_wait(&sh.full[s], ph, limit))))
            break;
          const uint32_t st = base + (uint32_t)s * stage_bytes;
          const uint64_t dx = desc_sw128(st), dy = desc_sw128(st + kXBytes);
          const uint32_t id = idesc_scale_byte(idesc, (uint32_t)kb & 3u);
          uint64_t* const done = &sh.empty[s];
          if (++s == p.stages) {
            s = 0;
            ph ^= 1u;
          }
          landed = mbar_test<false>(&sh.full[s], ph);
          if ((kb & 3) == 3) scales = mbar_test<CG == 2>(&sh.sf_full[q], qph);
          // 32 bytes of K a step (2 in the descriptors' units), the last block only as far as K goes
          const uint32_t add = kb > kb0 ? 1u : 0u;
          const int64_t left = a.K - (int64_t)kb * 128;
          umma_mxf8<CG>(d, dx, dy, id, sfx, sfy, add, one);
          if (left > 32) umma_mxf8<CG>(d, dx + 2, dy + 2, id, sfx, sfy, 1u, one);
          if (left > 64) umma_mxf8<CG>(d, dx + 4, dy + 4, id, sfx, sfy, 1u, one);
          if (left > 96) umma_mxf8<CG>(d, dx + 6, dy + 6, id, sfx, sfy, 1u, one);
          umma_commit<CG>(done, one);
        }
        if (ok) umma_commit<CG>(&sh.acc_full[n & 1u], one);
      }
      if (!ok && lane == 0) report_status(a.status, kStatusMatmulWaitTimeout);
      umma_commit<CG>(&sh.drain, one);
      mbar_wait_cluster(&sh.drain, 0, limit);  // nothing in flight when tensor memory is freed
    }
  } else if (warp < 4) {
    // ---- scales -------------------------------------------------------------------
    const int tid = threadIdx.x - 64;
    const uint8_t* xs = SWAP ? a.b_scale : a.a_scale;
    const uint8_t* ys = SWAP ? a.a_scale : a.b_scale;
    const int64_t xld = SWAP ? a.ldb_scale : a.lda_scale, yld = SWAP ? a.lda_scale : a.ldb_scale;
    const int xshift = (SWAP ? a.b_scale_rows : a.a_scale_rows) == 1 ? 0 : 7;
    const int yshift = (SWAP ? a.a_scale_rows : a.b_scale_rows) == 1 ? 0 : 7;
    int q = 0;
    uint32_t qph = 0;
    bool ok = true;
    for (uint32_t t = first; t < tiles && ok; t += step) {
      int32_t tx, ty;
      tile_at(p, t, tx, ty);
      const int64_t x0 = (int64_t)(tx * CG + (CG == 2 ? (int32_t)rank : 0)) * kXRows, y0 = (int64_t)ty * p.BN;
      uint4 w[6];  // the words of groups 4m .. 4m + 3 of rows tid, tid + 64, ... of X (128), then of Y
      for (int g = kb0 >> 2; g <= (kb1 - 1) >> 2 && kb0 < kb1; ++g) {
        if (g == kb0 >> 2 || (g & 3) == 0) {
#pragma unroll
          for (int i = 0; i < 6; ++i) {
            const int r = tid + 64 * i - (i < 2 ? 0 : kXRows);
            const int64_t row = (i < 2 ? x0 : y0) + r;
            w[i] = make_uint4(0x7F7F7F7Fu, 0x7F7F7F7Fu, 0x7F7F7F7Fu, 0x7F7F7F7Fu);  // rows outside: zeros times one
            if (i < 2 ? row < XR : r < p.BN && row < YR)
              w[i] = ld_cached((i < 2 ? xs + (row >> xshift) * xld : ys + (row >> yshift) * yld) + 16 * (g >> 2));
          }
        }
        if (!mbar_wait_cluster(&sh.sf_empty[q], qph ^ 1u, limit)) {
          ok = false;
          break;
        }
        unsigned char* dst = dsm + (uint32_t)p.stages * stage_bytes + (uint32_t)q * sf_bytes;
#pragma unroll
        for (int i = 0; i < 6; ++i) {
          const int r = tid + 64 * i;  // row r & 127 of atom r >> 7
          if (r < 128 * (1 + (int)scale_atoms_y(p.BN)))
            *reinterpret_cast<uint32_t*>(dst + (r >> 7) * kScaleAtom + (r & 31) * 16 + ((r & 127) >> 5) * 4) =
                (g & 2) ? ((g & 1) ? w[i].w : w[i].z) : ((g & 1) ? w[i].y : w[i].x);
        }
        fence_async_shared();
        __syncwarp();
        if (lane == 0) {
          if (CG == 2)
            mbar_arrive_cluster(map_cta(smem_addr(&sh.sf_full[q]), 0));
          else
            mbar_arrive(&sh.sf_full[q]);
        }
        if (++q == kScaleSlots) {
          q = 0;
          qph ^= 1u;
        }
      }
    }
    if (!ok && tid == 0) report_status(a.status, kStatusMatmulWaitTimeout);
  } else {
    // ---- epilogue -----------------------------------------------------------------
    const int w4 = warp & 3, half = (warp - 4) >> 2, halves = epilogue_warps(SWAP) / 4;
    unsigned char* stage_c = dsm + (uint32_t)p.stages * stage_bytes + kScaleSlots * sf_bytes + (warp - 4) * kStoreBytes;
    // this warp has read the columns of tile n that the next products wait for.
    // (Once per tile, after the tile is complete: no warp can be a phase ahead.)
    auto free_acc = [&](uint32_t n) {
      tmem_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (CG == 2)
          mbar_arrive_cluster(map_cta(smem_addr(&sh.acc_free[n & 1u]), 0));
        else
          mbar_arrive(&sh.acc_free[n & 1u]);
      }
    };
    uint32_t n = 0;
    bool ok = true;
    for (uint32_t t = first; t < tiles; t += step, ++n) {
      int32_t tx, ty;
      tile_at(p, t, tx, ty);
      const int64_t x = (int64_t)(tx * CG + (CG == 2 ? (int32_t)rank : 0)) * kXRows + 32 * w4 + lane, y0 = (int64_t)ty * p.BN;
      const uint32_t acc = tmem + (n & 1u ? p.acc1 : 0u) + ((uint32_t)(32 * w4) << 16);
      if (kb0 < kb1 && ok) ok = __all_sync(0xFFFFFFFFu, mbar_wait_cluster(&sh.acc_full[n & 1u], (n >> 1) & 1u, limit));
      if (!ok && lane == 0 && w4 == 0) report_status(a.status, kStatusMatmulWaitTimeout);
      tmem_fence_after();
      // columns a chunk: 128 bytes of a row of C, the columns that the
      // accumulators may share first
      const int width = SWAP || a.c_f32 ? 32 : 64, chunks = (p.BN + width - 1) / width;
      // The overlap is in the first piece of the first half's warps; without
      // one the whole tile has to be read.
      if (half >= chunks || (p.overlap && half > 0)) free_acc(n);
      for (int c = half; c < chunks; c += halves) {
        const int col0 = width * (n & 1u ? c : chunks - 1 - c);
        if (!SWAP) __syncwarp();  // the staged piece before this one has been read
        const int pieces = (min(width, p.BN - col0) + 31) / 32;
        for (int k = 0; k < pieces; ++k) {
          const int col = col0 + 32 * (n & 1u ? k : pieces - 1 - k);
          uint32_t v[32];
          if (kb0 < kb1 && ok) {
            if (p.BN - col >= 32) {
              tmem_ld32(acc + col, v);
            } else {
              uint32_t u[16];
              tmem_ld16(acc + col, u);
#pragma unroll
              for (int i = 0; i < 16; ++i) v[i] = u[i];
            }
            tmem_ld_wait();
          } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = ok ? 0u : 0x7FC00000u;
          }
          if (p.overlap ? half == 0 && c == 0 && k == 0 : c + halves >= chunks && k == pieces - 1) free_acc(n);
          if constexpr (SWAP) {
            const int ny = (int)min((int64_t)min(32, p.BN - col), YR - (y0 + col));  // columns inside C
            if (p.ks > 1) {
              float* part = reinterpret_cast<float*>(dsm) + col * kXRows + 32 * w4 + lane;
#pragma unroll
              for (int i = 0; i < 32; ++i)
                if (i < ny) part[i * kXRows] = __uint_as_float(v[i]);
            } else if (x < XR) {
              // a lane's columns are rows of C: 32 lanes write neighbouring elements
#pragma unroll
              for (int i = 0; i < 32; ++i)
                if (i < ny) store_one(a, (y0 + col + i) * a.ldc + x, __uint_as_float(v[i]));
            }
          } else if (a.c_f32) {
#pragma unroll
            for (int q = 0; q < 8; ++q)
              stage_piece(stage_c, lane, q, make_uint4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]));
          } else {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              float f[8];
#pragma unroll
              for (int e = 0; e < 8; ++e) f[e] = __uint_as_float(v[8 * q + e]);
              stage_piece(stage_c, lane, q + (col - col0) / 8, Act16<__nv_bfloat16>::pack(f));
            }
          }
        }
        if constexpr (!SWAP) {
          __syncwarp();
          const int ny = (int)min((int64_t)min(width, p.BN - col0), YR - (y0 + col0));
          if (a.c_f32)
            store_piece<float>(a, stage_c, x - lane, XR, y0 + col0, ny, lane);
          else
            store_piece<__nv_bfloat16>(a, stage_c, x - lane, XR, y0 + col0, ny, lane);
        }
      }
    }
    tmem_fence_before();
  }
  __syncwarp();

  // ---- the cluster's sums over K, in rank order ------------------------------------
  if (CG == 2) {
    cluster_sync();
    // The commits arrive at the barriers of both CTAs.  The leader has waited
    // for the last one of its own; the other CTA's may still be on its way (a
    // cluster barrier orders threads, not these), and has to find its barrier.
    if (warp == 1 && !leader) mbar_wait_cluster(&sh.drain, 0, limit);
    __syncwarp();
  } else if (p.ks > 1) {
    cluster_sync();  // one tile per cluster: every CTA's part is in its shared memory
    if constexpr (SWAP) {
      int32_t tx, ty;
      tile_at(p, first, tx, ty);
      const int l = threadIdx.x & 127;
      const int64_t x = (int64_t)tx * kXRows + l;
      const int cols = (int)min((int64_t)p.BN, YR - (int64_t)ty * p.BN);
      for (int col = (int)rank + p.ks * (threadIdx.x >> 7); col < cols; col += threads(SWAP) / 128 * p.ks) {
        float sum = 0.f;
        for (int r = 0; r < p.ks; ++r) sum += ld_cluster_f32(map_cta(base + (uint32_t)(col * kXRows + l) * 4u, r));
        if (x < XR) store_one(a, ((int64_t)ty * p.BN + col) * a.ldc + x, sum);
      }
    }
    cluster_sync();  // nobody's shared memory goes before it is read
  } else {
    __syncthreads();
  }
  if (warp == 1) {
    tmem_fence_after();
    tmem_dealloc<CG>(tmem, p.tmem_cols);
  }
}

// cuTensorMapEncodeTiled of the loaded driver.
using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                 const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

struct Encoder {
  EncodeTiled fn;
  cudaError_t error;
};

Encoder find_encoder() {
  void* f = nullptr;
  cudaDriverEntryPointQueryResult found = cudaDriverEntryPointSymbolNotFound;
  const cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &found);
  if (e != cudaSuccess) return {nullptr, e};
  if (found != cudaDriverEntryPointSuccess || !f) return {nullptr, cudaErrorNotSupported};
  return {reinterpret_cast<EncodeTiled>(f), cudaSuccess};
}

}  // namespace

cudaError_t byte_map(const void* p, int64_t rows, int64_t K, int64_t ld, int box, bool swizzle, CUtensorMap* map) {
  static const Encoder encoder = find_encoder();  // once per process, whichever thread asks first
  if (encoder.error != cudaSuccess) return encoder.error;
  const cuuint64_t dims[2] = {(cuuint64_t)K, (cuuint64_t)rows}, strides[1] = {(cuuint64_t)ld};
  const cuuint32_t boxes[2] = {128, (cuuint32_t)box}, ones[2] = {1, 1};
  const CUresult r = encoder.fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(p), dims, strides, boxes, ones,
                            CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE,
                            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

namespace {

uint32_t pow2_at_least(uint32_t n) {
  uint32_t c = 32;
  while (c < n) c *= 2;
  return c;
}

struct Choice {
  int cg;
  bool swap;
};

// With the operands swapped: a short side leaves room for a second CTA on an SM.
constexpr int kShortSide = 64;
int ctas_per_sm(int BN) { return BN <= kShortSide ? 2 : 1; }

int64_t ceil_div(int64_t n, int64_t d) { return (n + d - 1) / d; }

// Tile shape and split of K: the least of an estimate of the time, in clocks,
// whose constants are measured (back to back on one GB300 at about 2 GHz):
//   a block of K costs a CTA the largest of its products (2 BN clocks for 128
//   x BN x 128), its loads (62 bytes a clock from L2 to an SM, 50 of each SM of
//   a pair) and the issue of its instructions (0.22 us whatever BN is);
//   an epilogue takes 0.6 us per 128 columns of bf16, 0.35 us per 64 of fp32, a
//   sixth more where the tile cuts a piece of a row, five times that where C's
//   rows are not aligned (2305 x 4999 x 129 in 128 columns: 24 us), and 90
//   clocks a column with the operands swapped, whose stores are narrow; it runs
//   under the next tile's products, whose start it holds up where the
//   accumulators overlap;
//   starting and ending a kernel costs 2.6 us, a pair's cluster barriers and the
//   turns of its tiles more (8192 x 8192 x 1024: 55 us in single CTAs of 224
//   columns, 64 us in pairs of 256; 16384 x 4096 x 8192: 349 and 300 us);
//   nothing is faster than its bytes from memory.
Choice choose_plan(const MatmulArgs& a, int sms, int optin, MatmulPlan* best) {
  constexpr double kLoadRate = 62.0, kPairLoadRate = 50.0, kIssue = 430.0, kStart = 5200.0, kSwapColumn = 90.0, kJoin = 1500.0, kMemoryRate = 3300.0;
  constexpr double kRoundF32 = 700.0, kRoundBf16 = 1200.0, kScalar = 5.0, kRagged = 1.15;
  constexpr double kPair = 2000.0, kPairTurn = 3000.0, kTurn = 300.0, kOverlapTurn = 1500.0, kSwapTurn = 5000.0;
  Choice ch = {1, false};
  double least = 1e300;
  const double memory = ((double)(a.M + a.N) * a.K + (double)a.M * a.N * (a.c_f32 ? 4 : 2)) / kMemoryRate;
  const int64_t nkb = ceil_div(a.K, 128);
  const int piece = a.c_f32 ? 32 : 64;  // columns of C in a 128-byte piece of a row
  for (int mode = 0; mode < 3; ++mode) {  // one CTA, a pair of CTAs, one CTA with the operands swapped
    const int cg = mode == 1 ? 2 : 1;
    const bool swap = mode == 2;
    if (cg > sms) continue;
    const int64_t XR = swap ? a.N : a.M, YR = swap ? a.M : a.N;
    for (int BN = 256; BN >= 16; BN -= 16) {
      if (cg == 2 && BN % 32 != 0) continue;
      if (BN - 16 >= YR && BN > 16 * cg) continue;  // a narrower tile holds every row of Y
      const int64_t xt = ceil_div(XR, (int64_t)kXRows * cg), yt = ceil_div(YR, BN);
      for (int ks = 1; ks <= 8; ks *= 2) {
        // of clusters of 2, 4 and 8 CTAs 152, 144 and 120 CTAs are resident at once on 152 SMs
        const int per_sm = swap ? ctas_per_sm(BN) : 1;
        const int64_t room = per_sm * (ks == 8 ? sms * 15 / 19 : ks == 4 ? sms * 18 / 19 : sms);
        if (ks > 1 && (!swap || ks > nkb || xt * yt * ks > room)) break;
        const int64_t ctas = xt * yt * ks * cg;
        const int64_t turns = ceil_div(ctas, per_sm * sms / cg * cg);
        const double load = (kXRows + BN / cg) * 128 / (cg == 2 ? kPairLoadRate : kLoadRate) * (ctas > sms ? per_sm : 1);
        const int64_t rounds = ceil_div(ceil_div(BN, piece), 2);  // pieces of a row that each epilogue warp takes
        const double epilogue = swap ? kSwapColumn * BN : rounds * (a.c_f32 ? kRoundF32 : kRoundBf16) *
                                                              (a.c_vec ? 1.0 : kScalar) * (BN % piece ? kRagged : 1.0);
        const double main = ceil_div(nkb, ks) * fmax(fmax(2.0 * BN, load), kIssue);
        const double path = turns * fmax(main, epilogue) + (cg == 2 ? turns * kPairTurn : swap ? (turns - 1) * kSwapTurn : turns * (BN > 240 ? kOverlapTurn : kTurn));
        const double t = kStart + fmax(path, memory) + 0.1 * path + epilogue + (cg == 2 ? kPair : 0.0) + (ks > 1 ? kJoin : 0.0);
        if (t < least) {
          least = t;
          ch = {cg, swap};
          best->BN = BN;
          best->ks = ks;
          best->xtiles = (int32_t)xt;
          best->ytiles = (int32_t)yt;
        }
      }
    }
  }
  MatmulPlan& p = *best;
  p.nkb = (int32_t)nkb;
  p.width = 16 / ch.cg;
  const uint32_t sf_cols = 16;  // 4 for X and 4 or 8 for Y; every start a multiple of 16
  p.tmem_cols = pow2_at_least((p.ks > 1 ? p.BN : 2 * p.BN) + sf_cols);
  if (p.tmem_cols > 512) p.tmem_cols = 512;
  p.sf_col = p.tmem_cols - sf_cols;
  p.acc1 = p.sf_col - p.BN;
  p.overlap = (int)p.acc1 < p.BN;  // BN 256: by 16 columns (or a split's one accumulator)
  const uint32_t stage = kXBytes + (uint32_t)(p.BN / ch.cg) * 128u;
  const uint32_t rest = 1024 + kScaleSlots * kScaleAtom * (1 + scale_atoms_y(p.BN)) + (ch.swap ? 0 : epilogue_warps(false) * kStoreBytes);
  // 2048: the kernel's static shared memory and the driver's, rounded up
  const int64_t budget = (ch.swap ? optin / ctas_per_sm(p.BN) : optin) - 2048;
  int64_t stages = (budget - rest) / stage;
  if (stages > kMaxStages) stages = kMaxStages;
  const int64_t need = ceil_div(nkb, p.ks) * ceil_div((int64_t)p.xtiles * p.ytiles * p.ks * ch.cg, sms);
  // no more than the CTA ever fills, but room for the join's fp32 sums
  int64_t least_stages = p.ks > 1 ? ceil_div((int64_t)p.BN * kXRows * 4, stage) : 2;
  if (need > least_stages) least_stages = need;
  p.stages = (int32_t)(stages < least_stages ? stages : least_stages);
  p.smem = rest + p.stages * stage;
  return ch;
}

// A CTA (pair, cluster) per tile, or as many as are resident at once.
int64_t grid_of(const MatmulPlan& p, const Choice& ch, int sms) {
  const int64_t tiles = (int64_t)p.xtiles * p.ytiles, resident = (int64_t)(ch.swap ? ctas_per_sm(p.BN) : 1) * sms / ch.cg;
  return (p.ks > 1 || tiles < resident ? tiles : resident) * ch.cg * p.ks;
}

template <int CG, bool SWAP>
cudaError_t launch(const MatmulArgs& a, MatmulPlan p, int sms, cudaStream_t st) {
  CUtensorMap mx = {}, my = {};
  if (p.nkb > 0) {
    const int64_t XR = SWAP ? a.N : a.M, YR = SWAP ? a.M : a.N;
    cudaError_t e = byte_map(SWAP ? a.b : a.a, XR, a.K, SWAP ? a.ldb : a.lda, kXRows, true, &mx);
    if (e == cudaSuccess) e = byte_map(SWAP ? a.a : a.b, YR, a.K, SWAP ? a.lda : a.ldb, p.BN / CG, true, &my);
    if (e != cudaSuccess) return e;
  }
  auto k = sp_matmul_q8_kernel<CG, SWAP>;
  cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)p.smem);
  if (e != cudaSuccess) return e;
  const int group = CG * p.ks;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid_of(p, {CG, SWAP}, sms));
  cfg.blockDim = dim3(threads(SWAP));
  cfg.dynamicSmemBytes = p.smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)group;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = group > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, k, a, p, mx, my);
}

}  // namespace

void describe_matmul_q8(const MatmulArgs& a, int sms, int optin, sp_matmul_q8_plan_t* out) {
  MatmulPlan p = {};
  const Choice ch = choose_plan(a, sms, optin, &p);
  out->pair = ch.cg == 2 ? 1 : 0;
  out->swapped = ch.swap ? 1 : 0;
  out->bn = p.BN;
  out->split_k = p.ks;
  out->stages = p.stages;
  out->block = threads(ch.swap);
  out->tmem_cols = (int32_t)p.tmem_cols;
  out->acc1_col = (int32_t)p.acc1;
  out->scale_col = (int32_t)p.sf_col;
  out->ctas_per_sm = ch.swap ? ctas_per_sm(p.BN) : 1;
  out->stage_bytes = kXBytes + (int64_t)(p.BN / ch.cg) * 128;
  out->smem_bytes = p.smem;
  out->tiles = (int64_t)p.xtiles * p.ytiles;
  out->ctas = grid_of(p, ch, sms);
}

cudaError_t launch_matmul_q8(const MatmulArgs& a, cudaStream_t st) {
  int dev = 0, sms = 0, optin = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&optin, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev);
  if (e != cudaSuccess) return e;

  MatmulPlan p = {};
  const Choice ch = choose_plan(a, sms, optin, &p);
  if (ch.cg == 2) return launch<2, false>(a, p, sms, st);
  return ch.swap ? launch<1, true>(a, p, sms, st) : launch<1, false>(a, p, sms, st);
}

}  // namespace spf
