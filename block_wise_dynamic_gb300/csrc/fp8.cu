// 8-bit floating point with a power-of-two scale for each block of 128:
// quantizers and the matrix product of two quantized operands (sm_103a).
//
// Quantization.  A block (1 x 128, 128 x 1 or 128 x 128 elements) has the
// scale 2^e with the smallest e >= -127 for which no magnitude of the block
// exceeds 448 * 2^e (448 is the largest e4m3 value), and each element the
// e4m3 code nearest to x 2^-e, ties to even.  The scaling is exact, so the
// code takes one rounding.  e + 127 is the scale's byte (E8M0).  A block
// that holds an infinity or a NaN gets the byte 255 (NaN) and NaN codes, so
// that every product with it is NaN.
//
// Scale layout.  The matrix instruction reads scales from tensor memory, 32
// lanes x 4 columns of 32-bit words for 128 rows: row r's word is in lane
// r % 32, column r / 32, and its four bytes belong to four consecutive
// blocks of 128 along the summed axis.  Scales are kept in that order in
// global memory, in tiles of 512 bytes for 128 rows x 4 blocks
// (scale_offset), so a tile is fetched by one bulk copy and moved to tensor
// memory by one copy instruction.
//
// Product.  out[m, n] = sum_k A(m, k) B(n, k) + bias[n].  Each operand is
// stored either row-major (k contiguous) or transposed (m or n contiguous);
// the matrix instruction takes both orders.  Rows and sizes need no
// multiple: the tensor maps fill what lies outside with zeros.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <mutex>

#include "bwd.h"
#include "host_util.h"

namespace {

using bwd::host::aligned16;
using bwd::host::aligned_to;
using bwd::host::check_launch;
using bwd::host::cuda_fail;
using bwd::host::fail;

constexpr int kTile = 128;       // a scale block's length, and a quantizer tile's edge
constexpr int kSfTile = 512;     // bytes of scales for 128 rows x 4 blocks
constexpr int kF32 = BWD_F32, kBF16 = BWD_BF16, kF16 = BWD_F16;

template <int kT>
__host__ __device__ constexpr int elem_bytes() { return kT == kF32 ? 4 : 2; }

// Byte of (row r, block kb) in a scale array whose rows have `groups` groups
// of four blocks.
__device__ __forceinline__ int64_t scale_offset(int64_t r, int64_t kb, int64_t groups) {
  return ((r >> 7) * groups + (kb >> 2)) * kSfTile + (r & 31) * 16 + ((r >> 5) & 3) * 4 + (kb & 3);
}

// --------------------------------------------------------------------------
// quantize

// Scale byte of a block from the bits of its largest magnitude.  448 is
// 1.75 * 2^8, so with a = f * 2^p, 1 <= f < 2, the exponent is p - 8 where
// f <= 1.75 and p - 7 above: adding the distance from 1.75 to 2 in units of
// the last place, less one, carries into the exponent field exactly there.
// A subnormal maximum clamps to e = -127.
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax_bits) {
  if (amax_bits >= 0x7f800000u) return 255u;
  const int b = static_cast<int>((amax_bits + 0x1fffffu) >> 23) - 8;
  return static_cast<uint32_t>(b < 0 ? 0 : b);
}

// 2^-e for a scale byte (finite: bytes of finite maxima are at most 248).
__device__ __forceinline__ float inv_scale(uint32_t byte) { return __uint_as_float((254u - byte) << 23); }

// Four codes, packed.  255 marks a block with non-finite values.
__device__ __forceinline__ uint32_t codes4(const float (&x)[4], const uint32_t (&byte)[4]) {
  float y[4];
#pragma unroll
  for (int j = 0; j < 4; ++j)
    y[j] = byte[j] == 255u ? __uint_as_float(0x7fffffffu) : __fmul_rn(x[j], inv_scale(byte[j]));
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(y[1]), "f"(y[0]));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(y[3]), "f"(y[2]));
  return static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
}

template <int kT>
__device__ __forceinline__ float load1(const void* x, int64_t i) {
  if (kT == kF32) return static_cast<const float*>(x)[i];
  const unsigned short h = static_cast<const unsigned short*>(x)[i];
  if (kT == kBF16) return __uint_as_float(static_cast<uint32_t>(h) << 16);
  return __half2float(__ushort_as_half(h));
}

// Four consecutive elements; the address is aligned to their size.
template <int kT>
__device__ __forceinline__ void load4(const void* x, int64_t i, float (&o)[4]) {
  if (kT == kF32) {
    const float4 a = __ldcs(reinterpret_cast<const float4*>(static_cast<const float*>(x) + i));
    o[0] = a.x; o[1] = a.y; o[2] = a.z; o[3] = a.w;
  } else {
    const uint2 a = __ldcs(reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(x) + i));
    if (kT == kBF16) {
      o[0] = __uint_as_float(a.x << 16); o[1] = __uint_as_float(a.x & 0xffff0000u);
      o[2] = __uint_as_float(a.y << 16); o[3] = __uint_as_float(a.y & 0xffff0000u);
    } else {
      o[0] = __half2float(__ushort_as_half(static_cast<unsigned short>(a.x & 0xffffu)));
      o[1] = __half2float(__ushort_as_half(static_cast<unsigned short>(a.x >> 16)));
      o[2] = __half2float(__ushort_as_half(static_cast<unsigned short>(a.y & 0xffffu)));
      o[3] = __half2float(__ushort_as_half(static_cast<unsigned short>(a.y >> 16)));
    }
  }
}

struct QuantArgs {
  const void* x;
  int64_t rows, cols, ld;  // elements; ld between rows
  int64_t pitch;           // bytes between the rows of either code array
  int64_t groups_r;        // scale groups along a row (blocks 1 x 128)
  int64_t groups_c;        // scale groups along a column (blocks 128 x 1)
  uint8_t* codes_r;        // 1 x 128 blocks, or 128 x 128 ones
  uint8_t* scales_r;
  uint8_t* codes_c;        // 128 x 1 blocks
  uint8_t* scales_c;
  float* col_sums;         // [row tiles][cols] partial column sums, or null
  int vec;                 // rows start on 4-element boundaries
};

// One CTA for a tile of 128 x 128 elements: warp w holds rows w, w + 8, ...,
// lane l the columns 4 l to 4 l + 3, so a warp's load covers a row's 128
// elements.  kMode is a set of BWD_FP8_ROWS, BWD_FP8_COLS, BWD_FP8_TILES.
constexpr int kQThreads = 256, kQWarps = kQThreads / 32, kQRows = kTile / kQWarps;

template <int kT, int kMode>
__global__ void __launch_bounds__(kQThreads)
fp8_quantize_kernel(const QuantArgs a) {
  constexpr bool kRows = kMode & BWD_FP8_ROWS, kCols = kMode & BWD_FP8_COLS, kTiles = kMode & BWD_FP8_TILES;
  __shared__ uint32_t s_col[kQWarps][kTile];
  __shared__ float s_sum[kQWarps][kTile];
  __shared__ uint32_t s_tile[kQWarps];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int64_t r0 = static_cast<int64_t>(blockIdx.y) * kTile, c0 = static_cast<int64_t>(blockIdx.x) * kTile;
  const int64_t c = c0 + 4 * lane;
  float x[kQRows][4];
  const bool vec = a.vec && c + 4 <= a.cols;
#pragma unroll
  for (int i = 0; i < kQRows; ++i) {
    const int64_t r = r0 + warp + kQWarps * i;
    if (vec && r < a.rows) {
      load4<kT>(a.x, r * a.ld + c, x[i]);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) x[i][j] = (r < a.rows && c + j < a.cols) ? load1<kT>(a.x, r * a.ld + c + j) : 0.0f;
    }
  }

  if (kRows) {
#pragma unroll
    for (int i = 0; i < kQRows; ++i) {
      const int64_t r = r0 + warp + kQWarps * i;
      uint32_t top = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) top = max(top, __float_as_uint(x[i][j]) & 0x7fffffffu);
      const uint32_t b = scale_byte(__reduce_max_sync(0xffffffffu, top));
      const uint32_t bytes[4] = {b, b, b, b};
      if (r < a.rows && c < a.pitch) *reinterpret_cast<uint32_t*>(a.codes_r + r * a.pitch + c) = codes4(x[i], bytes);
      if (lane == 0) a.scales_r[scale_offset(r, blockIdx.x, a.groups_r)] = static_cast<uint8_t>(b);
    }
  }
  if (kCols || kTiles) {
    uint32_t top[4] = {0, 0, 0, 0};
    float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < kQRows; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        top[j] = max(top[j], __float_as_uint(x[i][j]) & 0x7fffffffu);
        if (kCols) sum[j] += x[i][j];
      }
    if (kCols) {
#pragma unroll
      for (int j = 0; j < 4; ++j) { s_col[warp][4 * lane + j] = top[j]; s_sum[warp][4 * lane + j] = sum[j]; }
    } else {
      const uint32_t t = __reduce_max_sync(0xffffffffu, max(max(top[0], top[1]), max(top[2], top[3])));
      if (lane == 0) s_tile[warp] = t;
    }
    __syncthreads();
    uint32_t bytes[4];
    if (kCols) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        uint32_t t = 0;
#pragma unroll
        for (int w = 0; w < kQWarps; ++w) t = max(t, s_col[w][4 * lane + j]);
        bytes[j] = scale_byte(t);
      }
      if (warp == 0) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          a.scales_c[scale_offset(c + j, blockIdx.y, a.groups_c)] = static_cast<uint8_t>(bytes[j]);
      }
      if (a.col_sums && threadIdx.x < kTile && c0 + threadIdx.x < a.cols) {
        float s = 0.0f;
#pragma unroll
        for (int w = 0; w < kQWarps; ++w) s += s_sum[w][threadIdx.x];
        a.col_sums[blockIdx.y * a.cols + c0 + threadIdx.x] = s;
      }
    } else {
      uint32_t t = 0;
#pragma unroll
      for (int w = 0; w < kQWarps; ++w) t = max(t, s_tile[w]);
      const uint32_t b = scale_byte(t);
#pragma unroll
      for (int j = 0; j < 4; ++j) bytes[j] = b;
      // the tile's scale, once for each of its rows and once for each of its columns
      if (threadIdx.x < kTile) a.scales_r[scale_offset(r0 + threadIdx.x, blockIdx.x, a.groups_r)] = static_cast<uint8_t>(b);
      else a.scales_c[scale_offset(c0 + threadIdx.x - kTile, blockIdx.y, a.groups_c)] = static_cast<uint8_t>(b);
    }
    uint8_t* const codes = kCols ? a.codes_c : a.codes_r;
#pragma unroll
    for (int i = 0; i < kQRows; ++i) {
      const int64_t r = r0 + warp + kQWarps * i;
      if (r < a.rows && c < a.pitch) *reinterpret_cast<uint32_t*>(codes + r * a.pitch + c) = codes4(x[i], bytes);
    }
  }
}

// Column sums from the quantizer's partial sums, in the order of the rows.
template <int kT>
__device__ __forceinline__ void store1(void* out, int64_t i, float v) {
  if (kT == kF32) static_cast<float*>(out)[i] = v;
  else if (kT == kBF16) static_cast<__nv_bfloat16*>(out)[i] = __float2bfloat16_rn(v);
  else static_cast<__half*>(out)[i] = __float2half_rn(v);
}

template <int kT>
__global__ void __launch_bounds__(256)
col_sums_kernel(const float* __restrict__ partial, int64_t tiles, int64_t cols, void* __restrict__ out) {
  const int64_t c = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  if (c >= cols) return;
  float s = 0.0f;
  for (int64_t t = 0; t < tiles; ++t) s += partial[t * cols + c];
  store1<kT>(out, c, s);
}

// --------------------------------------------------------------------------
// dequantize: code * 2^e, exact in fp32 for e >= -117 and in bf16 above that too

template <int kT>
__global__ void __launch_bounds__(256)
fp8_dequantize_kernel(const uint8_t* __restrict__ codes, int64_t pitch, const uint8_t* __restrict__ scales, int64_t groups,
                      int along_rows, int64_t rows, int64_t cols, void* __restrict__ out) {
  const int64_t n = rows * cols, stride = static_cast<int64_t>(gridDim.x) * blockDim.x;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < n; i += stride) {
    const int64_t r = i / cols, c = i - r * cols;
    const uint32_t b = scales[along_rows ? scale_offset(r, c >> 7, groups) : scale_offset(c, r >> 7, groups)];
    const uint16_t code = codes[r * pitch + c];
    uint32_t h2;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"(code));
    const float v = __half2float(__ushort_as_half(static_cast<unsigned short>(h2 & 0xffffu)));
    const float s = b == 255u ? __uint_as_float(0x7fffffffu) : __uint_as_float(b ? b << 23 : 1u << 22);
    store1<kT>(out, i, __fmul_rn(v, s));
  }
}

// --------------------------------------------------------------------------
// matrix product

__device__ unsigned int g_fp8_fault;  // set when a bounded wait gives up

__device__ __forceinline__ uint32_t smem_u32(const void* p) { return static_cast<uint32_t>(__cvta_generic_to_shared(p)); }

__device__ __forceinline__ void mbar_init(uint64_t* bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(bar)), "r"(count) : "memory");
}
__device__ __forceinline__ void mbar_expect_tx(uint64_t* bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(bar)), "r"(bytes) : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ bool mbar_try(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile("{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}"
               : "=r"(ok) : "r"(smem_u32(bar)), "r"(parity) : "memory");
  return ok != 0;
}

// Every wait is bounded: after about a second (or 2^24 polls) it sets the
// CTA's fail flag and the device's fault word, and from then on every other
// wait of the CTA gives up at once.
__device__ __noinline__ bool mbar_wait_slow(uint64_t* bar, uint32_t parity, volatile int* fail_flag) {
  uint64_t t0, t1;
  asm volatile("mov.u64 %0, %globaltimer;" : "=l"(t0));
  for (int i = 0; i < (1 << 24); ++i) {
    if (mbar_try(bar, parity)) return true;
    if (fail_flag && *fail_flag) return false;
    asm volatile("mov.u64 %0, %globaltimer;" : "=l"(t1));
    if (t1 - t0 > 1000000000ull) break;
  }
  if (fail_flag) *fail_flag = 1;
  atomicOr(&g_fp8_fault, 1u);
  return false;
}
__device__ __forceinline__ bool mbar_wait(uint64_t* bar, uint32_t parity, volatile int* fail_flag) {
  return mbar_try(bar, parity) || mbar_wait_slow(bar, parity, fail_flag);
}

// x is the innermost coordinate: a multiple of 128 bytes everywhere here.
__device__ __forceinline__ void tma_load(void* dst, const CUtensorMap* map, int x, int y, uint64_t* bar) {
  asm volatile("cp.async.bulk.tensor.2d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];"
               ::"r"(smem_u32(dst)), "l"(map), "r"(x), "r"(y), "r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cta.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
               ::"r"(smem_u32(dst)), "l"(src), "r"(bytes), "r"(smem_u32(bar)) : "memory");
}

// Shared-memory matrix descriptor: address, leading and stride byte offsets
// in units of 16 bytes, version 1, swizzle mode (0 none, 2 128-byte).
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr, uint32_t lead, uint32_t stride, uint32_t swizzle) {
  return static_cast<uint64_t>((addr >> 4) & 0x3fffu) | (static_cast<uint64_t>(lead >> 4) << 16) |
         (static_cast<uint64_t>(stride >> 4) << 32) | (1ull << 46) | (static_cast<uint64_t>(swizzle) << 61);
}

constexpr int kBM = 128;          // rows of a tile
constexpr int kBN = 128;          // columns of a tile
constexpr int kBK = 128;          // bytes of the summed axis in one stage: one scale block
constexpr int kStages = 5;
constexpr int kMmThreads = 192;   // warp 0 copies, warp 1 issues products, warps 2 to 5 store
constexpr int kStageBytes = (kBM + kBN) * kBK;
constexpr int kStageSf = 2 * kSfTile;
constexpr int kMmSmem = 1024 + kStages * (kStageBytes + kStageSf);
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kTmemSf = 2 * kBN;  // scales after the two accumulators

// The matrix instruction adds into its fp32 accumulator with truncation, an
// error with a sign that grows with the number of additions (measured
// relative to 64 bits: 1.9e-7 after 1024 products, 7.6e-7 after 4096,
// 2.0e-5 after 65536).  Sums therefore leave the accumulator every
// kChunk blocks and are added up in registers, rounded to nearest.
constexpr int kChunk = 8;

struct MmArgs {
  const uint8_t* sfa;
  const uint8_t* sfb;
  const void* bias;  // [n] or null, of the output's type
  void* out;
  int64_t ldo;
  int m, n, k;
  int a_trans, b_trans;  // operand stored with its own index contiguous
  int tiles_n;
};

template <int kT>
__global__ void __launch_bounds__(kMmThreads, 1)
fp8_matmul_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b, const MmArgs p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* const sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* const sf = sm + kStages * kStageBytes;
  __shared__ __align__(8) uint64_t s_full[kStages], s_empty[kStages], s_acc_full[2], s_acc_empty[2];
  __shared__ uint32_t s_tmem;
  __shared__ int s_fail;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  if (threadIdx.x == 0) {
    s_fail = 0;
    for (int i = 0; i < kStages; ++i) { mbar_init(&s_full[i], 1); mbar_init(&s_empty[i], 1); }
    for (int i = 0; i < 2; ++i) { mbar_init(&s_acc_full[i], 1); mbar_init(&s_acc_empty[i], 4); }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&s_tmem)), "r"(kTmemCols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  const uint32_t tmem = s_tmem;
  const int kblocks = (p.k + kBK - 1) / kBK, groups = (kblocks + 3) / 4;
  const int m0 = static_cast<int>(blockIdx.x) / p.tiles_n * kBM, n0 = static_cast<int>(blockIdx.x) % p.tiles_n * kBN;

  if (warp == 0 && lane == 0) {
    int kb = 0;
    for (; kb < kblocks; ++kb) {
      const int s = kb % kStages;
      if (!mbar_wait(&s_empty[s], ((kb / kStages) & 1) ^ 1, &s_fail)) break;
      const bool scales = (kb & 3) == 0;  // four blocks' scales come with the first of them
      mbar_expect_tx(&s_full[s], kStageBytes + (scales ? kStageSf : 0));
      uint8_t* const a = sm + s * kStageBytes;
      uint8_t* const b = a + kBM * kBK;
      if (p.a_trans) tma_load(a, &map_a, m0, kb * kBK, &s_full[s]); else tma_load(a, &map_a, kb * kBK, m0, &s_full[s]);
      if (p.b_trans) tma_load(b, &map_b, n0, kb * kBK, &s_full[s]); else tma_load(b, &map_b, kb * kBK, n0, &s_full[s]);
      if (scales) {
        bulk_load(sf + s * kStageSf, p.sfa + (static_cast<int64_t>(m0 / 128) * groups + kb / 4) * kSfTile, kSfTile, &s_full[s]);
        bulk_load(sf + s * kStageSf + kSfTile, p.sfb + (static_cast<int64_t>(n0 / 128) * groups + kb / 4) * kSfTile, kSfTile, &s_full[s]);
      }
    }
    // After a failure, let the copies issued so far land (bounded) before the
    // shared memory goes away.
    if (kb < kblocks)
      for (int q = kb > kStages ? kb - kStages : 0; q < kb; ++q) mbar_wait(&s_full[q % kStages], (q / kStages) & 1, nullptr);
  } else if (warp == 1 && lane == 0) {
    // e4m3 x e4m3, E8M0 scales, 128 x 128, fp32 accumulators; bits 15 and 16: transposed operands
    const uint32_t idesc = (static_cast<uint32_t>(p.a_trans) << 15) | (static_cast<uint32_t>(p.b_trans) << 16) |
                           ((kBN / 8) << 17) | (1u << 23) | ((kBM / 16) << 24);
    int chunk = 0;
    bool ok = true;
    for (int k0 = 0; ok && k0 < kblocks; k0 += kChunk, ++chunk) {
      const int buf = chunk & 1;
      ok = mbar_wait(&s_acc_empty[buf], ((chunk >> 1) & 1) ^ 1, &s_fail);
      asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
      for (int kb = k0; ok && kb < kblocks && kb < k0 + kChunk; ++kb) {
        const int s = kb % kStages;
        if (!(ok = mbar_wait(&s_full[s], (kb / kStages) & 1, &s_fail))) break;
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        const uint32_t a = smem_u32(sm + s * kStageBytes), b = a + kBM * kBK;
        const uint32_t tsf = tmem + kTmemSf + 8 * ((kb >> 2) & 1);
        if ((kb & 3) == 0) {
          const uint32_t d = smem_u32(sf + s * kStageSf);
          asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(tsf), "l"(smem_desc(d, 16, 128, 0)) : "memory");
          asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(tsf + 4), "l"(smem_desc(d + kSfTile, 16, 128, 0)) : "memory");
        }
        const uint32_t id = idesc | (static_cast<uint32_t>(kb & 3) << 4) | (static_cast<uint32_t>(kb & 3) << 29);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const uint64_t da = p.a_trans ? smem_desc(a + q * 4096, 16384, 1024, 2) : smem_desc(a + q * 32, 16, 1024, 2);
          const uint64_t db = p.b_trans ? smem_desc(b + q * 4096, 16384, 1024, 2) : smem_desc(b + q * 32, 16, 1024, 2);
          asm volatile("{\n .reg .pred p;\n setp.ne.b32 p, %6, 0;\n"
                       "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n}"
                       ::"r"(tmem + buf * kBN), "l"(da), "l"(db), "r"(id), "r"(tsf), "r"(tsf + 4),
                       "r"(static_cast<uint32_t>(kb != k0 || q != 0)) : "memory");
        }
        asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(&s_empty[s])) : "memory");
      }
      asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(&s_acc_full[buf])) : "memory");
    }
  } else if (warp >= 2) {
    const int quarter = warp & 3;  // the lanes of tensor memory that this warp may read
    const int m = m0 + quarter * 32 + lane;
    float sum[kBN];
#pragma unroll
    for (int j = 0; j < kBN; ++j) sum[j] = 0.0f;
    bool ok = true;
    int chunk = 0;
    for (int k0 = 0; ok && k0 < kblocks; k0 += kChunk, ++chunk) {
      const int buf = chunk & 1;
      ok = mbar_wait(&s_acc_full[buf], (chunk >> 1) & 1, &s_fail);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
#pragma unroll
      for (int c = 0; c < kBN; c += 16) {
        uint32_t r[16];
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
                       "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
                     : "r"(tmem + (static_cast<uint32_t>(quarter * 32) << 16) + buf * kBN + c));
        asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
        for (int u = 0; u < 16; ++u) sum[c + u] = __fadd_rn(sum[c + u], __uint_as_float(r[u]));
      }
      asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
      __syncwarp();
      if (lane == 0) mbar_arrive(&s_acc_empty[buf]);
    }
    if (ok && m < p.m) {
#pragma unroll
      for (int j = 0; j < kBN; ++j)
        if (n0 + j < p.n)
          store1<kT>(p.out, m * p.ldo + n0 + j, p.bias ? __fadd_rn(sum[j], load1<kT>(p.bias, n0 + j)) : sum[j]);
    }
  }
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  if (warp == 1) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols));
}

// --------------------------------------------------------------------------
// host side

using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                              const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

std::once_flag g_encode_once;
EncodeFn g_encode = nullptr;

bwd_status encode_fn(EncodeFn* out) {
  std::call_once(g_encode_once, [] {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      g_encode = reinterpret_cast<EncodeFn>(fn);
  });
  if (!g_encode) return fail(BWD_ERR_CUDA, "the driver does not provide cuTensorMapEncodeTiled");
  *out = g_encode;
  return BWD_OK;
}

// Map of a row-major byte matrix for boxes of 128 bytes x box_rows rows.
bwd_status code_map(CUtensorMap* map, const uint8_t* codes, int64_t rows, int64_t cols, int64_t pitch, int box_rows) {
  EncodeFn encode = nullptr;
  bwd_status s = encode_fn(&encode);
  if (s != BWD_OK) return s;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(pitch)};
  const cuuint32_t box[2] = {128, static_cast<cuuint32_t>(box_rows)}, step[2] = {1, 1};
  const CUresult r = encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(codes), dims, strides, box, step,
                            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(BWD_ERR_CUDA, "cuTensorMapEncodeTiled: error %d", static_cast<int>(r));
  return BWD_OK;
}

constexpr int64_t kMaxDim = int64_t{1} << 30;

bool valid_type(int t) { return t == BWD_F32 || t == BWD_BF16 || t == BWD_F16; }
int64_t tiles_of(int64_t n) { return (n + kTile - 1) / kTile; }
int64_t groups_of(int64_t n) { return (tiles_of(n) + 3) / 4; }

template <int kT>
bwd_status launch_quantize(int mode, const QuantArgs& a, cudaStream_t st) {
  const dim3 grid(static_cast<unsigned>(tiles_of(a.cols)), static_cast<unsigned>(tiles_of(a.rows)));
  if (mode == BWD_FP8_ROWS) fp8_quantize_kernel<kT, BWD_FP8_ROWS><<<grid, kQThreads, 0, st>>>(a);
  else if (mode == BWD_FP8_COLS) fp8_quantize_kernel<kT, BWD_FP8_COLS><<<grid, kQThreads, 0, st>>>(a);
  else if (mode == BWD_FP8_TILES) fp8_quantize_kernel<kT, BWD_FP8_TILES><<<grid, kQThreads, 0, st>>>(a);
  else fp8_quantize_kernel<kT, BWD_FP8_ROWS | BWD_FP8_COLS><<<grid, kQThreads, 0, st>>>(a);
  return check_launch("fp8_quantize_kernel launch");
}

template <int kT>
bwd_status launch_matmul(const CUtensorMap& ma, const CUtensorMap& mb, const MmArgs& p, int tiles, cudaStream_t st) {
  const cudaError_t e = cudaFuncSetAttribute(fp8_matmul_kernel<kT>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMmSmem);
  if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute(MaxDynamicSharedMemorySize)");
  fp8_matmul_kernel<kT><<<tiles, kMmThreads, kMmSmem, st>>>(ma, mb, p);
  return check_launch("fp8_matmul_kernel launch");
}

}  // namespace

namespace bwd {
namespace host {

bwd_status take_fp8_fault(unsigned int* fault) {
  cudaError_t e = cudaMemcpyFromSymbol(fault, g_fp8_fault, sizeof *fault);
  if (e != cudaSuccess) return cuda_fail(e, "cudaMemcpyFromSymbol(fault word)");
  if (*fault == 0) return BWD_OK;
  const unsigned int zero = 0;
  e = cudaMemcpyToSymbol(g_fp8_fault, &zero, sizeof zero);
  return e == cudaSuccess ? BWD_OK : cuda_fail(e, "cudaMemcpyToSymbol(fault word)");
}

}  // namespace host
}  // namespace bwd

extern "C" {

int64_t bwd_fp8_scale_bytes(int64_t count, int64_t length) {
  if (count < 0 || length < 0 || count > kMaxDim || length > kMaxDim) return -1;
  return tiles_of(count) * groups_of(length) * kSfTile;
}

int64_t bwd_fp8_pitch(int64_t cols) { return cols < 0 || cols > kMaxDim ? -1 : (cols + 15) / 16 * 16; }

bwd_status bwd_fp8_quantize(const void* x, bwd_dtype dtype, int64_t rows, int64_t cols, int64_t ld, int32_t blocks,
                            uint8_t* row_codes, uint8_t* row_scales, uint8_t* col_codes, uint8_t* col_scales,
                            void* col_sums, float* col_sums_work, void* stream) {
  if (!valid_type(dtype)) return fail(BWD_ERR_UNSUPPORTED_DTYPE, "dtype %d", (int)dtype);
  if (blocks != BWD_FP8_ROWS && blocks != BWD_FP8_COLS && blocks != BWD_FP8_TILES && blocks != (BWD_FP8_ROWS | BWD_FP8_COLS))
    return fail(BWD_ERR_INVALID_ARG, "bad block set %d", blocks);
  if (rows < 0 || cols < 0 || rows > kMaxDim || cols > kMaxDim) return fail(BWD_ERR_INVALID_ARG, "bad size");
  if (tiles_of(rows) > 65535) return fail(BWD_ERR_INVALID_ARG, "more than 65535 * 128 rows");
  if (ld < cols) return fail(BWD_ERR_INVALID_ARG, "ld is less than cols");
  if (col_sums && !(blocks & BWD_FP8_COLS)) return fail(BWD_ERR_INVALID_ARG, "column sums need blocks along the columns");
  if (cols == 0 || (rows == 0 && !col_sums)) return BWD_OK;
  const int eb = dtype == BWD_F32 ? 4 : 2;
  if (rows > 0) {
    if (!x) return fail(BWD_ERR_INVALID_ARG, "NULL pointer");
    if (!aligned_to(x, eb)) return fail(BWD_ERR_INVALID_ARG, "x is not aligned to its element size");
    const bool r = blocks & (BWD_FP8_ROWS | BWD_FP8_TILES), c = blocks & BWD_FP8_COLS;
    if ((r && (!row_codes || !row_scales)) || (c && !col_codes) || ((c || blocks == BWD_FP8_TILES) && !col_scales))
      return fail(BWD_ERR_INVALID_ARG, "NULL pointer");
    if ((r && !aligned16(row_codes)) || (c && !aligned16(col_codes)))
      return fail(BWD_ERR_INVALID_ARG, "codes must be 16-byte aligned");
  }
  if (col_sums && (!col_sums_work || !aligned_to(col_sums, eb) || !aligned_to(col_sums_work, 4)))
    return fail(BWD_ERR_INVALID_ARG, "column sums need a workspace, both aligned to their element size");
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  bwd_status s = BWD_OK;
  if (rows > 0) {
    QuantArgs a{};
    a.x = x; a.rows = rows; a.cols = cols; a.ld = ld;
    a.pitch = bwd_fp8_pitch(cols);
    a.groups_r = groups_of(cols); a.groups_c = groups_of(rows);
    a.codes_r = row_codes; a.scales_r = row_scales; a.codes_c = col_codes; a.scales_c = col_scales;
    a.col_sums = col_sums ? col_sums_work : nullptr;
    a.vec = ld % 4 == 0 && aligned_to(x, 4 * eb);
    s = dtype == BWD_F32 ? launch_quantize<kF32>(blocks, a, st) : dtype == BWD_BF16 ? launch_quantize<kBF16>(blocks, a, st)
                                                                                   : launch_quantize<kF16>(blocks, a, st);
  }
  if (s == BWD_OK && col_sums) {
    const unsigned grid = static_cast<unsigned>((cols + 255) / 256);
    const int64_t tiles = tiles_of(rows);
    if (dtype == BWD_F32) col_sums_kernel<kF32><<<grid, 256, 0, st>>>(col_sums_work, tiles, cols, col_sums);
    else if (dtype == BWD_BF16) col_sums_kernel<kBF16><<<grid, 256, 0, st>>>(col_sums_work, tiles, cols, col_sums);
    else col_sums_kernel<kF16><<<grid, 256, 0, st>>>(col_sums_work, tiles, cols, col_sums);
    s = check_launch("col_sums_kernel launch");
  }
  return s;
}

bwd_status bwd_fp8_dequantize(const uint8_t* codes, const uint8_t* scales, int32_t along_rows, int64_t rows, int64_t cols,
                              void* out, bwd_dtype dtype, void* stream) {
  if (!valid_type(dtype)) return fail(BWD_ERR_UNSUPPORTED_DTYPE, "dtype %d", (int)dtype);
  if (rows < 0 || cols < 0 || rows > kMaxDim || cols > kMaxDim) return fail(BWD_ERR_INVALID_ARG, "bad size");
  if (rows == 0 || cols == 0) return BWD_OK;
  if (!codes || !scales || !out) return fail(BWD_ERR_INVALID_ARG, "NULL pointer");
  if (!aligned_to(out, dtype == BWD_F32 ? 4 : 2)) return fail(BWD_ERR_INVALID_ARG, "out is not aligned to its element size");
  const int64_t groups = along_rows ? groups_of(cols) : groups_of(rows);
  const int64_t need = (rows * cols + 1023) / 1024;
  const unsigned grid = static_cast<unsigned>(need < 152 * 8 ? need : 152 * 8);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int64_t pitch = bwd_fp8_pitch(cols);
  if (dtype == BWD_F32) fp8_dequantize_kernel<kF32><<<grid, 256, 0, st>>>(codes, pitch, scales, groups, along_rows, rows, cols, out);
  else if (dtype == BWD_BF16) fp8_dequantize_kernel<kBF16><<<grid, 256, 0, st>>>(codes, pitch, scales, groups, along_rows, rows, cols, out);
  else fp8_dequantize_kernel<kF16><<<grid, 256, 0, st>>>(codes, pitch, scales, groups, along_rows, rows, cols, out);
  return check_launch("fp8_dequantize_kernel launch");
}

bwd_status bwd_fp8_matmul(int64_t m, int64_t n, int64_t k, const uint8_t* a, int32_t a_trans, const uint8_t* a_scales,
                          const uint8_t* b, int32_t b_trans, const uint8_t* b_scales, const void* bias, void* out,
                          int64_t ldo, bwd_dtype dtype, void* stream) {
  if (!valid_type(dtype)) return fail(BWD_ERR_UNSUPPORTED_DTYPE, "dtype %d", (int)dtype);
  if (m < 0 || n < 0 || k < 0 || m > kMaxDim || n > kMaxDim || k > kMaxDim) return fail(BWD_ERR_INVALID_ARG, "bad size");
  if (ldo < n) return fail(BWD_ERR_INVALID_ARG, "ldo is less than n");
  if (m == 0 || n == 0) return BWD_OK;
  const int eb = dtype == BWD_F32 ? 4 : 2;
  if (!out || (k > 0 && (!a || !b || !a_scales || !b_scales))) return fail(BWD_ERR_INVALID_ARG, "NULL pointer");
  if (!aligned_to(out, eb) || (bias && !aligned_to(bias, eb))) return fail(BWD_ERR_INVALID_ARG, "out and bias must be aligned to their element size");
  if (k > 0 && (!aligned16(a) || !aligned16(b) || !aligned16(a_scales) || !aligned16(b_scales)))
    return fail(BWD_ERR_INVALID_ARG, "codes and scales must be 16-byte aligned");
  CUtensorMap ma{}, mb{};
  bwd_status s;
  if (k > 0) {
    s = a_trans ? code_map(&ma, a, k, m, bwd_fp8_pitch(m), kBK) : code_map(&ma, a, m, k, bwd_fp8_pitch(k), kBM);
    if (s != BWD_OK) return s;
    s = b_trans ? code_map(&mb, b, k, n, bwd_fp8_pitch(n), kBK) : code_map(&mb, b, n, k, bwd_fp8_pitch(k), kBN);
    if (s != BWD_OK) return s;
  }
  const int64_t tiles_n = tiles_of(n), tiles = tiles_of(m) * tiles_n;
  if (tiles > 0x7fffffff) return fail(BWD_ERR_INVALID_ARG, "too many output tiles");
  MmArgs p{a_scales, b_scales, bias, out, ldo, static_cast<int>(m), static_cast<int>(n), static_cast<int>(k),
           a_trans ? 1 : 0, b_trans ? 1 : 0, static_cast<int>(tiles_n)};
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (dtype == BWD_F32) return launch_matmul<kF32>(ma, mb, p, static_cast<int>(tiles), st);
  if (dtype == BWD_BF16) return launch_matmul<kBF16>(ma, mb, p, static_cast<int>(tiles), st);
  return launch_matmul<kF16>(ma, mb, p, static_cast<int>(tiles), st);
}

}  // extern "C"
