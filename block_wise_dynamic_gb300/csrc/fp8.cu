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
#include <type_traits>

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

__device__ __forceinline__ uint32_t smem_u32(const void* p) { return static_cast<uint32_t>(__cvta_generic_to_shared(p)); }

// Every kernel here is launched so that it may begin before the kernel ahead
// of it in the stream has ended, and waits for that kernel's results before
// it uses any; and it lets the next one begin once it has waited itself, so
// that what came before the kernel ahead has ended too.
__device__ __forceinline__ void wait_for_inputs() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void let_next_begin() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

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

// 2^-e for a scale byte (bytes of finite maxima are at most 248); NaN for a
// block that is not finite, which makes all its codes NaN.
__device__ __forceinline__ float inv_scale(uint32_t byte) {
  return __uint_as_float(byte == 255u ? 0x7fffffffu : (254u - byte) << 23);
}

// Two codes: cvt rounds to nearest even, and no finite value here exceeds 448.
__device__ __forceinline__ uint32_t codes2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

template <int kT>
__device__ __forceinline__ float load1(const void* x, int64_t i) {
  if (kT == kF32) return static_cast<const float*>(x)[i];
  const unsigned short h = static_cast<const unsigned short*>(x)[i];
  if (kT == kBF16) return __uint_as_float(static_cast<uint32_t>(h) << 16);
  return __half2float(__ushort_as_half(h));
}

// The quantizer keeps what it has read as it was stored: words of one fp32
// value or two 16-bit ones.  Magnitudes of any of the types order like their
// bits (infinities and NaN above all numbers), so maxima are integer ones.
template <int kT>
__device__ __forceinline__ uint32_t max_words(uint32_t a, uint32_t b) { return kT == kF32 ? max(a, b) : __vmaxu2(a, b); }
template <int kT>
__device__ __forceinline__ uint32_t magnitude(uint32_t w) { return w & (kT == kF32 ? 0x7fffffffu : 0x7fff7fffu); }

template <int kT>
__device__ __forceinline__ uint32_t max_piece(const uint4& w) {
  return max_words<kT>(max_words<kT>(magnitude<kT>(w.x), magnitude<kT>(w.y)), max_words<kT>(magnitude<kT>(w.z), magnitude<kT>(w.w)));
}

// fp32 bits of a magnitude given by its own type's bits.
template <int kT>
__device__ __forceinline__ uint32_t widen_bits(uint32_t b) {
  if (kT == kF32) return b;
  if (kT == kBF16) return b << 16;
  return __float_as_uint(__half2float(__ushort_as_half(static_cast<unsigned short>(b))));
}

// Value j (0 .. 16 / size - 1) of a 16-byte piece.
template <int kT>
__device__ __forceinline__ float piece(const uint4& w, int j) {
  const uint32_t q = (&w.x)[kT == kF32 ? j : j / 2];
  if (kT == kF32) return __uint_as_float(q);
  if (kT == kBF16) return __uint_as_float(j % 2 ? q & 0xffff0000u : q << 16);
  return __half2float(__ushort_as_half(static_cast<unsigned short>(j % 2 ? q >> 16 : q & 0xffffu)));
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
  int vec;                 // rows start on 16-byte boundaries and hold whole pieces,
  int unit;                // or on boundaries of so many bytes and hold whole units
};

// One CTA for a tile of 128 x 128 elements, which it reads once.  A thread
// owns eight pieces of 16 bytes, one from every eighth part of the tile's
// rows, and keeps them as they were stored: 16-bit ones in shared memory
// (cp.async), fp32 ones, half as many values, in registers.  A warp's load
// covers whole rows.  Both maxima and all codes come from that one copy.
// kMode is a set of BWD_FP8_ROWS, BWD_FP8_COLS, BWD_FP8_TILES.
//
// Bound by DRAM: 8192 x 11008 bf16 takes 41 us for one form (3 bytes a value,
// 6.5 TB/s) and 57 us for both (4 bytes, 6.3 TB/s); with the values widened
// in registers the two forms took 426 us (150 registers, one CTA per SM),
// with the pieces in registers as stored 75 (spills).  Five CTAs of 256
// threads per SM; six ran as fast and spilled with column sums (82 against
// 77 us).  The scales' single bytes are a byte to a sector here and there,
// 1/128 of the codes.
template <int kT> __host__ __device__ constexpr int q_vals() { return 16 / elem_bytes<kT>(); }  // values of a piece
template <int kT> __host__ __device__ constexpr int q_lanes() { return kTile / q_vals<kT>(); }  // lanes to a row
template <int kT> __host__ __device__ constexpr int q_rows() { return 32 / q_lanes<kT>(); }     // rows to a warp's load
constexpr int kQPieces = 8;
template <int kT> __host__ __device__ constexpr int q_warps() { return kTile / kQPieces / q_rows<kT>(); }

template <int kT, int kMode, bool kSums, bool kVec>
__global__ void __launch_bounds__(32 * q_warps<kT>(), kT == kF32 ? 2 : 5)
fp8_quantize_kernel(const QuantArgs a) {
  constexpr bool kRows = kMode & BWD_FP8_ROWS, kCols = kMode & BWD_FP8_COLS, kTiles = kMode & BWD_FP8_TILES;
  constexpr int kVals = q_vals<kT>(), kLanes = q_lanes<kT>(), kPerLoad = q_rows<kT>(), kWarps = q_warps<kT>();
  __shared__ __align__(16) uint4 s_col[kCols ? kWarps : 1][kLanes];
  __shared__ __align__(16) float s_sum[kSums ? kWarps : 1][kTile];
  __shared__ uint32_t s_tile[kWarps];
  __shared__ uint8_t s_byte[kTile];
  wait_for_inputs();
  let_next_begin();
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, part = lane % kLanes;
  const int64_t r0 = static_cast<int64_t>(blockIdx.y) * kTile, c0 = static_cast<int64_t>(blockIdx.x) * kTile;
  const int64_t c = c0 + kVals * part;
  const int row = warp * kPerLoad + lane / kLanes;  // piece i: row + i * kTile / kQPieces
  const int rows_here = a.rows - r0 < kTile ? static_cast<int>(a.rows - r0) : kTile;
  const char* const src0 = static_cast<const char*>(a.x) + ((r0 + row) * a.ld + c) * elem_bytes<kT>();
  const int64_t src_step = a.ld * (kTile / kQPieces) * elem_bytes<kT>();
  const auto fetch = [&](int i) {
    const char* const src = src0 + i * src_step;
    uint4 w = make_uint4(0u, 0u, 0u, 0u);
    const bool in = row + i * (kTile / kQPieces) < rows_here;
    if constexpr (kVec) {
      if (in && c < a.cols) w = *reinterpret_cast<const uint4*>(src);
    } else {
#pragma unroll
      for (int j = 0; j < kVals; ++j)
        if (in && c + j < a.cols) (&w.x)[j] = reinterpret_cast<const uint32_t*>(src)[j];
    }
    return w;
  };
  constexpr bool kStaged = kT != kF32;
  __shared__ __align__(16) uint4 s_x[kStaged ? kQPieces : 1][kStaged ? 32 * kWarps : 1];
  uint4 x[kStaged ? 1 : kQPieces];
  if constexpr (!kStaged) {
#pragma unroll
    for (int i = 0; i < kQPieces; ++i) x[i] = fetch(i);
  } else if constexpr (kVec) {
#pragma unroll
    for (int i = 0; i < kQPieces; ++i) {
      const bool in = row + i * (kTile / kQPieces) < rows_here && c < a.cols;
      // copies nothing and fills with zeros past the edge
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;"
                   ::"r"(smem_u32(&s_x[i][threadIdx.x])), "l"(in ? src0 + i * src_step : src0), "r"(in ? 16u : 0u) : "memory");
    }
  } else {
    // Rows of no 16-byte alignment: as many bytes to a lane as their
    // alignment allows, consecutive lanes along a row.  For both forms, whose
    // two passes keep a CTA long enough, eight bytes asynchronously (6391 x
    // 9012 44.5 us against 49.4); through registers for one form (33.0 so
    // against 31.3) and smaller units (6391 x 1002 10.2 so against 9.5).
    const int bytes_here = static_cast<int>(a.cols - c0 < kTile ? a.cols - c0 : kTile) * 2;
    const auto get_rows = [&](auto unit) {
      using Unit = decltype(unit);
      constexpr int kBytes = sizeof(Unit), kLoads = 2 * kTile / (32 * kBytes);
#pragma unroll
      for (int i = 0; i < kQPieces; ++i)
#pragma unroll
        for (int h = 0; h < kPerLoad; ++h) {
          const int r = warp * kPerLoad + h + i * (kTile / kQPieces), here = r < rows_here ? bytes_here : 0;
          const char* const src = static_cast<const char*>(a.x) + ((r0 + r) * a.ld + c0) * 2;
          char* const dst = reinterpret_cast<char*>(&s_x[i][32 * warp + kLanes * h]);
          if constexpr (kRows && kCols && kBytes == 8) {
#pragma unroll
            for (int q = 0; q < kLoads; ++q) {
              const int at = (32 * q + lane) * kBytes;
              const bool in = at < here;
              asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;"
                           ::"r"(smem_u32(dst + at)), "l"(in ? src + at : static_cast<const char*>(a.x)), "r"(in ? 8 : 0) : "memory");
            }
          } else {
            Unit v[kLoads];
#pragma unroll
            for (int q = 0; q < kLoads; ++q) {
              const int at = (32 * q + lane) * kBytes;
              v[q] = at < here ? __ldcs(reinterpret_cast<const Unit*>(src + at)) : Unit{};
            }
#pragma unroll
            for (int q = 0; q < kLoads; ++q) *reinterpret_cast<Unit*>(dst + (32 * q + lane) * kBytes) = v[q];
          }
        }
    };
    if (a.unit == 8) get_rows(uint2{});
    else if (a.unit == 4) get_rows(uint32_t{});
    else get_rows(uint16_t{});
  }
  if constexpr (kStaged) asm volatile("cp.async.wait_all;" ::: "memory");
  if constexpr (kStaged && !kVec) __syncwarp();  // a warp's rows are its own
  const auto load = [&](int i) {
    if constexpr (kStaged) return s_x[i][threadIdx.x];
    else return x[i];
  };

  // Codes of piece i, zeros past the matrix; the pitch is a multiple of 16, so
  // a piece's codes lie before it or past it.
  const int64_t at = (r0 + row) * a.pitch + c, step = a.pitch * (kTile / kQPieces);
  const bool in_pitch = c < a.pitch;
  const auto put = [&](uint8_t* codes, int i, const uint4& w16, const float (&inv)[kVals]) {
    uint32_t w[kVals / 4];
#pragma unroll
    for (int j = 0; j < kVals; j += 4)
      w[j / 4] = codes2(__fmul_rn(piece<kT>(w16, j), inv[j]), __fmul_rn(piece<kT>(w16, j + 1), inv[j + 1])) |
                 codes2(__fmul_rn(piece<kT>(w16, j + 2), inv[j + 2]), __fmul_rn(piece<kT>(w16, j + 3), inv[j + 3])) << 16;
    if (in_pitch && row + i * (kTile / kQPieces) < rows_here) {
      uint32_t* const dst = reinterpret_cast<uint32_t*>(codes + i * step);
      if constexpr (kVals == 8) *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
      else *dst = w[0];
    }
  };

  if constexpr (kCols) {
    uint4 top = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
    for (int i = 0; i < kQPieces; ++i) {
      const uint4 w = load(i);
      top.x = max_words<kT>(top.x, magnitude<kT>(w.x)); top.y = max_words<kT>(top.y, magnitude<kT>(w.y));
      top.z = max_words<kT>(top.z, magnitude<kT>(w.z)); top.w = max_words<kT>(top.w, magnitude<kT>(w.w));
    }
    if (kPerLoad == 2) {
      top.x = max_words<kT>(top.x, __shfl_xor_sync(0xffffffffu, top.x, 16)); top.y = max_words<kT>(top.y, __shfl_xor_sync(0xffffffffu, top.y, 16));
      top.z = max_words<kT>(top.z, __shfl_xor_sync(0xffffffffu, top.z, 16)); top.w = max_words<kT>(top.w, __shfl_xor_sync(0xffffffffu, top.w, 16));
    }
    if (lane < kLanes) s_col[warp][lane] = top;
  } else if constexpr (kTiles) {
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < kQPieces; ++i) top = max_words<kT>(top, max_piece<kT>(load(i)));
    if (kT != kF32) top = max(top & 0xffffu, top >> 16);
    top = __reduce_max_sync(0xffffffffu, top);
    if (lane == 0) s_tile[warp] = top;
  }
  if constexpr (kRows) {
    // two rows at a time, whose 16-bit maxima share a word; fp32 pieces, in
    // registers anyway, all at once where no other form needs some
    constexpr int kStep = kT == kF32 && !kCols ? kQPieces : 2;
#pragma unroll (kStaged ? 1 : kQPieces / kStep)
    for (int i = 0; i < kQPieces; i += kStep) {
      uint4 w[kStep];
      uint32_t top[kStep];
#pragma unroll
      for (int h = 0; h < kStep; ++h) {
        w[h] = load(i + h);
        top[h] = max_piece<kT>(w[h]);
      }
#pragma unroll
      for (int h = 0; h < kStep; h += 2) {
        if constexpr (kT == kF32) {
          top[h] = __reduce_max_sync(0xffffffffu, top[h]);
          top[h + 1] = __reduce_max_sync(0xffffffffu, top[h + 1]);
        } else {
          uint32_t both = __vmaxu2(__byte_perm(top[h], top[h + 1], 0x5410), __byte_perm(top[h], top[h + 1], 0x7632));
#pragma unroll
          for (int o = kLanes / 2; o > 0; o >>= 1) both = __vmaxu2(both, __shfl_xor_sync(0xffffffffu, both, o));
          top[h] = both & 0xffffu;
          top[h + 1] = both >> 16;
        }
      }
#pragma unroll
      for (int h = 0; h < kStep; ++h) {
        const uint32_t b = scale_byte(widen_bits<kT>(top[h]));
        if (part == 0) s_byte[row + (i + h) * (kTile / kQPieces)] = static_cast<uint8_t>(b);
        float inv[kVals];
#pragma unroll
        for (int j = 0; j < kVals; ++j) inv[j] = inv_scale(b);
        put(a.codes_r + at, i + h, w[h], inv);
      }
    }
  }
  __syncthreads();
  if (kRows && threadIdx.x < kTile)
    a.scales_r[scale_offset(r0 + threadIdx.x, blockIdx.x, a.groups_r)] = s_byte[threadIdx.x];
  if constexpr (kCols) {
    uint4 top = s_col[0][part];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) {
      const uint4 t = s_col[w][part];
      top.x = max_words<kT>(top.x, t.x); top.y = max_words<kT>(top.y, t.y);
      top.z = max_words<kT>(top.z, t.z); top.w = max_words<kT>(top.w, t.w);
    }
    float inv[kVals];
#pragma unroll
    for (int j = 0; j < kVals; ++j) {
      const uint32_t q = (&top.x)[kT == kF32 ? j : j / 2];
      const uint32_t b = scale_byte(widen_bits<kT>(kT == kF32 ? q : j % 2 ? q >> 16 : q & 0xffffu));
      inv[j] = inv_scale(b);
      if (warp == 0 && lane < kLanes) a.scales_c[scale_offset(c + j, blockIdx.y, a.groups_c)] = static_cast<uint8_t>(b);
    }
    float sum[kVals] = {};
#pragma unroll (kStaged ? 2 : kQPieces)
    for (int i = 0; i < kQPieces; ++i) {
      const uint4 w = load(i);
      put(a.codes_c + at, i, w, inv);
      if constexpr (kSums) {
#pragma unroll
        for (int j = 0; j < kVals; ++j) sum[j] += piece<kT>(w, j);
      }
    }
    if constexpr (kSums) {
#pragma unroll
      for (int j = 0; j < kVals; ++j) {
        if (kPerLoad == 2) sum[j] += __shfl_xor_sync(0xffffffffu, sum[j], 16);
        if (lane < kLanes) s_sum[warp][kVals * part + j] = sum[j];
      }
      __syncthreads();
    }
  } else if constexpr (kTiles) {
    uint32_t top = s_tile[0];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) top = max(top, s_tile[w]);
    const uint32_t b = scale_byte(widen_bits<kT>(top));
    // the tile's scale, once for each of its rows and once for each of its columns
    if (threadIdx.x < kTile) a.scales_r[scale_offset(r0 + threadIdx.x, blockIdx.x, a.groups_r)] = static_cast<uint8_t>(b);
    else if (threadIdx.x < 2 * kTile) a.scales_c[scale_offset(c0 + threadIdx.x - kTile, blockIdx.y, a.groups_c)] = static_cast<uint8_t>(b);
    float inv[kVals];
#pragma unroll
    for (int j = 0; j < kVals; ++j) inv[j] = inv_scale(b);
#pragma unroll
    for (int i = 0; i < kQPieces; ++i) put(a.codes_r + at, i, load(i), inv);
  }
  if constexpr (kSums) {
    if (threadIdx.x < kTile && c0 + threadIdx.x < a.cols) {
      float s = 0.0f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) s += s_sum[w][threadIdx.x];
      a.col_sums[blockIdx.y * a.cols + c0 + threadIdx.x] = s;
    }
  }
}

template <int kT>
__device__ __forceinline__ void store1(void* out, int64_t i, float v) {
  if (kT == kF32) static_cast<float*>(out)[i] = v;
  else if (kT == kBF16) static_cast<__nv_bfloat16*>(out)[i] = __float2bfloat16_rn(v);
  else static_cast<__half*>(out)[i] = __float2half_rn(v);
}

// Two values as a packed pair of 16-bit ones, rounded to nearest even.
template <int kT>
__device__ __forceinline__ uint32_t pack16(float lo, float hi) {
  uint32_t r;
  if (kT == kBF16) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  else asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Column sums from the quantizer's partial sums, one for each tile of rows.
struct ColSums {
  const float* partial;  // [tiles][cols]
  int64_t tiles, cols;
  void* out;             // or null: none
};

// As a kernel of its own: eight warps of a CTA each add every eighth of a
// column's partial sums, in order, and the first then adds the eight.
constexpr int kSumWarps = 8;

template <int kT>
__global__ void __launch_bounds__(32 * kSumWarps)
col_sums_kernel(const ColSums a) {
  __shared__ float s_part[kSumWarps][32];
  wait_for_inputs();
  let_next_begin();
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int64_t c = static_cast<int64_t>(blockIdx.x) * 32 + lane;
  float s = 0.0f;
  if (c < a.cols) {
#pragma unroll 8
    for (int64_t t = warp; t < a.tiles; t += kSumWarps) s += a.partial[t * a.cols + c];
  }
  s_part[warp][lane] = s;
  __syncthreads();
  if (warp != 0 || c >= a.cols) return;
#pragma unroll
  for (int w = 1; w < kSumWarps; ++w) s += s_part[w][lane];
  store1<kT>(a.out, c, s);
}

// Beside a product: every `step`-th group of 32 columns to a warp, in the same
// order of additions.
template <int kT>
__device__ __forceinline__ void col_sums_of_warp(const ColSums& a, int64_t first, int64_t step) {
  for (int64_t c = 32 * first + threadIdx.x % 32; c < a.cols; c += 32 * step) {
    float s[kSumWarps] = {};
    for (int64_t t = 0; t < a.tiles; t += kSumWarps)
#pragma unroll
      for (int w = 0; w < kSumWarps; ++w)
        if (t + w < a.tiles) s[w] += a.partial[(t + w) * a.cols + c];
#pragma unroll
    for (int w = 1; w < kSumWarps; ++w) s[0] += s[w];
    store1<kT>(a.out, c, s[0]);
  }
}

// --------------------------------------------------------------------------
// dequantize: code * 2^e, one product, rounded once to the output's type.  For
// looking at codes; no product goes through it.

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

__device__ __forceinline__ void mbar_init(uint64_t* bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(bar)), "r"(count) : "memory");
}
__device__ __forceinline__ void mbar_expect_tx(uint64_t* bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(bar)), "r"(bytes) : "memory");
}
__device__ __forceinline__ bool mbar_try(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile("{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}"
               : "=r"(ok) : "r"(smem_u32(bar)), "r"(parity) : "memory");
  return ok != 0;
}

__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}
// Arrival on the same barrier of the pair's first CTA.
__device__ __forceinline__ void mbar_arrive_leader(uint64_t* bar) {
  asm volatile("{\n .reg .b32 r;\n mapa.shared::cluster.u32 r, %0, 0;\n mbarrier.arrive.shared::cluster.b64 _, [r];\n}"
               ::"r"(smem_u32(bar)) : "memory");
}

// Every wait is bounded: after about a second (or 2^24 polls) it sets the
// CTA's fail flag and the device's fault word, and from then on every other
// wait of the CTA gives up at once.
// (The timer is read after 64 polls for the first time: reading it takes
// longer than a stage's products.)
__device__ __noinline__ bool mbar_wait_slow(uint64_t* bar, uint32_t parity, volatile int* fail_flag) {
  uint64_t t0 = 0, t1;
  for (int i = 1; i < (1 << 24); ++i) {
    if (mbar_try(bar, parity)) return true;
    if (fail_flag && *fail_flag) return false;
    if (i % 64 != 0) continue;
    asm volatile("mov.u64 %0, %globaltimer;" : "=l"(t1));
    if (t0 == 0) t0 = t1;
    if (t1 - t0 > 1000000000ull) break;
  }
  if (fail_flag) *fail_flag = 1;
  atomicOr(&g_fp8_fault, 1u);
  return false;
}
__device__ __forceinline__ bool mbar_wait(uint64_t* bar, uint32_t parity, volatile int* fail_flag) {
  return mbar_try(bar, parity) || mbar_wait_slow(bar, parity, fail_flag);
}

// After a failed wait, copies and products may still be under way: leaves
// them two milliseconds before the memory they use goes away.
__device__ __noinline__ void let_copies_land() {
  uint64_t t0, t1;
  asm volatile("mov.u64 %0, %globaltimer;" : "=l"(t0));
  for (int i = 0; i < (1 << 20); ++i) {
    asm volatile("mov.u64 %0, %globaltimer;" : "=l"(t1));
    if (t1 - t0 > 2000000ull) break;
  }
}

// One lane of a converged warp.  The copying and issuing warps run their loops
// with all lanes and elect the one that issues, so that the compiler keeps
// addresses and descriptors in uniform registers (with a loop of one lane,
// 0.36 us per stage of a 256 x 128 tile against 0.18).
__device__ __forceinline__ bool elect_one() {
  uint32_t ok;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(ok));
  return ok != 0;
}

// A stage of a ring of kStages barriers and the parity of its phase.
template <int kStages>
struct Ring {
  int s = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void next() {
    if (++s == kStages) { s = 0; phase ^= 1u; }
  }
};

// Address of a barrier of this CTA in the shared memory of the pair's first
// CTA, which issues the products for both.
__device__ __forceinline__ uint32_t leader_addr(const uint64_t* bar) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(smem_u32(bar)));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Tensor copy into this CTA's shared memory that completes on a barrier of
// the pair's first CTA.  x is the innermost coordinate: a multiple of 64
// bytes everywhere here.
__device__ __forceinline__ void tma_load(void* dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
  asm volatile("cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];"
               ::"r"(smem_u32(dst)), "l"(map), "r"(x), "r"(y), "r"(bar) : "memory");
}
__device__ __forceinline__ void prefetch_map(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}
__device__ __forceinline__ void tma_store(const CUtensorMap* map, int x, int y, const void* src) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];"
               ::"l"(map), "r"(x), "r"(y), "r"(smem_u32(src)) : "memory");
}

// Shared-memory matrix descriptor: address, leading and stride byte offsets
// in units of 16 bytes, version 1, swizzle mode (0 none, 2 128-byte, 4
// 64-byte).
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr, uint32_t lead, uint32_t stride, uint32_t swizzle) {
  return static_cast<uint64_t>((addr >> 4) & 0x3fffu) | (static_cast<uint64_t>(lead >> 4) << 16) |
         (static_cast<uint64_t>(stride >> 4) << 32) | (1ull << 46) | (static_cast<uint64_t>(swizzle) << 61);
}

// Arrival on a barrier of both CTAs when the pair's products and scale
// copies issued so far have finished.
__device__ __forceinline__ void commit_pair(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;"
               ::"r"(smem_u32(bar)), "h"(static_cast<uint16_t>(3)) : "memory");
}

// 32 columns of this warp's 32 lanes.
__device__ __forceinline__ void tmem_load32(uint32_t addr, uint32_t (&r)[32]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 "
               "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
               "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
                 "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
                 "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
                 "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
               : "r"(addr));
}

// A pair of CTAs (a cluster of two, one per SM) works on a tile of 256 rows
// and kBN columns: each holds its 128 rows of A and its half of B's lines,
// the first CTA issues products that read both halves (cta_group::2) and
// each CTA's tensor memory holds its own rows' sums.  Against one CTA with
// 128 x 128 this halves the operand bytes that an SM reads per product.
// Pairs are persistent and walk the tiles with a grid stride; warp 0 copies,
// warp 1 issues, the other kWarps store the tile before (each a quarter of its
// rows; four warps all of its columns, eight half of them), all meeting at
// mbarriers only.  Eight are faster where a tile is stored in less time than
// the next one takes (8192 x 128 x 9728 28 us against 35); four draw less
// power where it is not (16384 x 4096 x 11008 474 us against 484 with the
// quantizer), and have a sixth stage in the other four's staging.
//
// Bound by the matrix instruction at the clock that its power leaves: 16384 x
// 4096 x 11008 takes 330 us with the copies left out (0.28 us for a stage of
// 512 cycles, the instruction's rate at 1.86 GHz), 351 on zeros, and 395 to
// 410 (3.6 to 3.7 PFLOP/s, 1.9 times the bf16 library product) on random
// values, with the clock at 1.6 GHz.  Five stages run as fast as six, four 7%
// slower.  Order of the tiles and cache hints for loads and stores changed
// it by 1% at most.
constexpr int kBM = 256;
constexpr int kBK = 128;          // bytes of the summed axis in one stage: one scale block
__host__ __device__ constexpr int mm_threads(int store_warps) { return 64 + 32 * store_warps; }
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kTmemSf = 480; // scales after the accumulators: two sets of 4 + 8 columns
constexpr int kStoreBytes = 4096; // staging of one storing warp: 32 rows of 128 bytes

// The matrix instruction adds into its fp32 accumulator with truncation, an
// error with a sign that grows with the number of additions (measured
// relative to 64 bits: 1.9e-7 after 1024 products, 7.6e-7 after 4096,
// 2.0e-5 after 65536).  That is far below a 16-bit output's rounding.  For
// fp32 outputs (kSum) the sums leave the accumulator every kChunk blocks,
// 2,048 products, and are added up in registers, rounded to nearest.  Each
// time the next products wait for the columns that the accumulators share:
// 8192 x 4096 x 11008 takes 264 us with eight blocks, 257 with sixteen and
// 254 without (with 128 columns, whose accumulators share none but which
// read more bytes per product, 306, 296 and 295).
constexpr int kChunk = 16;

template <int kBN, int kWarps> __host__ __device__ constexpr int mm_stages() { return kBN == 128 ? 7 : kWarps == 4 ? 6 : 5; }
template <int kBN> __host__ __device__ constexpr int mm_a_bytes() { return kBM / 2 * kBK; }
template <int kBN> __host__ __device__ constexpr int mm_b_bytes() { return kBN / 2 * kBK; }
template <int kBN> __host__ __device__ constexpr int mm_sf_bytes() { return kSfTile + kBN / 128 * kSfTile; }
template <int kBN, int kWarps> __host__ __device__ constexpr int mm_smem() {
  return 1024 + mm_stages<kBN, kWarps>() * (mm_a_bytes<kBN>() + mm_b_bytes<kBN>() + mm_sf_bytes<kBN>()) + kWarps * kStoreBytes;
}

struct MmArgs {
  const void* bias;  // [n] or null, of the output's type
  void* out;
  int64_t ldo;
  int m, n, k;
  int a_trans, b_trans;  // operand stored with its own index contiguous
  int tiles_m, tiles_n;
  int whole;             // the first tiles; the rest are worked on as two halves of 128 columns each
  int sf_rows_b;         // row tiles of B's scales
  int store;             // columns that tensor stores take: all, whole groups only, or none;
  int unit;              // the others go in stores of so many bytes
};

struct MmMaps {
  CUtensorMap a, b, sfa, sfb, out;
};

// One product, or two of one call in one launch: the pairs go on from the
// first one's tiles to the second one's, with no kernel's end and start
// between them.
template <int kCount>
struct MmCall {
  MmMaps maps[kCount];
  MmArgs p[kCount];
  int items[2];   // of the first, of both
  ColSums sums;   // column sums to finish beside the products
};

// What a pair works on: a tile, or half of one (its columns from n0 on).  A
// last wave that less than half fills the device is cut into halves, which
// take half as long.
struct Item {
  int m0, n0, cols, call;
};
template <int kBN, bool kTwo>
__device__ __forceinline__ Item item_of(const MmCall<kTwo ? 2 : 1>& c, int i) {
  const int call = kTwo && i >= c.items[0] ? 1 : 0;
  if (call) i -= c.items[0];
  const MmArgs& p = c.p[call];
  if (kBN == 128 || i < p.whole) return Item{i / p.tiles_n * kBM, i % p.tiles_n * kBN, kBN, call};
  const int t = p.whole + (i - p.whole) / 2;
  return Item{t / p.tiles_n * kBM, t % p.tiles_n * kBN + (i - p.whole) % 2 * 128, 128, call};
}

// The two accumulators.  With 256 columns each they overlap by 32 columns,
// which leaves room for the scales: the storing warps read the shared
// columns first and the next tile's products start when they have.
template <int kBN> __device__ __forceinline__ uint32_t acc_col(int buf) { return buf ? (kBN == 256 ? 224u : 128u) : 0u; }

// kTwo: the call may have two products.  (Its arguments are then read through
// an index: 4096 x 7 x 4096 13.5 us with it, 11.8 without.)
template <int kT, int kBN, bool kSum, int kWarps, bool kTwo>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(mm_threads(kWarps), 1)
fp8_matmul_kernel(const __grid_constant__ MmCall<kTwo ? 2 : 1> c) {
  static_assert(kWarps == 8 || (kWarps == 4 && !kSum), "a thread's registers hold the sums of 128 columns at most");
  constexpr int kStages = mm_stages<kBN, kWarps>(), kA = mm_a_bytes<kBN>(), kB = mm_b_bytes<kBN>(), kSf = mm_sf_bytes<kBN>();
  extern __shared__ uint8_t smem_raw[];
  uint8_t* const sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* const store = sm + kStages * (kA + kB);
  uint8_t* const sf = store + kWarps * kStoreBytes;
  __shared__ __align__(8) uint64_t s_full[kStages], s_empty[kStages], s_acc_full[2], s_acc_empty[2], s_overlap;
  __shared__ __align__(16) float s_bias[kWarps][64];
  __shared__ uint32_t s_tmem;
  __shared__ int s_fail;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  uint32_t rank;
  asm("mov.u32 %0, %cluster_ctarank;" : "=r"(rank));
  if (threadIdx.x == 0) {
    prefetch_map(&c.maps[0].a);
    prefetch_map(&c.maps[0].b);
    prefetch_map(&c.maps[0].sfa);
    prefetch_map(&c.maps[0].sfb);
    s_fail = 0;
    for (int i = 0; i < kStages; ++i) { mbar_init(&s_full[i], 1); mbar_init(&s_empty[i], 1); }
    for (int i = 0; i < 2; ++i) { mbar_init(&s_acc_full[i], 1); mbar_init(&s_acc_empty[i], 2 * kWarps); }
    mbar_init(&s_overlap, 8);  // four warps of either CTA read the shared columns
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&s_tmem)), "r"(kTmemCols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
  }
  __syncwarp();
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  cluster_sync();
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  const uint32_t tmem = s_tmem;
  // one product's arguments stay where the launch left them
  using Args = std::conditional_t<kTwo, const MmArgs&, const MmArgs>;
  const int items = c.items[1], pairs = static_cast<int>(gridDim.x) / 2;
  // two products' tiles forth and back: whoever has one of the longer sums
  // first has none of the wave behind that is not full (2048 x 1024 x 1024's
  // backward pass 18.0 us against 21.5)
  const int first = static_cast<int>(blockIdx.x) / 2, turn = 2 * (pairs - first) - 1;

  if (warp == 0) {
    wait_for_inputs();
    let_next_begin();
    const bool one = elect_one();
    Ring<kStages> ring;
    bool ok = true;
    for (int t = first, step = turn; ok && t < items; t += kTwo ? step : pairs, step = 2 * pairs - step) {
      const Item item = item_of<kBN, kTwo>(c, t);
      const Args p = c.p[kTwo ? item.call : 0];
      const MmMaps& maps = c.maps[kTwo ? item.call : 0];
      const int kblocks = (p.k + kBK - 1) / kBK, groups = (kblocks + 3) / 4;
      // of a half, the copies of B bring as many lines as of a whole
      const int m0 = item.m0 + static_cast<int>(rank) * (kBM / 2), nt = item.n0, n0 = nt + static_cast<int>(rank) * (item.cols / 2);
      for (int kb = 0; kb < kblocks; ++kb, ring.next()) {
        if (!(ok = mbar_wait(&s_empty[ring.s], ring.phase ^ 1u, &s_fail))) break;
        if (one) {
          const bool scales = (kb & 3) == 0;  // four blocks' scales come with the first of them
          const uint32_t bar = leader_addr(&s_full[ring.s]);
          if (rank == 0) mbar_expect_tx(&s_full[ring.s], 2 * (kA + kB + (scales ? kSf : 0)));
          uint8_t* const a = sm + ring.s * (kA + kB);
          uint8_t* const b = a + kA;
          tma_load(a, &maps.a, p.a_trans ? m0 : kb * kBK, p.a_trans ? kb * kBK : m0, bar);
          tma_load(b, &maps.b, p.b_trans ? n0 : kb * kBK, p.b_trans ? kb * kBK : n0, bar);
          if (scales) {
            // A's for this CTA's rows, B's for the whole tile
            tma_load(sf + ring.s * kSf, &maps.sfa, 0, m0 / 128 * groups + kb / 4, bar);
#pragma unroll
            for (int h = 0; h < kBN / 128; ++h) {
              const int rt = nt / 128 + h;  // past the last row tile: columns past n, whatever they hold
              tma_load(sf + ring.s * kSf + (1 + h) * kSfTile, &maps.sfb, 0, (rt < p.sf_rows_b ? rt : p.sf_rows_b - 1) * groups + kb / 4, bar);
            }
          }
        }
        __syncwarp();
      }
    }
  } else if (warp == 1) {
    if (rank != 0) {
      // the issuing warp of the second CTA has nothing to issue
      if (c.sums.out) {
        wait_for_inputs();
        col_sums_of_warp<kT>(c.sums, first, pairs);
      }
    } else {
      const bool one = elect_one();
      // descriptors of stage 0, and the step of 32 along the summed axis
      const uint64_t da0 = smem_desc(smem_u32(sm), 16, 1024, 2), dsf0 = smem_desc(smem_u32(sf), 16, 128, 0);
      Ring<kStages> ring;
      int use = 0;  // accumulators used so far
      bool ok = true;
      for (int t = first, step = turn; ok && t < items; t += kTwo ? step : pairs, step = 2 * pairs - step) {
        const Item item = item_of<kBN, kTwo>(c, t);
        const Args p = c.p[kTwo ? item.call : 0];
        const int kblocks = (p.k + kBK - 1) / kBK, chunk = kSum ? kChunk : kblocks;
        const int a_trans = p.a_trans, b_trans = p.b_trans;
        // e4m3 x e4m3, E8M0 scales, fp32 accumulators; bits 15 and 16: transposed operands
        const uint32_t idesc = (static_cast<uint32_t>(a_trans) << 15) | (static_cast<uint32_t>(b_trans) << 16) |
                               (static_cast<uint32_t>(item.cols / 8) << 17) | (1u << 23) | ((kBM / 16) << 24);
        const uint64_t db0 = b_trans && kBN == 128 ? smem_desc(smem_u32(sm + kA), 16, 512, 4) : smem_desc(smem_u32(sm + kA), 16, 1024, 2);
        const uint32_t sa = a_trans ? 4096 / 16 : 32 / 16, sb = b_trans ? kBN / 2 * 32 / 16 : 32 / 16;
        for (int k0 = 0; ok && k0 < kblocks; k0 += chunk, ++use) {
          const int buf = use & 1;
          ok = mbar_wait(&s_acc_empty[buf], ((use >> 1) & 1) ^ 1, &s_fail);
          if (kBN == 256 && ok && use > 0) ok = mbar_wait(&s_overlap, (use - 1) & 1, &s_fail);
          asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
          const int k1 = kblocks < k0 + chunk ? kblocks : k0 + chunk;
          const uint32_t acc = tmem + acc_col<kBN>(buf);
          for (int kb = k0; ok && kb < k1; ++kb, ring.next()) {
            if (!(ok = mbar_wait(&s_full[ring.s], ring.phase, &s_fail))) break;
            asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
            if (one) {
              const uint64_t da = da0 + static_cast<uint32_t>(ring.s * ((kA + kB) / 16)), db = db0 + static_cast<uint32_t>(ring.s * ((kA + kB) / 16));
              const uint32_t tsf = tmem + kTmemSf + 16 * ((kb >> 2) & 1);
              if ((kb & 3) == 0) {
#pragma unroll
                for (int h = 0; h < 1 + kBN / 128; ++h)
                  asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(tsf + 4 * h),
                               "l"(dsf0 + static_cast<uint32_t>(ring.s * (kSf / 16) + h * (kSfTile / 16))) : "memory");
              }
              // which of the four bytes: bits 4 and 29
              const uint32_t id = idesc + static_cast<uint32_t>(kb & 3) * ((1u << 4) | (1u << 29));
#pragma unroll
              for (uint32_t q = 0; q < 4; ++q)
                asm volatile("{\n .reg .pred p;\n setp.ne.b32 p, %6, 0;\n"
                             "tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n}"
                             ::"r"(acc), "l"(da + q * sa), "l"(db + q * sb), "r"(id), "r"(tsf), "r"(tsf + 4),
                             "r"(static_cast<uint32_t>(kb != k0 || q != 0)) : "memory");
              commit_pair(&s_empty[ring.s]);
            }
            __syncwarp();
          }
          if (one) commit_pair(&s_acc_full[buf]);
          __syncwarp();
        }
      }
    }
  } else {
    const int quarter = warp & 3;      // the lanes of tensor memory that this warp may read
    const int half = (warp - 2) / 4;   // with eight warps, which half of the columns is its own
    constexpr int kHalf = kWarps == 8 ? kBN / 2 : kBN;  // columns of one warp
    const uint32_t own = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + half * kHalf;
    uint8_t* const stage = store + (warp - 2) * kStoreBytes;
    float* const bias_s = s_bias[warp - 2];
    constexpr int kCols = kT == kF32 ? 32 : 64;  // columns of one staged group: 128 bytes
    constexpr int kGroups = kHalf / kCols;
    int use = 0;
    bool ok = true;
    // Done with the accumulators' shared columns, or with all of its own: the
    // first accumulator's last columns and the second one's first are shared.
    const auto done_shared = [&](int buf) {
      if (kBN != 256 || (kWarps == 8 && buf == half)) return;
      asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
      __syncwarp();
      if (lane == 0) mbar_arrive_leader(&s_overlap);
    };
    const auto done_all = [&](int buf) {
      asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
      __syncwarp();
      if (lane == 0) mbar_arrive_leader(&s_acc_empty[buf]);
    };
    for (int t = first, step = turn; ok && t < items; t += kTwo ? step : pairs, step = 2 * pairs - step) {
      const Item item = item_of<kBN, kTwo>(c, t);
      const Args p = c.p[kTwo ? item.call : 0];
      const int m0 = item.m0 + static_cast<int>(rank) * (kBM / 2) + quarter * 32, n0 = item.n0 + half * kHalf;
      const int cols = item.cols - half * kHalf;  // of a half tile, some columns are not there
      float sum[kSum ? kHalf : 1];
      if constexpr (kSum) {
#pragma unroll
        for (int j = 0; j < kHalf; ++j) sum[j] = 0.0f;
        for (int k0 = 0; ok && k0 < p.k; k0 += kChunk * kBK, ++use) {
          const int buf = use & 1;
          ok = __all_sync(0xffffffffu, mbar_wait(&s_acc_full[buf], (use >> 1) & 1, &s_fail));
          if (!ok) break;
          asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
          const auto add = [&](auto at) {
            constexpr int c = decltype(at)::value;
            uint32_t r[32];
            tmem_load32(own + acc_col<kBN>(buf) + c, r);
            asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
            for (int u = 0; u < 32; ++u) sum[c + u] = __fadd_rn(sum[c + u], __uint_as_float(r[u]));
          };
          using C0 = std::integral_constant<int, 0>;
          using C1 = std::integral_constant<int, 32 % kHalf>;
          using C2 = std::integral_constant<int, 64 % kHalf>;
          using C3 = std::integral_constant<int, 96 % kHalf>;
          if (half == 0) {  // shared columns first
            add(C0{}); done_shared(buf); add(C1{});
            if constexpr (kHalf == 128) { add(C2{}); add(C3{}); }
          } else {
            if constexpr (kHalf == 128) { add(C3{}); done_shared(buf); add(C2{}); }
            add(C1{}); add(C0{});
          }
          done_all(buf);
        }
        if (!ok) break;
      }
      const int buf = use & 1;
      if constexpr (!kSum) {
        ok = __all_sync(0xffffffffu, mbar_wait(&s_acc_full[buf], (use >> 1) & 1, &s_fail));
        if (!ok) break;
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
      }
#pragma unroll
      for (int i = 0; i < kGroups; ++i) {
        // shared columns first
        const int gr = kSum ? i : kWarps == 4 ? (buf == 0 ? (i + kGroups - 1) % kGroups : i) : half == 0 ? i : kGroups - 1 - i;
        const int col = gr * kCols;
        float v[kCols];
        if constexpr (kSum) {
#pragma unroll
          for (int j = 0; j < kCols; ++j) v[j] = sum[i * kCols + j];
        } else {
          uint32_t r[kCols / 32][32];
#pragma unroll
          for (int h = 0; h < kCols / 32; ++h) tmem_load32(own + acc_col<kBN>(buf) + col + 32 * h, r[h]);
          asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
          if (i == 0) done_shared(buf);
          if (i == kGroups - 1) done_all(buf);
#pragma unroll
          for (int j = 0; j < kCols; ++j) v[j] = __uint_as_float(r[j / 32][j % 32]);
        }
        if (col >= cols) continue;
        if (p.bias) {
          __syncwarp();
#pragma unroll
          for (int h = 0; h < kCols; h += 32) bias_s[h + lane] = n0 + col + h + lane < p.n ? load1<kT>(p.bias, n0 + col + h + lane) : 0.0f;
          __syncwarp();
#pragma unroll
          for (int j = 0; j < kCols; j += 4) {
            const float4 b = *reinterpret_cast<const float4*>(bias_s + j);
            v[j] = __fadd_rn(v[j], b.x); v[j + 1] = __fadd_rn(v[j + 1], b.y);
            v[j + 2] = __fadd_rn(v[j + 2], b.z); v[j + 3] = __fadd_rn(v[j + 3], b.w);
          }
        }
        // a row of 128 bytes per lane, its 16-byte pieces swizzled as the tensor map says
        if ((kTwo || p.store) && lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
        __syncwarp();
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          uint4 w;
          if constexpr (kT == kF32) {
            w = make_uint4(__float_as_uint(v[4 * q]), __float_as_uint(v[4 * q + 1]), __float_as_uint(v[4 * q + 2]), __float_as_uint(v[4 * q + 3]));
          } else {
            w = make_uint4(pack16<kT>(v[8 * q], v[8 * q + 1]), pack16<kT>(v[8 * q + 2], v[8 * q + 3]),
                           pack16<kT>(v[8 * q + 4], v[8 * q + 5]), pack16<kT>(v[8 * q + 6], v[8 * q + 7]));
          }
          *reinterpret_cast<uint4*>(stage + lane * 128 + ((q ^ (lane & 7)) << 4)) = w;
        }
        if (n0 + col < p.store) {
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();
          if (lane == 0 && m0 < p.m) {
            tma_store(&c.maps[kTwo ? item.call : 0].out, n0 + col, m0, stage);
            asm volatile("cp.async.bulk.commit_group;" ::: "memory");
          }
        } else {
          // rows of no 16-byte multiple, or a group that they end in: as many
          // bytes to a lane as their alignment allows, consecutive lanes along
          // a row
          __syncwarp();
          constexpr int kEb = elem_bytes<kT>();
          char* const dst = static_cast<char*>(p.out) + (m0 * p.ldo + n0 + col) * kEb;
          const int64_t row_bytes = p.ldo * kEb;
          const auto put_rows = [&](auto unit) {
            using Unit = decltype(unit);
            constexpr int kBytes = sizeof(Unit), kLanes = 128 / kBytes, kRows = kLanes < 32 ? 32 / kLanes : 1;
            const int byte = lane * kBytes % 128, row = lane / kLanes;
            char* at = dst + row * row_bytes + byte;
#pragma unroll 16
            for (int r = row; r < 32; r += kRows, at += kRows * row_bytes)
#pragma unroll
              for (int h = 0; h < 128; h += 32 * kBytes)  // 2-byte units: two to a lane
                *reinterpret_cast<Unit*>(at + h) =
                    *reinterpret_cast<const Unit*>(stage + r * 128 + ((((byte + h) >> 4) ^ (r & 7)) << 4) + (byte & 15));
          };
          if (m0 + 32 <= p.m && n0 + col + kCols <= p.n) {
            if (p.unit == 8) put_rows(uint2{});
            else if (kT == kF32 || p.unit == 4) put_rows(uint32_t{});
            else put_rows(uint16_t{});
          } else if (n0 + col < p.n) {
            using Elem = std::conditional_t<kT == kF32, uint32_t, uint16_t>;
            for (int r = 0; r < 32 && m0 + r < p.m; ++r)
#pragma unroll
              for (int h = 0; h < kCols; h += 32) {
                const int byte = (h + lane) * kEb;
                if (n0 + col + h + lane < p.n)
                  *reinterpret_cast<Elem*>(dst + r * row_bytes + byte) =
                      *reinterpret_cast<const Elem*>(stage + r * 128 + (((byte >> 4) ^ (r & 7)) << 4) + (byte & 15));
              }
          }
          __syncwarp();
        }
      }
      if (!kSum) ++use;
    }
    if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
  }
  if (s_fail && lane == 0 && warp < 2) let_copies_land();
  __syncwarp();
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  cluster_sync();
  if (warp == 1) asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols));
}

// --------------------------------------------------------------------------
// product with few rows, or few tiles
//
// For few lines of A (tokens) the roles change: the 128 rows of the matrix
// instruction are lines of B (the weight's outputs) and its columns the few
// lines of A, so no product is wasted on rows that are not there.  Such a
// product is bound by reading B once, and a cluster of `split` CTAs divides
// the summed axis, so that all SMs read.  Each CTA keeps its part's sums in
// its tensor memory; at the end CTA r gathers, from all of the cluster over
// distributed shared memory, the r-th share of the columns and adds the parts
// in the order of the ranks.  (Four columns to a store: 33 x 4096 x 11008 8.0
// us against 9.7 a column at a time, 500 x 1024 x 1000 in four parts 6.8
// against 12.4.)  Products of more lines that have few tiles and a long sum
// are split here too, 128 lines to a tile: 353 x 9883 x 135 8.4 us against
// 21.3 in pairs.
//
// Up to kFuse lines, A may also come unquantized: the warps that store in the
// end then quantize each stage's 128 columns on the way into shared memory
// while the weight's copies are under way, which saves the quantizer's launch
// and its results' way through memory.  Every CTA of a rank quantizes the
// same part of A again, so this pays for few lines only (33 x 4096 x 11008,
// timed with a version of it for 64 lines: 19.2 us; in two kernels 11.3).
//
// Measured, call after call in a captured graph, through weights of over 500
// MB, so that each is read from DRAM: 1 x 4096 x 4096 6.0 us (its 16.8 MB take
// 2.5 at the copy rate), 1 x 4096 x 11008 10.2 (6.7), 33 x 4096 x 11008 11.4
// (6.9) without the quantizer and 14.1 with it.  With one weight again and
// again, then in L2, 4.8, 6.8, 8.0 and 11.6; the other times here are of that
// kind.  What it takes beyond the reading is a launch, the first copies'
// latency and the gathering, 1 us or so each.

constexpr int kFuse = 16;
constexpr int kFewThreads = 320;  // warp 0 copies, warp 1 issues, warps 2 to 9 quantize and store
constexpr int kFewWarps = 8;
template <int kBN> __host__ __device__ constexpr int few_stages() { return kBN == 128 ? 3 : kBN >= 48 ? 4 : 5; }
template <int kBN> __host__ __device__ constexpr int few_stage_bytes() { return kTile * kBK + kBN * kBK; }
// Columns of sums that go to the CTA that gathers them in one store.
template <int kBN> __host__ __device__ constexpr int few_unit() { return kBN >= 32 ? 4 : 2; }
// Stages and their scales; the gathered parts, at most seven units more than
// kBN columns of 128 fp32 sums, take the stages' place.
template <int kBN> __host__ __device__ constexpr int few_smem() {
  static_assert((kBN + 7 * few_unit<kBN>()) * kTile * 4 <= few_stages<kBN>() * few_stage_bytes<kBN>(), "the parts fit the stages");
  return 1024 + few_stages<kBN>() * (few_stage_bytes<kBN>() + 2 * kSfTile);
}
// Two CTAs share an SM and its tensor memory.  Accumulators that fit beside
// the scales: sums move on to the next after kChunk blocks, or later where
// that would take more of them.
constexpr uint32_t kFewCols = kTmemCols / 2, kFewSfCol = kFewCols - 16;
template <int kBN> __host__ __device__ constexpr int few_accs() { return static_cast<int>(kFewSfCol) / kBN; }
constexpr int kMaxSplit = 8;  // CTAs of a portable cluster
// Longest line of A that the kernel quantizes for fp32 results: longer ones
// leave the accumulators of a cluster's CTAs more than kChunk blocks each.
constexpr int64_t kFuseCols = int64_t{kMaxSplit} * few_accs<kFuse>() * kChunk * kBK;

__device__ __forceinline__ void tma_load_one(void* dst, const CUtensorMap* map, int x, int y, uint64_t* bar) {
  asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];"
               ::"r"(smem_u32(dst)), "l"(map), "r"(x), "r"(y), "r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void commit_one(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
               ::"r"(smem_u32(dst)), "l"(src), "r"(bytes), "r"(smem_u32(bar)) : "memory");
}

struct FewArgs {
  const uint8_t* sfw;
  const uint8_t* sfx;
  const void* bias;
  void* out;
  int64_t ldo;
  const void* x;         // A itself, `ldx` elements between lines, where the kernel quantizes it
  int64_t ldx;
  int vec;               // its lines start on 16-byte boundaries and hold whole 16-byte pieces
  int m, n, k;           // lines of A (columns here), lines of B (rows here), summed axis
  int a_trans, b_trans;
  int split;             // CTAs of a cluster, along the summed axis
  int tiles_n;           // tiles of 128 lines of B
  int b_ready;           // B is no result of the kernel ahead
};

// Eight consecutive values of a line of A from element e on, zero past k.
template <int kT>
__device__ __forceinline__ void few_load(const FewArgs& p, int line, int e, uint4 (&w)[kT == kF32 ? 2 : 1]) {
  constexpr int kPieces = kT == kF32 ? 2 : 1, kVals = 16 / elem_bytes<kT>();
  const char* const src = static_cast<const char*>(p.x) + (line * p.ldx + e) * elem_bytes<kT>();
#pragma unroll
  for (int q = 0; q < kPieces; ++q) {
    w[q] = make_uint4(0u, 0u, 0u, 0u);
    if (line >= p.m) continue;
    if (p.vec) {
      if (e + q * kVals < p.k) w[q] = __ldg(reinterpret_cast<const uint4*>(src) + q);
    } else {
#pragma unroll
      for (int j = 0; j < kVals; ++j)
        if (e + q * kVals + j < p.k) {
          if (kT == kF32) (&w[q].x)[j] = reinterpret_cast<const uint32_t*>(src)[q * kVals + j];
          else (&w[q].x)[j / 2] |= static_cast<uint32_t>(reinterpret_cast<const uint16_t*>(src)[q * kVals + j]) << (16 * (j % 2));
        }
    }
  }
}

// map_w: lines of B in boxes of 128; map_x: lines of A in boxes of kBN, all of
// them in one where it is less than 128 (a transposed A's box has 128: a
// swizzled row of it).
template <int kT, int kBN, bool kFused>
__global__ void __launch_bounds__(kFewThreads, 2)
fp8_matmul_few_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_x, const FewArgs p) {
  static_assert(!kFused || kBN == kFuse, "scales of up to 32 lines lie in one column");
  constexpr int kStages = few_stages<kBN>(), kW = kTile * kBK, kStage = few_stage_bytes<kBN>(), kAccs = few_accs<kBN>();
  extern __shared__ uint8_t smem_raw[];
  uint8_t* const sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* const sf = sm + kStages * kStage;
  float* const parts = reinterpret_cast<float*>(sm);  // [rank][unit of the share][128][kQ], once the stages are done with
  __shared__ __align__(8) uint64_t s_full[kStages], s_empty[kStages], s_done;
  __shared__ uint32_t s_tmem;
  __shared__ int s_fail;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  uint32_t rank;
  asm("mov.u32 %0, %cluster_ctarank;" : "=r"(rank));
  const int kblocks = (p.k + kBK - 1) / kBK, groups = (kblocks + 3) / 4;
  const int tile = static_cast<int>(blockIdx.x) / p.split, n0 = tile % p.tiles_n * kTile, m0 = kBN == 128 ? tile / p.tiles_n * kBN : 0;
  const int lines = p.m - m0 < kBN ? p.m - m0 : kBN;
  // this CTA's blocks of the summed axis, and its accumulators' share of them
  const int kb0 = static_cast<int>(static_cast<int64_t>(kblocks) * rank / p.split);
  const int count = static_cast<int>(static_cast<int64_t>(kblocks) * (rank + 1) / p.split) - kb0;
  const int least = (count + kAccs - 1) / kAccs, chunk = least > kChunk ? least : kChunk;
  const int accs = (count + chunk - 1) / chunk;

  const auto weight = [&](int i, int s) {  // block i of this CTA's, into stage s
    const int kb = kb0 + i;
    const bool scales = i == 0 || (kb & 3) == 0;
    mbar_expect_tx(&s_full[s], (kFused ? kW : kStage) + (scales ? (kFused ? 1 : 2) * kSfTile : 0));
    tma_load_one(sm + s * kStage, &map_w, p.b_trans ? n0 : kb * kBK, p.b_trans ? kb * kBK : n0, &s_full[s]);
    if (scales)
      bulk_load(sf + s * 2 * kSfTile, p.sfw + (static_cast<int64_t>(n0 / 128) * groups + kb / 4) * kSfTile, kSfTile, &s_full[s]);
  };
  const int ahead = count < kStages ? count : kStages;
  if (warp == 0) {
    if (elect_one()) {
      s_fail = 0;
      for (int i = 0; i < kStages; ++i) { mbar_init(&s_full[i], kFused ? 2 : 1); mbar_init(&s_empty[i], 1); }
      mbar_init(&s_done, 1);
      asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
      // the first stages' weights, at once where they do not depend on the kernel ahead
      if (!p.b_ready) wait_for_inputs();
      for (int i = 0; i < ahead; ++i) weight(i, i);
    }
    __syncwarp();
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&s_tmem)), "r"(kFewCols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  __syncwarp();
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  const uint32_t tmem = s_tmem;

  if (warp == 0) {
    const bool one = elect_one();
    wait_for_inputs();
    let_next_begin();
    Ring<kStages> ring;
    for (int i = 0; i < count; ++i, ring.next()) {
      if (i >= ahead && !mbar_wait(&s_empty[ring.s], ring.phase ^ 1u, &s_fail)) break;
      if (one) {
        if (i >= ahead) weight(i, ring.s);
        if constexpr (!kFused) {
          const int kb = kb0 + i;
          tma_load_one(sm + ring.s * kStage + kW, &map_x, p.a_trans ? m0 : kb * kBK, p.a_trans ? kb * kBK : m0, &s_full[ring.s]);
          if (i == 0 || (kb & 3) == 0)
            bulk_load(sf + ring.s * 2 * kSfTile + kSfTile, p.sfx + (static_cast<int64_t>(m0 / 128) * groups + kb / 4) * kSfTile, kSfTile,
                      &s_full[ring.s]);
        }
      }
      __syncwarp();
    }
  } else if (warp == 1) {
    const bool one = elect_one();
    const uint32_t idesc = (static_cast<uint32_t>(p.b_trans) << 15) | (static_cast<uint32_t>(p.a_trans) << 16) |
                           ((kBN / 8) << 17) | (1u << 23) | ((kTile / 16) << 24);
    const uint64_t dw0 = smem_desc(smem_u32(sm), 16, 1024, 2), dx0 = smem_desc(smem_u32(sm + kW), 16, 1024, 2);
    const uint64_t dsf0 = smem_desc(smem_u32(sf), 16, 128, 0);
    const uint32_t sw = p.b_trans ? 4096 / 16 : 32 / 16, sx = p.a_trans ? 4096 / 16 : 32 / 16;
    Ring<kStages> ring;
    uint32_t acc = tmem;
    int left = chunk;  // blocks that this accumulator still takes
    for (int i = 0; i < count; ++i, ring.next()) {
      const int kb = kb0 + i;
      if (!mbar_wait(&s_full[ring.s], ring.phase, &s_fail)) break;
      asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
      if (one) {
        const uint64_t dw = dw0 + static_cast<uint32_t>(ring.s * (kStage / 16)), dx = dx0 + static_cast<uint32_t>(ring.s * (kStage / 16));
        const uint64_t d = dsf0 + static_cast<uint32_t>(ring.s * (2 * kSfTile / 16));
        // two sets of scales of either operand; where A is quantized here, its stage holds that one block's
        const uint32_t tw = tmem + kFewSfCol + 4 * ((kb >> 2) & 1), tx = tmem + kFewSfCol + 8 + 4 * ((kFused ? kb : kb >> 2) & 1);
        const bool scales = i == 0 || (kb & 3) == 0;
        if (scales) asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(tw), "l"(d) : "memory");
        if (scales || kFused) asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(tx), "l"(d + kSfTile / 16) : "memory");
        const uint32_t id = idesc + static_cast<uint32_t>(kb & 3) * (kFused ? 1u << 29 : (1u << 4) | (1u << 29));
#pragma unroll
        for (uint32_t q = 0; q < 4; ++q)
          asm volatile("{\n .reg .pred p;\n setp.ne.b32 p, %6, 0;\n"
                       "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n}"
                       ::"r"(acc), "l"(dw + q * sw), "l"(dx + q * sx), "r"(id), "r"(tw), "r"(tx),
                       "r"(static_cast<uint32_t>(left != chunk || q != 0)) : "memory");
        commit_one(&s_empty[ring.s]);
      }
      __syncwarp();
      if (--left == 0) { left = chunk; acc += kBN; }
    }
    if (one) commit_one(&s_done);
  } else if constexpr (kFused) {
    // A warp to each stage, sixteen lanes to a line, eight columns to a lane:
    // the blocks' latencies overlap across the warps.  (All warps on each
    // block, two lines to a warp: 1 x 4096 x 11008 10.7 us.)  A warp sees
    // every phase of its own stage's barrier: it never runs two ahead, where
    // a wait on the parity alone would let it pass.
    static_assert(kStages <= kFewWarps, "a warp to each stage");
    constexpr int kHalves = kBN / 2, kPieces = kT == kF32 ? 2 : 1;
    const int part = lane % 16, first = lane / 16;
    wait_for_inputs();
    const int s = warp - 2;
    uint32_t phase = 1;
    for (int i = s < kStages ? s : count; i < count; i += kStages, phase ^= 1u) {
      uint4 w[kHalves][kPieces];
#pragma unroll
      for (int h = 0; h < kHalves; ++h)
        if (2 * h < p.m) few_load<kT>(p, first + 2 * h, (kb0 + i) * kBK + 8 * part, w[h]);
      if (i >= kStages && !__all_sync(0xffffffffu, mbar_wait(&s_empty[s], phase, &s_fail))) break;
#pragma unroll
      for (int h = 0; h < kHalves; ++h) {
        if (2 * h >= p.m) break;
        const int line = first + 2 * h;
        uint32_t top = max_piece<kT>(w[h][0]);
        if (kPieces == 2) top = max(top, max_piece<kT>(w[h][kPieces - 1]));
        if (kT != kF32) top = max(top & 0xffffu, top >> 16);
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
        const uint32_t b = scale_byte(widen_bits<kT>(top));
        const float inv = inv_scale(b);
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = __fmul_rn(kT == kF32 ? piece<kT>(w[h][j / 4 % kPieces], j % 4) : piece<kT>(w[h][0], j), inv);
        const uint2 codes = make_uint2(codes2(v[0], v[1]) | codes2(v[2], v[3]) << 16, codes2(v[4], v[5]) | codes2(v[6], v[7]) << 16);
        // the 128-byte swizzle: 16-byte piece c of line l at c ^ (l mod 8)
        *reinterpret_cast<uint2*>(sm + s * kStage + kW + line * kBK + (((part / 2) ^ (line & 7)) << 4) + (part & 1) * 8) = codes;
        if (part == 0) *reinterpret_cast<uint32_t*>(sf + s * 2 * kSfTile + kSfTile + line * 16) = b;
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) mbar_arrive(&s_full[s]);
    }
  }
  __syncwarp();
  // warps w and w + 4 share a quarter of the rows and take turns at the columns
  const int quarter = warp & 3, half = (warp - 2) / 4;
  // columns that a CTA gathers, in units of kQ that move as one; u / share is
  // (u * magic) >> 16 for the few units there are
  constexpr int kQ = few_unit<kBN>();
  const uint32_t share = (kBN / kQ + p.split - 1) / p.split, magic = (65536 + share - 1) / share;
  const int row = quarter * 32 + lane;
  bool ok = true;
  if (warp >= 2) {
    ok = __all_sync(0xffffffffu, mbar_wait(&s_done, 0, &s_fail));
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  }
  if (s_fail && lane == 0 && warp < 2) let_copies_land();
  __syncwarp();
  cluster_sync();  // every CTA is done with its stages: the parts may take their place
  if (warp >= 2) {
#pragma unroll
    for (int c0 = 0; c0 < kBN; c0 += 32) {
      const int c = c0 + 16 * half;
      if (c >= kBN || c >= lines) break;
      float sum[16];
#pragma unroll
      for (int u = 0; u < 16; ++u) sum[u] = 0.0f;
      for (int a = 0; a < accs; ++a) {
        uint32_t r[16];
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
                       "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
                     : "r"(tmem + (static_cast<uint32_t>(quarter * 32) << 16) + a * kBN + c));
        asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
        for (int u = 0; u < 16; ++u) sum[u] = __fadd_rn(sum[u], __uint_as_float(r[u]));
      }
#pragma unroll
      for (int u = 0; u < 16; u += kQ) {
        if (c + u >= lines) break;
        const uint32_t unit = (c + u) / kQ, to = unit * magic >> 16, at = (rank * share + unit - to * share) * kTile + row;
        uint32_t dst;
        asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(dst) : "r"(smem_u32(parts + kQ * at)), "r"(to));
        if constexpr (kQ == 4)
          asm volatile("st.shared::cluster.v4.f32 [%0], {%1,%2,%3,%4};"
                       ::"r"(dst), "f"(sum[u]), "f"(sum[u + 1]), "f"(sum[u + 2]), "f"(sum[u + 3]) : "memory");
        else
          asm volatile("st.shared::cluster.v2.f32 [%0], {%1,%2};" ::"r"(dst), "f"(sum[u]), "f"(sum[u + 1]) : "memory");
      }
    }
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  }
  __syncwarp();
  cluster_sync();
  if (warp >= 2 && ok && n0 + row < p.n) {
    const float bias = p.bias ? load1<kT>(p.bias, n0 + row) : 0.0f;
    for (uint32_t u = half; u < share; u += 2) {
      const int m = static_cast<int>((rank * share + u) * kQ);
      if (m >= lines) break;
      float sum[kQ];
      const auto add = [&](uint32_t r, bool first) {
        const float* const from = parts + kQ * ((r * share + u) * kTile + row);
        float v[kQ];
        if constexpr (kQ == 4) *reinterpret_cast<float4*>(v) = *reinterpret_cast<const float4*>(from);
        else *reinterpret_cast<float2*>(v) = *reinterpret_cast<const float2*>(from);
#pragma unroll
        for (int j = 0; j < kQ; ++j) sum[j] = first ? v[j] : __fadd_rn(sum[j], v[j]);
      };
      add(0, true);
      for (int r = 1; r < p.split; ++r) add(r, false);
#pragma unroll
      for (int j = 0; j < kQ; ++j)
        if (m + j < lines) store1<kT>(p.out, (m0 + m + j) * p.ldo + n0 + row, p.bias ? __fadd_rn(sum[j], bias) : sum[j]);
    }
  }
  if (warp == 1) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kFewCols));
}

// A product over nothing: the bias, or zero.
template <int kT>
__global__ void __launch_bounds__(256)
fill_rows_kernel(const void* __restrict__ bias, void* __restrict__ out, int64_t ldo, int64_t m, int64_t n) {
  wait_for_inputs();
  let_next_begin();
  const int64_t stride = static_cast<int64_t>(gridDim.x) * blockDim.x;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < m * n; i += stride)
    store1<kT>(out, i / n * ldo + i % n, bias ? load1<kT>(bias, i % n) : 0.0f);
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

// Map of a row-major matrix for boxes of box_cols x box_rows elements.
bwd_status matrix_map(CUtensorMap* map, CUtensorMapDataType type, const void* base, int64_t rows, int64_t cols,
                      int64_t pitch_bytes, int box_cols, int box_rows, CUtensorMapSwizzle swizzle) {
  EncodeFn encode = nullptr;
  bwd_status s = encode_fn(&encode);
  if (s != BWD_OK) return s;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(pitch_bytes)};
  const cuuint32_t box[2] = {static_cast<cuuint32_t>(box_cols), static_cast<cuuint32_t>(box_rows)}, step[2] = {1, 1};
  const CUresult r = encode(map, type, 2, const_cast<void*>(base), dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
                            swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(BWD_ERR_CUDA, "cuTensorMapEncodeTiled: error %d", static_cast<int>(r));
  return BWD_OK;
}

// Map of one operand's codes: `lines` lines of k codes, box of box_lines lines.
// It reaches over the rows' pads (zeros along k; lines that no result shows),
// because a box that ends inside 32 bytes is copied more slowly: 1000 x 8192 x
// 1000 transposed 15.9 us against 29.4, 8192 x 200 x 8192 24.7 against 29.0.
bwd_status code_map(CUtensorMap* map, const uint8_t* codes, int64_t lines, int64_t k, int trans, int box_lines) {
  if (trans)
    return matrix_map(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, codes, k, bwd_fp8_pitch(lines), bwd_fp8_pitch(lines), box_lines, kBK,
                      box_lines == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B);
  return matrix_map(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, codes, lines, bwd_fp8_pitch(k), bwd_fp8_pitch(k), kBK, box_lines,
                    CU_TENSOR_MAP_SWIZZLE_128B);
}

// Map of a scale array: one row of 512 bytes for each of its tiles.
bwd_status scale_map(CUtensorMap* map, const uint8_t* scales, int64_t tiles) {
  return matrix_map(map, CU_TENSOR_MAP_DATA_TYPE_UINT32, scales, tiles, kSfTile / 4, kSfTile, kSfTile / 4, 1, CU_TENSOR_MAP_SWIZZLE_NONE);
}

// The largest of 8, 4 and 2 bytes that divides a matrix's address and row.
int unit_of(const void* base, int64_t row_bytes) {
  return aligned_to(base, 8) && row_bytes % 8 == 0 ? 8 : aligned_to(base, 4) && row_bytes % 4 == 0 ? 4 : 2;
}

constexpr int64_t kMaxDim = int64_t{1} << 30;

bool valid_type(int t) { return t == BWD_F32 || t == BWD_BF16 || t == BWD_F16; }
int64_t tiles_of(int64_t n) { return (n + kTile - 1) / kTile; }
int64_t groups_of(int64_t n) { return (tiles_of(n) + 3) / 4; }

template <typename... Params, typename... Args>
bwd_status launch_ex(void (*kernel)(Params...), dim3 grid, int threads, int cluster, int smem, cudaStream_t st, const char* what,
                     const Args&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  if (cluster > 0) {
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim = {static_cast<unsigned>(cluster), 1, 1};
  }
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 0 ? 2 : 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
  return e == cudaSuccess ? BWD_OK : cuda_fail(e, what);
}

template <int kT>
bwd_status launch_quantize(int mode, const QuantArgs& a, cudaStream_t st) {
  const auto launch = [&](auto m, auto sums) {
    constexpr int kMode = decltype(m)::value;
    constexpr bool kSums = decltype(sums)::value;
    const dim3 grid(static_cast<unsigned>(tiles_of(a.cols)), static_cast<unsigned>(tiles_of(a.rows)));
    return launch_ex(a.vec ? fp8_quantize_kernel<kT, kMode, kSums, true> : fp8_quantize_kernel<kT, kMode, kSums, false>, grid,
                     32 * q_warps<kT>(), 0, 0, st, "fp8_quantize_kernel launch", a);
  };
  using Rows = std::integral_constant<int, BWD_FP8_ROWS>;
  using Cols = std::integral_constant<int, BWD_FP8_COLS>;
  using Both = std::integral_constant<int, BWD_FP8_ROWS | BWD_FP8_COLS>;
  if (mode == BWD_FP8_ROWS) return launch(Rows{}, std::false_type{});
  if (mode == BWD_FP8_TILES) return launch(std::integral_constant<int, BWD_FP8_TILES>{}, std::false_type{});
  if (mode == BWD_FP8_COLS) return a.col_sums ? launch(Cols{}, std::true_type{}) : launch(Cols{}, std::false_type{});
  return a.col_sums ? launch(Both{}, std::true_type{}) : launch(Both{}, std::false_type{});
}

// What a launch needs to know of the device, found once for each.
constexpr int kMaxDevices = 64;
struct DeviceState {
  bool ready = false;
  unsigned long long ctx = 0;
  int sms = 0;
  int pairs = 0;  // CTA pairs that are resident at a time
  int clusters[kMaxSplit + 1] = {};  // clusters of so many CTAs that find an SM for each CTA
};
std::mutex g_mu;
DeviceState g_dev[kMaxDevices];

template <typename F>
cudaError_t opt_in(F* kernel, int smem) {
  return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
}

template <int kT, int kBN, int kWarps>
cudaError_t opt_in_pairs() {
  const cudaError_t e = opt_in(fp8_matmul_kernel<kT, kBN, kT == kF32, kWarps, false>, mm_smem<kBN, kWarps>());
  return e == cudaSuccess ? opt_in(fp8_matmul_kernel<kT, kBN, kT == kF32, kWarps, true>, mm_smem<kBN, kWarps>()) : e;
}

template <int kT, int kBN, bool kFused = false>
cudaError_t opt_in_few() {
  return opt_in(fp8_matmul_few_kernel<kT, kBN, kFused>, few_smem<kBN>());
}

template <int kT>
cudaError_t opt_in_all_few() {
  const cudaError_t e[] = {opt_in_few<kT, 16>(), opt_in_few<kT, 32>(), opt_in_few<kT, 48>(), opt_in_few<kT, 64>(), opt_in_few<kT, 128>(),
                           opt_in_few<kT, kFuse, true>()};
  for (const cudaError_t x : e)
    if (x != cudaSuccess) return x;
  return cudaSuccess;
}

bwd_status ensure_device(const DeviceState** out) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
  if (dev < 0 || dev >= kMaxDevices) return fail(BWD_ERR_CUDA, "device ordinal %d unsupported", dev);
  unsigned long long ctx = 0;
  const bwd_status s = bwd::host::current_context_id(&ctx);
  if (s != BWD_OK) return s;
  std::lock_guard<std::mutex> lock(g_mu);
  DeviceState& d = g_dev[dev];
  *out = &d;
  if (d.ready && d.ctx == ctx) return BWD_OK;
  e = cudaDeviceGetAttribute(&d.sms, cudaDevAttrMultiProcessorCount, dev);
  if (e == cudaSuccess) e = opt_in_pairs<kF32, 256, 8>();
  if (e == cudaSuccess) e = opt_in_pairs<kF32, 128, 8>();
  if (e == cudaSuccess) e = opt_in_pairs<kBF16, 256, 8>();
  if (e == cudaSuccess) e = opt_in_pairs<kF16, 256, 8>();
  if (e == cudaSuccess) e = opt_in_pairs<kBF16, 256, 4>();
  if (e == cudaSuccess) e = opt_in_pairs<kF16, 256, 4>();
  if (e == cudaSuccess) e = opt_in_pairs<kBF16, 128, 8>();
  if (e == cudaSuccess) e = opt_in_pairs<kF16, 128, 8>();
  if (e == cudaSuccess) e = opt_in_all_few<kF32>();
  if (e == cudaSuccess) e = opt_in_all_few<kBF16>();
  if (e == cudaSuccess) e = opt_in_all_few<kF16>();
  if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute(MaxDynamicSharedMemorySize)");
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(d.sms / 2 * 2));
  cfg.blockDim = dim3(mm_threads(4));
  cfg.dynamicSmemBytes = mm_smem<256, 4>();
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim = {2, 1, 1};
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaOccupancyMaxActiveClusters(&d.pairs, fp8_matmul_kernel<kBF16, 256, false, 4, false>, &cfg);
  if (e != cudaSuccess) return cuda_fail(e, "cudaOccupancyMaxActiveClusters");
  if (d.pairs < 1) return fail(BWD_ERR_CUDA, "no room for a CTA pair of the matrix product");
  // so much shared memory that no SM takes two
  int smem = 0;
  e = cudaDeviceGetAttribute(&smem, cudaDevAttrMaxSharedMemoryPerMultiprocessor, dev);
  if (e != cudaSuccess) return cuda_fail(e, "cudaDeviceGetAttribute");
  smem = smem / 2 > few_smem<128>() ? smem / 2 : few_smem<128>();
  e = opt_in(fp8_matmul_few_kernel<kBF16, 128, false>, smem);
  if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute(MaxDynamicSharedMemorySize)");
  cfg.blockDim = dim3(kFewThreads);
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  d.clusters[1] = d.sms;
  for (int c = 2; c <= kMaxSplit; ++c) {
    cfg.gridDim = dim3(static_cast<unsigned>(d.sms / c * c));
    attr[0].val.clusterDim = {static_cast<unsigned>(c), 1, 1};
    e = cudaOccupancyMaxActiveClusters(&d.clusters[c], fp8_matmul_few_kernel<kBF16, 128, false>, &cfg);
    if (e != cudaSuccess) return cuda_fail(e, "cudaOccupancyMaxActiveClusters");
  }
  d.ctx = ctx;
  d.ready = true;
  return BWD_OK;
}

// One product's operands: codes and scales of `lines` lines of k elements.
struct Lines {
  const uint8_t* codes;
  const uint8_t* scales;
  int64_t lines;
  int trans;
};

// out = A B^T + bias, k > 0.
struct Product {
  Lines a, b;
  int64_t k;
  const void* bias;
  void* out;
  int64_t ldo;
};

template <int kT, int kBN, int kWarps>
bwd_status launch_matmul(const MmCall<2>& c, int pairs, cudaStream_t st) {
  constexpr bool kSum = kT == kF32;
  constexpr int kThreads = mm_threads(kWarps), kSmem = mm_smem<kBN, kWarps>();
  const dim3 grid(static_cast<unsigned>(2 * (c.items[1] < pairs ? c.items[1] : pairs)));
  if (c.items[0] < c.items[1])
    return launch_ex(fp8_matmul_kernel<kT, kBN, kSum, kWarps, true>, grid, kThreads, 0, kSmem, st, "fp8_matmul_kernel launch", c);
  const MmCall<1> one{{c.maps[0]}, {c.p[0]}, {c.items[0], c.items[1]}, c.sums};
  return launch_ex(fp8_matmul_kernel<kT, kBN, kSum, kWarps, false>, grid, kThreads, 0, kSmem, st, "fp8_matmul_kernel launch", one);
}

// 16-bit results.  Four storing warps where a tile's products (sixteen stages
// or more, some 6 us) outlast its tensor stores.
template <int kT>
bwd_status launch_matmul16(const MmCall<2>& c, bool long_sums, int bn, int pairs, cudaStream_t st) {
  if (bn == 128) return launch_matmul<kT, 128, 8>(c, pairs, st);
  if (long_sums) return launch_matmul<kT, 256, 4>(c, pairs, st);
  return launch_matmul<kT, 256, 8>(c, pairs, st);
}

int64_t tiles_of(const Product& q, int bn) { return (q.a.lines + kBM - 1) / kBM * ((q.b.lines + bn - 1) / bn); }

// Columns of a product's tiles.  A tile of 256 columns takes up to one and a
// half times as long as one of 128 (per stage 0.24 us against 0.17 where few
// pairs work, 0.36 against 0.30 where all do): the wider one where it saves
// more waves than that.  256 x 4096 x 11008 15.1 us against 17.7, 512 x 4096 x
// 4096 11.3 against 14.9 the other way.
int columns_of(const Product& q, int pairs) {
  const auto waves = [&](int bn) { return (tiles_of(q, bn) + pairs - 1) / pairs; };
  return 3 * waves(256) < 2 * waves(128) ? 256 : 128;
}

// One product, or two with tiles of as many columns, by CTA pairs.
// *sums, where given, are column sums that the kernel finishes on the way;
// they are cleared when it does.
bwd_status by_pairs(const Product* q, int count, bwd_dtype dtype, const DeviceState& d, ColSums* sums, cudaStream_t st) {
  const int eb = dtype == BWD_F32 ? 4 : 2, bn = columns_of(q[0], d.pairs);
  MmCall<2> c{};
  bool long_sums = true;
  int64_t total = 0;
  for (int i = 0; i < count; ++i) {
    const Product& o = q[i];
    const int64_t m = o.a.lines, n = o.b.lines, k = o.k, tiles = tiles_of(o, bn);
    total += tiles;
    if (total > 0x3fffffff || tiles_of(m) * groups_of(k) > 0x7fffffff || tiles_of(n) * groups_of(k) > 0x7fffffff)
      return fail(BWD_ERR_INVALID_ARG, "too many tiles");
    const int64_t last = total % d.pairs;
    const bool halves = i + 1 == count && bn == 256 && 2 * last <= d.pairs && last <= tiles;
    MmArgs& p = c.p[i];
    p.bias = o.bias; p.out = o.out; p.ldo = o.ldo;
    p.m = static_cast<int>(m); p.n = static_cast<int>(n); p.k = static_cast<int>(k);
    p.a_trans = o.a.trans; p.b_trans = o.b.trans;
    p.tiles_m = static_cast<int>((m + kBM - 1) / kBM); p.tiles_n = static_cast<int>((n + bn - 1) / bn);
    p.whole = static_cast<int>(halves ? tiles - last : tiles);
    p.sf_rows_b = static_cast<int>(tiles_of(n));
    // A tensor store writes whole pieces of 16 bytes: where a row ends inside
    // one, it would write up to 14 bytes past the end, so the map then covers
    // whole groups of 128 bytes and the rest is stored element by element.
    const int64_t mapped = n * eb % 16 == 0 ? n : n - n % (128 / eb);
    p.store = aligned16(o.out) && o.ldo * eb % 16 == 0 ? static_cast<int>(mapped) : 0;
    p.unit = unit_of(o.out, o.ldo * eb);
    long_sums = long_sums && p.store > 0 && k > 15 * kBK;
    c.items[1] = static_cast<int>(c.items[1] + 2 * tiles - p.whole);
    if (i == 0) c.items[0] = c.items[1];
    MmMaps& maps = c.maps[i];
    bwd_status s;
    if ((s = code_map(&maps.a, o.a.codes, m, k, o.a.trans, kBM / 2)) != BWD_OK) return s;
    if ((s = code_map(&maps.b, o.b.codes, n, k, o.b.trans, bn / 2)) != BWD_OK) return s;
    if ((s = scale_map(&maps.sfa, o.a.scales, tiles_of(m) * groups_of(k))) != BWD_OK) return s;
    if ((s = scale_map(&maps.sfb, o.b.scales, tiles_of(n) * groups_of(k))) != BWD_OK) return s;
    if (p.store) {
      const CUtensorMapDataType type = dtype == BWD_F32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                       : dtype == BWD_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
      if ((s = matrix_map(&maps.out, type, o.out, m, mapped, o.ldo * eb, 128 / eb, 32, CU_TENSOR_MAP_SWIZZLE_128B)) != BWD_OK) return s;
    }
  }
  if (sums) {
    c.sums = *sums;
    sums->out = nullptr;
  }
  if (dtype == BWD_F32)
    return bn == 256 ? launch_matmul<kF32, 256, 8>(c, d.pairs, st) : launch_matmul<kF32, 128, 8>(c, d.pairs, st);
  return dtype == BWD_BF16 ? launch_matmul16<kBF16>(c, long_sums, bn, d.pairs, st) : launch_matmul16<kF16>(c, long_sums, bn, d.pairs, st);
}

// Parts of the summed axis, of two blocks each at least: as many as find an SM
// for each CTA, so that the kernel behind finds room to begin (33 x 4096 x
// 4096 5.6 us with four parts, 6.9 with eight; 500 x 4096 x 1000 8.4 and
// 11.5).  Where up to 64 lines of A leave parts of sixteen blocks or more,
// reading B is what takes the time, and two CTAs on an SM read faster (1 x
// 11008 x 4096 7.9 us with four, 7.0 with eight).
int64_t few_split(int64_t tiles, int64_t blocks, int64_t lines, const DeviceState& d) {
  const int64_t most = blocks / 2 < kMaxSplit ? blocks / 2 : kMaxSplit;
  int64_t split = most < 1 ? 1 : most;
  while (split > 1 && tiles > d.clusters[split]) --split;
  if (lines > 64 || (blocks + split - 1) / split < 16) return split;
  const int64_t two = 2 * d.sms / tiles < most ? 2 * d.sms / tiles : most;
  return two > split ? two : split;
}

// x.codes null: A is p.x, quantized by the kernel.
template <int kT, int kBN, bool kFused>
bwd_status launch_few(const Lines& x, const Lines& w, FewArgs p, const DeviceState& d, cudaStream_t st) {
  CUtensorMap map_w, map_x{};
  bwd_status s;
  if ((s = code_map(&map_w, w.codes, w.lines, p.k, w.trans, kTile)) != BWD_OK) return s;
  if (!kFused && (s = code_map(&map_x, x.codes, x.lines, p.k, x.trans, kBN)) != BWD_OK) return s;
  const int64_t tiles = tiles_of(p.n) * ((p.m + kBN - 1) / kBN);
  p.tiles_n = static_cast<int>(tiles_of(p.n));
  const int64_t blocks = tiles_of(p.k), part = few_accs<kBN>() * kChunk;
  const int64_t split = few_split(tiles, blocks, p.m, d);
  // fp32 results: no accumulator may take more than kChunk blocks
  p.split = static_cast<int>(kT == kF32 && split * part < blocks ? (blocks + part - 1) / part : split);
  return launch_ex(fp8_matmul_few_kernel<kT, kBN, kFused>, dim3(static_cast<unsigned>(tiles * p.split)),
                   kFewThreads, p.split, few_smem<kBN>(), st, "fp8_matmul_few_kernel launch", map_w, map_x, p);
}

template <int kT>
bwd_status few(const Lines& x, const Lines& w, const FewArgs& p, const DeviceState& d, cudaStream_t st) {
  if (!x.codes) return launch_few<kT, kFuse, true>(x, w, p, d, st);
  if (x.trans || p.m > 64) return launch_few<kT, 128, false>(x, w, p, d, st);
  if (p.m > 48) return launch_few<kT, 64, false>(x, w, p, d, st);
  if (p.m > 32) return launch_few<kT, 48, false>(x, w, p, d, st);
  if (p.m > 16) return launch_few<kT, 32, false>(x, w, p, d, st);
  return launch_few<kT, 16, false>(x, w, p, d, st);
}

bwd_status few(const Lines& x, const Lines& w, const FewArgs& p, bwd_dtype dtype, const DeviceState& d, cudaStream_t st) {
  if (dtype == BWD_F32) return few<kF32>(x, w, p, d, st);
  if (dtype == BWD_BF16) return few<kBF16>(x, w, p, d, st);
  return few<kF16>(x, w, p, d, st);
}

// Whether a product goes to the kernel for few lines of A, or few tiles.  For
// more than 64 lines, between kernels of other kinds, it takes some 6 us and
// 0.27 for each block of a part, a pair 3.3 and 0.185 for each block of all;
// with CTAs on more than half of the SMs some 2 us more, because they begin
// later (quantizer and product together, in pairs and here: 128 x 4096 x 1000
// 11.9 and 9.1 us, 606 x 4096 x 270 13.7 and 11.8, 500 x 8192 x 1000 19.3 and
// 16.1; 500 x 2970 x 1000 10.9 and 13.8, 384 x 4096 x 1600 12.0 and 13.2).
bool use_few(const Lines& a, int64_t n, int64_t k, bwd_dtype dtype, const DeviceState& d) {
  const int64_t blocks = tiles_of(k), tiles = tiles_of(n) * tiles_of(a.lines);
  const int64_t split = few_split(tiles, blocks, a.lines, d), part = (blocks + split - 1) / split;
  // fp32 results: no accumulator may take more than kChunk blocks
  if (dtype == BWD_F32 && part > kChunk * (a.trans || a.lines > 64 ? few_accs<128>() : few_accs<64>())) return false;
  return a.lines <= 64 || 3 * part + (2 * tiles * split <= d.sms ? 24 : 48) < 2 * blocks;
}

// b_ready: a kernel that this call launched lies between whatever wrote B and
// this product.
bwd_status matmul(const Product& q, bwd_dtype dtype, int b_ready, ColSums* sums, cudaStream_t st) {
  const DeviceState* d = nullptr;
  const bwd_status s = ensure_device(&d);
  if (s != BWD_OK) return s;
  if (!use_few(q.a, q.b.lines, q.k, dtype, *d)) return by_pairs(&q, 1, dtype, *d, sums, st);
  const FewArgs p{q.b.scales, q.a.scales, q.bias, q.out, q.ldo, nullptr, 0, 0, static_cast<int>(q.a.lines), static_cast<int>(q.b.lines),
                  static_cast<int>(q.k), q.a.trans, q.b.trans, 1, 1, b_ready};
  return few(q.a, q.b, p, dtype, *d, st);
}

// Two products of one call.  In one launch where both are for pairs and want
// the same tiles, the longer sum first (4096 x 1024 x 4096's backward pass 39.4 us
// against 43.7, 700 x 600 x 500's 8.7 against 12.7).
bwd_status both(const Product& q, const Product& r, bwd_dtype dtype, ColSums* sums, cudaStream_t st) {
  const DeviceState* d = nullptr;
  bwd_status s = ensure_device(&d);
  if (s != BWD_OK) return s;
  if (!use_few(q.a, q.b.lines, q.k, dtype, *d) && !use_few(r.a, r.b.lines, r.k, dtype, *d) && columns_of(q, d->pairs) == columns_of(r, d->pairs)) {
    const Product two[2] = {q.k < r.k ? r : q, q.k < r.k ? q : r};
    return by_pairs(two, 2, dtype, *d, sums, st);
  }
  s = matmul(q, dtype, 1, sums, st);
  return s == BWD_OK ? matmul(r, dtype, 1, sums->out ? sums : nullptr, st) : s;
}

// The bias, or zero: a product over nothing.
bwd_status fill(int64_t m, int64_t n, const void* bias, void* out, int64_t ldo, bwd_dtype dtype, cudaStream_t st) {
  const int64_t need = (m * n + 255) / 256;
  const unsigned grid = static_cast<unsigned>(need < 1216 ? need : 1216);
  return launch_ex(dtype == BWD_F32 ? fill_rows_kernel<kF32> : dtype == BWD_BF16 ? fill_rows_kernel<kBF16> : fill_rows_kernel<kF16>,
                   dim3(grid), 256, 0, 0, st, "fill_rows_kernel launch", bias, out, ldo, m, n);
}

bwd_status product(const Product& q, bwd_dtype dtype, int b_ready, ColSums* sums, cudaStream_t st) {
  if (q.a.lines == 0 || q.b.lines == 0) return BWD_OK;
  return q.k == 0 ? fill(q.a.lines, q.b.lines, q.bias, q.out, q.ldo, dtype, st) : matmul(q, dtype, b_ready, sums, st);
}

bwd_status finish_col_sums(const ColSums& a, bwd_dtype dtype, cudaStream_t st) {
  if (!a.out || a.cols == 0) return BWD_OK;
  return launch_ex(dtype == BWD_F32 ? col_sums_kernel<kF32> : dtype == BWD_BF16 ? col_sums_kernel<kBF16> : col_sums_kernel<kF16>,
                   dim3(static_cast<unsigned>((a.cols + 31) / 32)), 32 * kSumWarps, 0, 0, st, "col_sums_kernel launch", a);
}

// Checks of a matrix that is quantized.
bwd_status check_matrix(const void* x, bwd_dtype dtype, int64_t rows, int64_t cols, int64_t ld) {
  if (!valid_type(dtype)) return fail(BWD_ERR_UNSUPPORTED_DTYPE, "dtype %d", (int)dtype);
  if (rows < 0 || cols < 0 || rows > kMaxDim || cols > kMaxDim) return fail(BWD_ERR_INVALID_ARG, "bad size");
  if (tiles_of(rows) > 65535) return fail(BWD_ERR_INVALID_ARG, "more than 65535 * 128 rows");
  if (ld < cols) return fail(BWD_ERR_INVALID_ARG, "ld is less than cols");
  if (rows > 0 && cols > 0) {
    if (!x) return fail(BWD_ERR_INVALID_ARG, "NULL pointer");
    if (!aligned_to(x, dtype == BWD_F32 ? 4 : 2)) return fail(BWD_ERR_INVALID_ARG, "x is not aligned to its element size");
  }
  return BWD_OK;
}

// Quantizes; with col_sums_work, leaves the column sums' parts there.
bwd_status quantize(const void* x, bwd_dtype dtype, int64_t rows, int64_t cols, int64_t ld, int blocks, uint8_t* row_codes,
                    uint8_t* row_scales, uint8_t* col_codes, uint8_t* col_scales, float* col_sums_work, cudaStream_t st) {
  const int eb = dtype == BWD_F32 ? 4 : 2;
  bwd_status s = BWD_OK;
  if (rows > 0 && cols > 0) {
    QuantArgs a{};
    a.x = x; a.rows = rows; a.cols = cols; a.ld = ld;
    a.pitch = bwd_fp8_pitch(cols);
    a.groups_r = groups_of(cols); a.groups_c = groups_of(rows);
    a.codes_r = row_codes; a.scales_r = row_scales; a.codes_c = col_codes; a.scales_c = col_scales;
    a.col_sums = col_sums_work;
    a.vec = ld * eb % 16 == 0 && cols * eb % 16 == 0 && aligned16(x);
    a.unit = unit_of(x, (ld | cols) * eb);
    s = dtype == BWD_F32 ? launch_quantize<kF32>(blocks, a, st) : dtype == BWD_BF16 ? launch_quantize<kBF16>(blocks, a, st)
                                                                                   : launch_quantize<kF16>(blocks, a, st);
  }
  return s;
}

// Divides a workspace into 256-byte aligned pieces.
struct Pieces {
  uint8_t* at;
  int64_t used = 0;
  uint8_t* take(int64_t bytes) {
    uint8_t* const p = at ? at + used : nullptr;
    used += (bytes + 255) / 256 * 256;
    return p;
  }
};

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

int64_t bwd_fp8_pitch(int64_t cols) {
  if (cols < 0 || cols > kMaxDim) return -1;
  // On 128-byte boundaries a stage's row of 128 bytes is one line of L2 and
  // not parts of two, and the copies' boxes never cross a row's end: 8192 x
  // 4097 x 11007 228 us against 300 at a pitch of 4,112, 353 x 8192 x 135
  // transposed 16.4 against 33.7 at pitches of 368 and 144.  Rows that are
  // padded to twice their length or more by it keep the 16 bytes that the
  // tensor maps need.
  return cols > 64 ? (cols + 127) / 128 * 128 : (cols + 15) / 16 * 16;
}

bwd_status bwd_fp8_quantize(const void* x, bwd_dtype dtype, int64_t rows, int64_t cols, int64_t ld, int32_t blocks,
                            uint8_t* row_codes, uint8_t* row_scales, uint8_t* col_codes, uint8_t* col_scales,
                            void* col_sums, float* col_sums_work, void* stream) {
  const bwd_status s = check_matrix(x, dtype, rows, cols, ld);
  if (s != BWD_OK) return s;
  if (blocks != BWD_FP8_ROWS && blocks != BWD_FP8_COLS && blocks != BWD_FP8_TILES && blocks != (BWD_FP8_ROWS | BWD_FP8_COLS))
    return fail(BWD_ERR_INVALID_ARG, "bad block set %d", blocks);
  if (col_sums && !(blocks & BWD_FP8_COLS)) return fail(BWD_ERR_INVALID_ARG, "column sums need blocks along the columns");
  if (cols == 0 || (rows == 0 && !col_sums)) return BWD_OK;
  if (rows > 0) {
    const bool r = blocks & (BWD_FP8_ROWS | BWD_FP8_TILES), c = blocks & BWD_FP8_COLS;
    if ((r && (!row_codes || !row_scales)) || (c && !col_codes) || ((c || blocks == BWD_FP8_TILES) && !col_scales))
      return fail(BWD_ERR_INVALID_ARG, "NULL pointer");
    if ((r && !aligned16(row_codes)) || (c && !aligned16(col_codes)))
      return fail(BWD_ERR_INVALID_ARG, "codes must be 16-byte aligned");
  }
  if (col_sums && (!col_sums_work || !aligned_to(col_sums, dtype == BWD_F32 ? 4 : 2) || !aligned_to(col_sums_work, 4)))
    return fail(BWD_ERR_INVALID_ARG, "column sums need a workspace, both aligned to their element size");
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bwd_status q = quantize(x, dtype, rows, cols, ld, blocks, row_codes, row_scales, col_codes, col_scales,
                                col_sums ? col_sums_work : nullptr, st);
  return q == BWD_OK && col_sums ? finish_col_sums(ColSums{col_sums_work, tiles_of(rows), cols, col_sums}, dtype, st) : q;
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
  return product(Product{Lines{a, a_scales, m, a_trans ? 1 : 0}, Lines{b, b_scales, n, b_trans ? 1 : 0}, k, bias, out, ldo}, dtype, 0,
                 nullptr, static_cast<cudaStream_t>(stream));
}

int64_t bwd_fp8_linear_work_bytes(int64_t rows, int64_t cols) {
  if (rows < 0 || cols < 0 || rows > kMaxDim || cols > kMaxDim) return -1;
  if (rows <= kFuse && cols <= kFuseCols) return 0;
  Pieces w{nullptr};
  w.take(rows * bwd_fp8_pitch(cols));
  w.take(bwd_fp8_scale_bytes(rows, cols));
  return w.used;
}

bwd_status bwd_fp8_linear(const void* x, bwd_dtype dtype, int64_t rows, int64_t cols, int64_t ld, const uint8_t* w,
                          const uint8_t* w_scales, int64_t n, const void* bias, void* y, int64_t ldy, uint8_t* x_col_codes,
                          uint8_t* x_col_scales, void* work, void* stream) {
  bwd_status s = check_matrix(x, dtype, rows, cols, ld);
  if (s != BWD_OK) return s;
  if (n < 0 || n > kMaxDim) return fail(BWD_ERR_INVALID_ARG, "bad size");
  if (ldy < n) return fail(BWD_ERR_INVALID_ARG, "ldy is less than n");
  if (!x_col_codes != !x_col_scales) return fail(BWD_ERR_INVALID_ARG, "column codes and scales go together");
  const int eb = dtype == BWD_F32 ? 4 : 2;
  const bool some = rows > 0 && cols > 0, fused = rows <= kFuse && (dtype != BWD_F32 || cols <= kFuseCols);
  if ((rows > 0 && n > 0 && !y) || (some && !fused && !work) || (some && n > 0 && (!w || !w_scales))) return fail(BWD_ERR_INVALID_ARG, "NULL pointer");
  if (!aligned_to(y, eb) || !aligned_to(bias, eb)) return fail(BWD_ERR_INVALID_ARG, "y and bias must be aligned to their element size");
  if (!aligned16(w) || !aligned16(w_scales) || !aligned16(x_col_codes) || !aligned16(work))
    return fail(BWD_ERR_INVALID_ARG, "codes, scales and work must be 16-byte aligned");
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (fused && some) {
    if (x_col_codes && (s = quantize(x, dtype, rows, cols, ld, BWD_FP8_COLS, nullptr, nullptr, x_col_codes, x_col_scales, nullptr, st)) != BWD_OK)
      return s;
    if (n == 0) return BWD_OK;
    const DeviceState* d = nullptr;
    if ((s = ensure_device(&d)) != BWD_OK) return s;
    const FewArgs p{w_scales, nullptr, bias, y, ldy, x, ld, ld * eb % 16 == 0 && cols * eb % 16 == 0 && aligned16(x),
                    static_cast<int>(rows), static_cast<int>(n), static_cast<int>(cols), 0, 0, 1, 1, x_col_codes != nullptr};
    return few(Lines{nullptr, nullptr, rows, 0}, Lines{w, w_scales, n, 0}, p, dtype, *d, st);
  }
  Pieces pieces{static_cast<uint8_t*>(work)};
  uint8_t* const codes = pieces.take(rows * bwd_fp8_pitch(cols));
  uint8_t* const scales = pieces.take(bwd_fp8_scale_bytes(rows, cols));
  s = quantize(x, dtype, rows, cols, ld, x_col_codes ? BWD_FP8_ROWS | BWD_FP8_COLS : BWD_FP8_ROWS, codes, scales, x_col_codes, x_col_scales,
               nullptr, st);
  if (s != BWD_OK) return s;
  return product(Product{Lines{codes, scales, rows, 0}, Lines{w, w_scales, n, 0}, cols, bias, y, ldy}, dtype, 1, nullptr, st);
}

int64_t bwd_fp8_linear_backward_work_bytes(int64_t rows, int64_t n) {
  if (rows < 0 || n < 0 || rows > kMaxDim || n > kMaxDim) return -1;
  Pieces w{nullptr};
  w.take(rows * bwd_fp8_pitch(n));
  w.take(bwd_fp8_scale_bytes(rows, n));
  w.take(rows * bwd_fp8_pitch(n));
  w.take(bwd_fp8_scale_bytes(n, rows));
  w.take(tiles_of(rows) * n * 4);
  return w.used;
}

bwd_status bwd_fp8_linear_backward(const void* dy, bwd_dtype dtype, int64_t rows, int64_t n, int64_t ld, const uint8_t* w,
                                   const uint8_t* w_col_scales, const uint8_t* x_col_codes, const uint8_t* x_col_scales, int64_t k,
                                   void* dx, int64_t lddx, void* dw, int64_t lddw, void* dbias, void* work, void* stream) {
  bwd_status s = check_matrix(dy, dtype, rows, n, ld);
  if (s != BWD_OK) return s;
  if (k < 0 || k > kMaxDim) return fail(BWD_ERR_INVALID_ARG, "bad size");
  if ((dx && lddx < k) || (dw && lddw < k)) return fail(BWD_ERR_INVALID_ARG, "lddx or lddw is less than k");
  const int eb = dtype == BWD_F32 ? 4 : 2;
  const bool some = rows > 0 && n > 0 && k > 0;
  if ((some && dx && (!w || !w_col_scales)) || (some && dw && (!x_col_codes || !x_col_scales)) || (rows > 0 && n > 0 && !work))
    return fail(BWD_ERR_INVALID_ARG, "NULL pointer");
  if (!aligned_to(dx, eb) || !aligned_to(dw, eb) || !aligned_to(dbias, eb))
    return fail(BWD_ERR_INVALID_ARG, "dx, dw and dbias must be aligned to their element size");
  if (!aligned16(w) || !aligned16(w_col_scales) || !aligned16(x_col_codes) || !aligned16(x_col_scales) || !aligned16(work))
    return fail(BWD_ERR_INVALID_ARG, "codes, scales and work must be 16-byte aligned");
  if (!dx && !dw && !dbias) return BWD_OK;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  Pieces pieces{static_cast<uint8_t*>(work)};
  uint8_t* const row_codes = pieces.take(rows * bwd_fp8_pitch(n));
  uint8_t* const row_scales = pieces.take(bwd_fp8_scale_bytes(rows, n));
  uint8_t* const col_codes = pieces.take(rows * bwd_fp8_pitch(n));
  uint8_t* const col_scales = pieces.take(bwd_fp8_scale_bytes(n, rows));
  float* const sums = reinterpret_cast<float*>(pieces.take(tiles_of(rows) * n * 4));
  const int blocks = (dx ? BWD_FP8_ROWS : 0) | (dw || dbias ? BWD_FP8_COLS : 0);
  s = quantize(dy, dtype, rows, n, ld, blocks, row_codes, row_scales, col_codes, col_scales, dbias ? sums : nullptr, st);
  ColSums left{sums, tiles_of(rows), n, dbias};  // until a product has taken them along
  const Product for_x{Lines{row_codes, row_scales, rows, 0}, Lines{w, w_col_scales, k, 1}, n, nullptr, dx, lddx};
  const Product for_w{Lines{col_codes, col_scales, n, 1}, Lines{x_col_codes, x_col_scales, k, 1}, rows, nullptr, dw, lddw};
  if (s == BWD_OK && dx && dw && some) {
    s = both(for_x, for_w, dtype, &left, st);
  } else {
    if (s == BWD_OK && dx) s = product(for_x, dtype, 1, &left, st);
    if (s == BWD_OK && dw) s = product(for_w, dtype, 1, &left, st);
  }
  if (s == BWD_OK) s = finish_col_sums(left, dtype, st);
  return s;
}

}  // extern "C"
