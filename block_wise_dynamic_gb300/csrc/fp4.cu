// Microscaled 4-bit floating point: quantizer, and the matrix product of two
// quantized operands (sm_103a).
//
// Quantization.  A block of 1 x 32 elements has the scale 2^e with the
// smallest e >= -127 for which no magnitude of the block exceeds 6 * 2^e (6 is
// the largest e2m1 value), and each element the e2m1 code nearest to x 2^-e
// (0, 0.5, 1, 1.5, 2, 3, 4, 6), ties to the even code.  The scaling is exact,
// so the code takes one rounding.  e + 127 is the scale's byte (E8M0); a block
// that holds an infinity or a NaN has the byte 255 (NaN).
//
// Layout.  Two codes to a byte, the earlier one in the low half.  Scales are
// kept as the matrix instruction reads them from tensor memory, in tiles of
// 512 bytes for 128 rows x 4 blocks (row r's word in lane r % 32, column r /
// 32), and two such tiles, 256 columns, follow one another: what one stage of
// the product takes of 128 rows, by one copy.  What lies past the last column
// up to a multiple of 256 has zero codes (up to the pitch) and scales of 0.
//
// Product.  out[m, n] = sum_k A(m, k) B(n, k) + bias[n], both operands' rows
// along k.
#include "tensor.cuh"

namespace {

using bwd::host::check_launch;

constexpr int kTile = 128;         // rows of a scale tile
constexpr int kStageK = 256;       // values of the summed axis in a stage of a product: 128 bytes of codes
constexpr int kStageBytes = 128;
constexpr int kSfTile = 1024;      // bytes of scales for 128 rows x 256 columns
constexpr int kSfGroup = 512;      // of 128 of them

// --------------------------------------------------------------------------
// quantize and dequantize
//
// A warp takes 256 columns of a row at a time, eight consecutive values to a
// lane and four lanes to a block; a CTA 32 rows, whose loads a warp has under
// way together.

// 6 is 1.5 * 2^2: with a = f * 2^p the exponent is p - 2 where f <= 1.5 and
// p - 1 above; adding the distance from 1.5 to 2 in units of the last place,
// less one, carries into the exponent field exactly there.
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax_bits) {
  if (amax_bits >= 0x7f800000u) return 255u;
  const int b = static_cast<int>((amax_bits + 0x3fffffu) >> 23) - 2;
  return static_cast<uint32_t>(b < 0 ? 0 : b);
}
// 2^-e for a scale byte (bytes of finite maxima are at most 253).
__device__ __forceinline__ float inv_scale(uint32_t byte) {
  return __uint_as_float(byte == 255u ? 0x7fffffffu : (254u - byte) << 23);
}
__device__ __forceinline__ float scale_value(uint32_t byte) {
  return __uint_as_float(byte == 255u ? 0x7fffffffu : byte ? byte << 23 : 1u << 22);
}

// Eight codes; cvt rounds to nearest even, and no finite value exceeds 6.
__device__ __forceinline__ uint32_t codes8(const float (&v)[8], float inv) {
  uint32_t r;
  asm("{\n .reg .b8 a, b, c, d;\n .reg .b64 s, x;\n .reg .f32 h, l;\n mov.b64 s, {%9, %9};\n"
      "mov.b64 x, {%1, %2};\n mul.rn.f32x2 x, x, s;\n mov.b64 {l, h}, x;\n cvt.rn.satfinite.e2m1x2.f32 a, h, l;\n"
      "mov.b64 x, {%3, %4};\n mul.rn.f32x2 x, x, s;\n mov.b64 {l, h}, x;\n cvt.rn.satfinite.e2m1x2.f32 b, h, l;\n"
      "mov.b64 x, {%5, %6};\n mul.rn.f32x2 x, x, s;\n mov.b64 {l, h}, x;\n cvt.rn.satfinite.e2m1x2.f32 c, h, l;\n"
      "mov.b64 x, {%7, %8};\n mul.rn.f32x2 x, x, s;\n mov.b64 {l, h}, x;\n cvt.rn.satfinite.e2m1x2.f32 d, h, l;\n"
      "mov.b32 %0, {a, b, c, d};\n}"
      : "=r"(r)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]), "f"(inv));
  return r;
}
__device__ __forceinline__ void values8(uint32_t codes, float (&v)[8]) {
  uint32_t h[4];
  asm("{\n .reg .b8 a, b, c, d;\n mov.b32 {a, b, c, d}, %4;\n"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n cvt.rn.f16x2.e2m1x2 %1, b;\n cvt.rn.f16x2.e2m1x2 %2, c;\n cvt.rn.f16x2.e2m1x2 %3, d;\n}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3]) : "r"(codes));
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[j]));
    v[2 * j] = f.x;
    v[2 * j + 1] = f.y;
  }
}

// Byte of the scale word (four blocks) of row r and group g of 128 columns.
__device__ __forceinline__ int64_t scale_word(int64_t r, int64_t g, int64_t groups) {
  return ((r >> 7) * groups + g) * kSfGroup + (r & 31) * 16 + ((r >> 5) & 3) * 4;
}

constexpr int kRows = 32;  // of a CTA
constexpr int kWarps = 8;
constexpr int kEach = kRows / kWarps;

struct QuantArgs {
  const void* x;
  int64_t rows, cols, ld;  // elements; ld between rows
  int64_t pitch;           // bytes between the rows of codes
  int64_t groups;          // of 128 columns, an even number
  uint8_t* codes;
  uint8_t* scales;
  int unit;                // rows start on boundaries of so many bytes, and hold whole units
};

// Eight values from column c on, zeros past the row's end.
template <int kT, typename Unit>
__device__ __forceinline__ void load8(const char* src, int64_t left, float (&v)[8]) {
  constexpr int kEb = elem_bytes<kT>(), kVals = sizeof(Unit) / kEb;
#pragma unroll
  for (int q = 0; q < 8 / kVals; ++q) {
    const Unit u = q * kVals < left ? __ldcs(reinterpret_cast<const Unit*>(src) + q) : Unit{};
#pragma unroll
    for (int j = 0; j < kVals; ++j) {
      if constexpr (kT == kF32) {
        v[q * kVals + j] = reinterpret_cast<const float*>(&u)[j];
      } else {
        const uint16_t h = reinterpret_cast<const uint16_t*>(&u)[j];
        v[q * kVals + j] = kT == kBF16 ? __uint_as_float(static_cast<uint32_t>(h) << 16) : __half2float(__ushort_as_half(h));
      }
    }
  }
}

// Bytes of a warp's 256 columns.  Where rows are not made of 16-byte pieces,
// they pass through shared memory on the way, so that a warp's access to them
// is one run of units (6391 x 9011 fp16 read back: 151 us with eight values to
// a lane).
template <int kT> __host__ __device__ constexpr int strip_bytes() { return kStageK * elem_bytes<kT>(); }
template <int kT, typename Unit> __host__ __device__ constexpr bool staged() { return sizeof(Unit) < 16; }

// A lane's eight codes, and the bytes of the four blocks that its half warp
// holds in one word.
__device__ __forceinline__ uint32_t quantize8(const float (&v)[8], int lane, uint32_t* word) {
  // magnitudes order like their bits, infinities and NaN above all numbers
  uint32_t top = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) top = max(top, __float_as_uint(v[j]) & 0x7fffffffu);
  top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
  top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
  const uint32_t b = scale_byte(top);
  uint32_t w = b << (lane / 4 % 4 * 8);
  w |= __shfl_xor_sync(0xffffffffu, w, 4);
  w |= __shfl_xor_sync(0xffffffffu, w, 8);
  *word = w;
  return codes8(v, inv_scale(b));
}

// The same of eight values as they lie in memory, and the byte of the lane's
// own block.  16-bit values' magnitudes are compared two at a time, and each
// block's byte is stored by itself (11008 x 4096 bf16: 19.5 us, 21.9 with
// quantize8; 32 rows to a CTA, 21.4 with 16 and 20.1 with 64).
template <int kT>
__device__ __forceinline__ uint32_t quantize_words(const uint32_t (&w)[2 * elem_bytes<kT>()], uint32_t* byte) {
  uint32_t top;
  if constexpr (kT == kF32) {
    top = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) top = max(top, w[j] & 0x7fffffffu);
  } else {
    constexpr uint32_t kMag = 0x7fff7fffu;
    top = __vimax3_u16x2(w[0] & kMag, w[1] & kMag, __vmaxu2(w[2] & kMag, w[3] & kMag));
    top = max(top & 0xffffu, top >> 16);
  }
  top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
  top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
  if constexpr (kT == kBF16) top <<= 16;
  if constexpr (kT == kF16) top = __float_as_uint(__half2float(__ushort_as_half(static_cast<unsigned short>(top))));
  const uint32_t b = scale_byte(top);
  const float inv = inv_scale(b);
  *byte = b;
  uint32_t r;
  if constexpr (kT == kF32) {
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = __uint_as_float(w[j]);
    r = codes8(v, inv);
  } else {
    float v[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (kT == kBF16) {
        v[2 * j] = __uint_as_float(w[j] << 16);
        v[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
      } else {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[j]));
        v[2 * j] = f.x;
        v[2 * j + 1] = f.y;
      }
    }
    r = codes8(v, inv);
  }
  return r;
}

template <int kT, typename Unit>
__global__ void __launch_bounds__(32 * kWarps)
fp4_quantize_kernel(const QuantArgs a) {
  constexpr bool kStaged = staged<kT, Unit>();
  constexpr int kLoads = strip_bytes<kT>() / (32 * static_cast<int>(sizeof(Unit)));
  __shared__ __align__(16) uint8_t s_strip[kStaged ? kWarps : 1][kStaged ? kEach * strip_bytes<kT>() : 16];
  wait_for_inputs();
  let_next_begin();
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int64_t c0 = static_cast<int64_t>(blockIdx.x) * kStageK, c = c0 + 8 * lane, left = a.cols - c;
  const int64_t r0 = static_cast<int64_t>(blockIdx.y) * kRows + warp;
  constexpr int kWords = 2 * elem_bytes<kT>();
  uint32_t v[kEach][kWords];
  if constexpr (kStaged) {
    Unit* const strip = reinterpret_cast<Unit*>(s_strip[warp]);
    const int64_t here = (a.cols - c0) * elem_bytes<kT>();
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const int64_t r = r0 + i * kWarps;
      const Unit* const src = reinterpret_cast<const Unit*>(static_cast<const char*>(a.x) + (r * a.ld + c0) * elem_bytes<kT>());
      Unit u[kLoads];
#pragma unroll
      for (int q = 0; q < kLoads; ++q)
        u[q] = r < a.rows && (32 * q + lane) * static_cast<int>(sizeof(Unit)) < here ? __ldcs(src + 32 * q + lane) : Unit{};
#pragma unroll
      for (int q = 0; q < kLoads; ++q) strip[(i * kLoads + q) * 32 + lane] = u[q];
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const uint4* const from = reinterpret_cast<const uint4*>(s_strip[warp] + i * strip_bytes<kT>()) + lane * (kWords / 4);
#pragma unroll
      for (int q = 0; q < kWords; ++q) v[i][q] = (&from[q / 4].x)[q % 4];
    }
  } else {
    const char* src = static_cast<const char*>(a.x) + (r0 * a.ld + c) * elem_bytes<kT>();
    const int64_t step = kWarps * a.ld * elem_bytes<kT>();
#pragma unroll
    for (int i = 0; i < kEach; ++i, src += step) {
#pragma unroll
      for (int q = 0; q < kWords / 4; ++q) {
        const bool in = r0 + i * kWarps < a.rows && q * (16 / elem_bytes<kT>()) < left;
        const uint4 u = in ? __ldcs(reinterpret_cast<const uint4*>(src) + q) : uint4{};
        v[i][4 * q] = u.x; v[i][4 * q + 1] = u.y; v[i][4 * q + 2] = u.z; v[i][4 * q + 3] = u.w;
      }
    }
  }
  uint8_t* to = a.codes + r0 * a.pitch + c / 2;
#pragma unroll
  for (int i = 0; i < kEach; ++i, to += kWarps * a.pitch) {
    const int64_t r = r0 + i * kWarps;
    if (r >= a.rows) break;
    uint32_t byte;
    const uint32_t codes = quantize_words<kT>(v[i], &byte);
    if (c / 2 < a.pitch) *reinterpret_cast<uint32_t*>(to) = codes;
    if (lane % 4 == 0) a.scales[scale_word(r, 2 * blockIdx.x + lane / 16, a.groups) + lane / 4 % 4] = static_cast<uint8_t>(byte);
  }
}

struct DequantArgs {
  const uint8_t* codes;
  const uint8_t* scales;
  int64_t rows, cols, pitch, groups;
  void* out;
};

template <int kT, typename Unit>
__global__ void __launch_bounds__(32 * kWarps)
fp4_dequantize_kernel(const DequantArgs a) {
  constexpr bool kStaged = staged<kT, Unit>();
  constexpr int kEb = elem_bytes<kT>(), kPieces = 8 * kEb / 16, kStores = strip_bytes<kT>() / (32 * static_cast<int>(sizeof(Unit)));
  __shared__ __align__(16) uint8_t s_strip[kStaged ? kWarps : 1][kStaged ? strip_bytes<kT>() : 16];
  wait_for_inputs();
  let_next_begin();
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int64_t c0 = static_cast<int64_t>(blockIdx.x) * kStageK, c = c0 + 8 * lane;
  const int64_t r0 = static_cast<int64_t>(blockIdx.y) * kRows + warp;
  uint32_t codes[kEach], byte[kEach];
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const int64_t r = r0 + i * kWarps;
    const bool in = r < a.rows && c < a.cols;
    codes[i] = in ? __ldcs(reinterpret_cast<const uint32_t*>(a.codes + r * a.pitch + c / 2)) : 0u;
    byte[i] = in ? a.scales[scale_word(r, 2 * blockIdx.x + lane / 16, a.groups) + lane / 4 % 4] : 0u;
  }
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const int64_t r = r0 + i * kWarps;
    if (r >= a.rows) break;
    float v[8];
    values8(codes[i], v);
    const float s = scale_value(byte[i]);
    uint4 w[kPieces];
#pragma unroll
    for (int j = 0; j < 8; j += kEb == 4 ? 1 : 2) {
      if constexpr (kT == kF32) (&w[j / 4].x)[j % 4] = __float_as_uint(__fmul_rn(v[j], s));
      else (&w[0].x)[j / 2] = pack16<kT>(__fmul_rn(v[j], s), __fmul_rn(v[j + 1], s));
    }
    char* const to = static_cast<char*>(a.out) + (r * a.cols + c0) * kEb;
    if constexpr (kStaged) {
      __syncwarp();
#pragma unroll
      for (int q = 0; q < kPieces; ++q) reinterpret_cast<uint4*>(s_strip[warp])[lane * kPieces + q] = w[q];
      __syncwarp();
      const int64_t here = (a.cols - c0) * kEb;
#pragma unroll
      for (int q = 0; q < kStores; ++q) {
        const int at = (32 * q + lane) * static_cast<int>(sizeof(Unit));
        if (at < here) *reinterpret_cast<Unit*>(to + at) = *reinterpret_cast<const Unit*>(s_strip[warp] + at);
      }
    } else if (c < a.cols) {
#pragma unroll
      for (int q = 0; q < kPieces; ++q)
        if (c + 16 / kEb * q < a.cols) reinterpret_cast<uint4*>(to)[lane * kPieces + q] = w[q];
    }
  }
}

// --------------------------------------------------------------------------
// matrix product
//
// A pair of CTAs (a cluster of two) works on a tile of 256 rows and kBN
// columns: each holds its 128 rows of A and its half of B's, the first CTA
// issues for both, and each CTA's tensor memory holds its own rows' sums and
// the scales.  Pairs walk the tiles with a grid stride; warp 0 copies, warp 1
// issues and eight warps store the tile before.
constexpr int kBM = 256;
constexpr int kThreads = 320;
constexpr int kStoreWarps = 8;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kTmemSf = 448;  // two sets of 24 columns behind the accumulators
constexpr uint32_t kSfSet = 24, kSfHalf = 12;  // for 256 values, for 128: A's 4 columns, B's 8
constexpr int kStoreBytes = 4096;  // staging of one storing warp: 32 rows of 128 bytes

// The matrix instruction adds into its fp32 accumulator with truncation, an
// error that grows with the number of additions.  It is far below a 16-bit
// result's rounding; for fp32 results (kSum) the sums leave the accumulator
// every kChunk stages, 2,048 products, and are added up in registers.
constexpr int kChunk = 8;

template <int kBN> __host__ __device__ constexpr int mm_stages() { return kBN == 128 ? 7 : 5; }
constexpr int kABytes = kBM / 2 * kStageBytes;
template <int kBN> __host__ __device__ constexpr int mm_b_bytes() { return kBN / 2 * kStageBytes; }
template <int kBN> __host__ __device__ constexpr int mm_sf_bytes() { return kSfTile + kBN / 128 * kSfTile; }
template <int kBN> __host__ __device__ constexpr int mm_smem() {
  return 1024 + mm_stages<kBN>() * (kABytes + mm_b_bytes<kBN>() + mm_sf_bytes<kBN>()) + kStoreWarps * kStoreBytes;
}

struct MmArgs {
  CUtensorMap a, b, sfa, sfb, out_map;
  const void* bias;  // [n] or null, of the output's type
  void* out;
  int64_t ldo;
  int m, n, stages;  // stages of the summed axis
  int tiles_n, items;
  int whole;         // the first tiles; the rest are worked on as two halves of 128 columns each
  int sf_rows_b;     // row tiles of B's scales
  int store;         // columns that tensor stores take: all, whole groups only, or none;
  int unit;          // the others go in stores of so many bytes
};

struct Item {
  int m0, n0, cols;
};
template <int kBN>
__device__ __forceinline__ Item item_of(const MmArgs& p, int i) {
  if (kBN == 128 || i < p.whole) return Item{i / p.tiles_n * kBM, i % p.tiles_n * kBN, kBN};
  const int t = p.whole + (i - p.whole) / 2;
  return Item{t / p.tiles_n * kBM, t % p.tiles_n * kBN + (i - p.whole) % 2 * 128, 128};
}

// The two accumulators.  With 256 columns each they share 64, which leaves
// room for the scales: the storing warps read the shared columns first, and
// the next tile's products start when they have.
template <int kBN> __device__ __forceinline__ uint32_t acc_col(int buf) { return buf ? (kBN == 256 ? 192u : 128u) : 0u; }

template <int kT, int kBN, bool kSum>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
fp4_matmul_kernel(const __grid_constant__ MmArgs p) {
  constexpr int kStages = mm_stages<kBN>(), kA = kABytes, kB = mm_b_bytes<kBN>(), kSf = mm_sf_bytes<kBN>();
  extern __shared__ uint8_t smem_raw[];
  uint8_t* const sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* const store = sm + kStages * (kA + kB);
  uint8_t* const sf = store + kStoreWarps * kStoreBytes;
  __shared__ __align__(8) uint64_t s_full[kStages], s_empty[kStages], s_acc_full[2], s_acc_empty[2], s_overlap;
  __shared__ __align__(16) float s_bias[kStoreWarps][64];
  __shared__ uint32_t s_tmem;
  __shared__ int s_fail;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  uint32_t rank;
  asm("mov.u32 %0, %cluster_ctarank;" : "=r"(rank));
  if (threadIdx.x == 0) {
    prefetch_map(&p.a);
    prefetch_map(&p.b);
    prefetch_map(&p.sfa);
    prefetch_map(&p.sfb);
    s_fail = 0;
    for (int i = 0; i < kStages; ++i) { mbar_init(&s_full[i], 1); mbar_init(&s_empty[i], 1); }
    for (int i = 0; i < 2; ++i) { mbar_init(&s_acc_full[i], 1); mbar_init(&s_acc_empty[i], 2 * kStoreWarps); }
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
  const int pairs = static_cast<int>(gridDim.x) / 2, first = static_cast<int>(blockIdx.x) / 2;

  if (warp == 0) {
    wait_for_inputs();
    let_next_begin();
    const bool one = elect_one();
    Ring<kStages> ring;
    bool ok = true;
    for (int t = first; ok && t < p.items; t += pairs) {
      const Item item = item_of<kBN>(p, t);
      // of a half, the copies of B bring as many lines as of a whole
      const int m0 = item.m0 + static_cast<int>(rank) * (kBM / 2), n0 = item.n0 + static_cast<int>(rank) * (item.cols / 2);
      for (int kb = 0; kb < p.stages; ++kb, ring.next()) {
        if (!(ok = mbar_wait(&s_empty[ring.s], ring.phase ^ 1u, &s_fail))) break;
        if (one) {
          const uint32_t bar = leader_addr(&s_full[ring.s]);
          if (rank == 0) mbar_expect_tx(&s_full[ring.s], 2 * (kA + kB + kSf));
          uint8_t* const a = sm + ring.s * (kA + kB);
          tma_load(a, &p.a, kb * kStageBytes, m0, bar);
          tma_load(a + kA, &p.b, kb * kStageBytes, n0, bar);
          // A's for this CTA's rows, B's for the whole tile
          tma_load(sf + ring.s * kSf, &p.sfa, 0, m0 / 128 * p.stages + kb, bar);
#pragma unroll
          for (int h = 0; h < kBN / 128; ++h) {
            const int rt = item.n0 / 128 + h;  // past the last row tile: columns past n, whatever they hold
            tma_load(sf + ring.s * kSf + (1 + h) * kSfTile, &p.sfb, 0, (rt < p.sf_rows_b ? rt : p.sf_rows_b - 1) * p.stages + kb, bar);
          }
        }
        __syncwarp();
      }
    }
  } else if (warp == 1) {
    if (rank == 0) {
      const bool one = elect_one();
      const uint64_t da0 = smem_desc(smem_u32(sm), 16, 1024, 2), db0 = smem_desc(smem_u32(sm + kA), 16, 1024, 2);
      const uint64_t dsf0 = smem_desc(smem_u32(sf), 16, 128, 0);
      Ring<kStages> ring;
      int use = 0;  // accumulators used so far
      bool ok = true;
      const int chunk = kSum ? kChunk : p.stages;
      for (int t = first; ok && t < p.items; t += pairs) {
        const Item item = item_of<kBN>(p, t);
        // e2m1 x e2m1, E8M0 scales, fp32 accumulators
        const uint32_t idesc = (1u << 7) | (1u << 10) | (static_cast<uint32_t>(item.cols / 8) << 17) | (1u << 23) | ((kBM / 128) << 27);
        for (int k0 = 0; ok && k0 < p.stages; k0 += chunk, ++use) {
          const int buf = use & 1;
          ok = mbar_wait(&s_acc_empty[buf], ((use >> 1) & 1) ^ 1, &s_fail);
          if (kBN == 256 && ok && use > 0) ok = mbar_wait(&s_overlap, (use - 1) & 1, &s_fail);
          asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
          const int k1 = p.stages < k0 + chunk ? p.stages : k0 + chunk;
          const uint32_t acc = tmem + acc_col<kBN>(buf);
          for (int kb = k0; ok && kb < k1; ++kb, ring.next()) {
            if (!(ok = mbar_wait(&s_full[ring.s], ring.phase, &s_fail))) break;
            asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
            if (one) {
              const uint64_t da = da0 + static_cast<uint32_t>(ring.s * ((kA + kB) / 16)), db = db0 + static_cast<uint32_t>(ring.s * ((kA + kB) / 16));
              const uint64_t dsf = dsf0 + static_cast<uint32_t>(ring.s * (kSf / 16));
              const uint32_t tsf = tmem + kTmemSf + kSfSet * (kb & 1);
#pragma unroll
              for (int g = 0; g < 2; ++g)
#pragma unroll
                for (int h = 0; h < 1 + kBN / 128; ++h)
                  asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(tsf + kSfHalf * g + 4 * h),
                               "l"(dsf + static_cast<uint32_t>(h * (kSfTile / 16) + g * (kSfGroup / 16))) : "memory");
#pragma unroll
              for (uint32_t q = 0; q < 4; ++q) {
                // 64 values, two blocks: the lower or the upper two of a word's bytes (bits 4 and 29)
                const uint32_t id = idesc + 2 * (q & 1) * ((1u << 4) | (1u << 29)), sfa = tsf + kSfHalf * (q >> 1);
                asm volatile("{\n .reg .pred p;\n setp.ne.b32 p, %6, 0;\n"
                             "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n}"
                             ::"r"(acc), "l"(da + 2 * q), "l"(db + 2 * q), "r"(id), "r"(sfa), "r"(sfa + 4),
                             "r"(static_cast<uint32_t>(kb != k0 || q != 0)) : "memory");
              }
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
    const int half = (warp - 2) / 4;   // which half of the columns is its own
    constexpr int kHalf = kBN / 2;
    const uint32_t own = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + half * kHalf;
    uint8_t* const stage = store + (warp - 2) * kStoreBytes;
    float* const bias_s = s_bias[warp - 2];
    constexpr int kCols = kT == kF32 ? 32 : 64;  // columns of one staged group: 128 bytes
    constexpr int kGroups = kHalf / kCols;
    int use = 0;
    bool ok = true;
    // Done with the accumulators' shared columns (the first one's last 64 and
    // the second one's first), or with all of its own.
    const auto done_shared = [&](int buf) {
      if (kBN != 256 || buf == half) return;
      asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
      __syncwarp();
      if (lane == 0) mbar_arrive_leader(&s_overlap);
    };
    const auto done_all = [&](int buf) {
      asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
      __syncwarp();
      if (lane == 0) mbar_arrive_leader(&s_acc_empty[buf]);
    };
    for (int t = first; ok && t < p.items; t += pairs) {
      const Item item = item_of<kBN>(p, t);
      const int m0 = item.m0 + static_cast<int>(rank) * (kBM / 2) + quarter * 32, n0 = item.n0 + half * kHalf;
      const int cols = item.cols - half * kHalf;  // of a half tile, some columns are not there
      float sum[kSum ? kHalf : 1];
      if constexpr (kSum) {
#pragma unroll
        for (int j = 0; j < kHalf; ++j) sum[j] = 0.0f;
        for (int k0 = 0; ok && k0 < p.stages; k0 += kChunk, ++use) {
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
          using C1 = std::integral_constant<int, 32>;
          using C2 = std::integral_constant<int, 64 % kHalf>;
          using C3 = std::integral_constant<int, 96 % kHalf>;
          if (kHalf == 128 && half != 0) {  // shared columns first
            add(C2{}); add(C3{}); done_shared(buf); add(C0{}); add(C1{});
          } else {
            add(C0{}); add(C1{}); done_shared(buf);
            if constexpr (kHalf == 128) { add(C2{}); add(C3{}); }
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
        const int gr = kSum || half == 0 ? i : kGroups - 1 - i;  // shared columns first
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
        if (p.store && lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
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
            tma_store(&p.out_map, n0 + col, m0, stage);
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
          const auto put_rows = [&](auto unit, int rows, int bytes) {
            using Unit = decltype(unit);
            constexpr int kBytes = sizeof(Unit);
#pragma unroll 16
            for (int at = lane * kBytes; at < rows * 128; at += 32 * kBytes) {
              const int r = at / 128, byte = at % 128;
              if (byte < bytes)
                *reinterpret_cast<Unit*>(dst + r * row_bytes + byte) =
                    *reinterpret_cast<const Unit*>(stage + r * 128 + (((byte >> 4) ^ (r & 7)) << 4) + (byte & 15));
            }
          };
          const int rows = p.m - m0 < 32 ? p.m - m0 : 32, bytes = (p.n - n0 - col < kCols ? p.n - n0 - col : kCols) * kEb;
          if (p.unit == 8) put_rows(uint2{}, rows, bytes);
          else if (kT == kF32 || p.unit == 4) put_rows(uint32_t{}, rows, bytes);
          else put_rows(uint16_t{}, rows, bytes);
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
// For few rows of A (tokens) the roles change: the 128 rows of the matrix
// instruction are rows of B (the weight's outputs) and its columns the few
// rows of A.  Such a product is bound by reading B once, and a cluster of
// `split` CTAs divides the summed axis, so that all SMs read.  Each CTA keeps
// its part's sums in its tensor memory; at the end CTA r gathers, from all of
// the cluster over distributed shared memory, the r-th share of the columns
// and adds the parts in the order of the ranks.  Products of more rows that
// have few tiles and a long sum are split here too, 128 rows to a tile.
//
// Up to kFuse rows, A may also come unquantized: the warps that store in the
// end then quantize each stage's 256 columns on the way into shared memory
// while the weight's copies are under way, which saves the quantizer's launch
// and its results' way through memory.  Every CTA of a rank quantizes the same
// part of A again, so this pays for few rows only (4096 x 4096, weight in L2: 1
// row 4.3 us, 8 rows 6.0 and 16 rows 8.6; 17 rows in two kernels 5.6, with some
// 4 more on the host).

constexpr int kFuse = 8;
constexpr int kFewest = 16;  // columns of its products
constexpr int kFewThreads = 320;  // warp 0 copies, warp 1 issues, warps 2 to 9 store
template <int kBN> __host__ __device__ constexpr int few_stages() { return kBN == 128 ? 3 : kBN >= 32 ? 4 : 5; }
template <int kBN> __host__ __device__ constexpr int few_stage_bytes() { return kTile * kStageBytes + kBN * kStageBytes; }
// Columns of sums that go to the CTA that gathers them in one store.
template <int kBN> __host__ __device__ constexpr int few_unit() { return kBN >= 32 ? 4 : 2; }
// Stages and their scales; the gathered parts, at most seven units more than
// kBN columns of 128 fp32 sums, take the stages' place.
template <int kBN> __host__ __device__ constexpr int few_smem() {
  static_assert((kBN + 7 * few_unit<kBN>()) * kTile * 4 <= few_stages<kBN>() * few_stage_bytes<kBN>(), "the parts fit the stages");
  return 1024 + few_stages<kBN>() * (few_stage_bytes<kBN>() + 2 * kSfTile);
}
// Two CTAs share an SM and its tensor memory: accumulators, and two sets of
// scales, of 16 columns each.
constexpr uint32_t kFewCols = kTmemCols / 2, kFewSfCol = kFewCols - 32;
template <int kBN> __host__ __device__ constexpr int few_accs() { return static_cast<int>(kFewSfCol) / kBN; }
constexpr int kMaxSplit = 8;  // CTAs of a portable cluster
// Longest row of A that the kernel quantizes for fp32 results: longer ones
// leave the accumulators of a cluster's CTAs more than kChunk stages each.
constexpr int64_t kFuseCols = int64_t{kMaxSplit} * few_accs<kFewest>() * kChunk * kStageK;

struct FewArgs {
  CUtensorMap map_w, map_x;  // rows of B in boxes of 128, of A in boxes of kBN
  const uint8_t* sfw;
  const uint8_t* sfx;
  const void* bias;
  void* out;
  int64_t ldo;
  int m, n, stages;      // rows of A (columns here), rows of B (rows here), stages of the summed axis
  int split;             // CTAs of a cluster, along the summed axis
  int tiles_n;           // tiles of 128 rows of B
  int b_ready;           // B is no result of the kernel ahead
  const void* x;         // A itself, `ldx` elements between rows of k, where the kernel quantizes it
  int64_t ldx;
  int k;
  int unit;              // its rows start on boundaries of so many bytes, and hold whole units
};

// Eight values of a row from column c on as they lie in memory, zeros past its end.
template <int kT>
__device__ __forceinline__ void few_load(const FewArgs& p, int line, int c, float (&v)[8]) {
  const char* const src = static_cast<const char*>(p.x) + (line * p.ldx + c) * elem_bytes<kT>();
  const int64_t left = line < p.m ? p.k - c : 0;
  if (p.unit == 16) load8<kT, uint4>(src, left, v);
  else if (p.unit == 8) load8<kT, uint2>(src, left, v);
  else if (kT == kF32 || p.unit == 4) load8<kT, uint32_t>(src, left, v);
  else if constexpr (kT != kF32) load8<kT, uint16_t>(src, left, v);
}

template <int kT, int kBN, bool kFused>
__global__ void __launch_bounds__(kFewThreads, 2)
fp4_matmul_few_kernel(const __grid_constant__ FewArgs p) {
  static_assert(!kFused || kBN == kFewest, "scales of up to 32 rows lie in one column");
  constexpr int kStages = few_stages<kBN>(), kW = kTile * kStageBytes, kStage = few_stage_bytes<kBN>(), kAccs = few_accs<kBN>();
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
  const int tile = static_cast<int>(blockIdx.x) / p.split, n0 = tile % p.tiles_n * kTile, m0 = kBN == 128 ? tile / p.tiles_n * kBN : 0;
  const int lines = p.m - m0 < kBN ? p.m - m0 : kBN;
  // this CTA's stages of the summed axis, and its accumulators' share of them
  const int kb0 = static_cast<int>(static_cast<int64_t>(p.stages) * rank / p.split);
  const int count = static_cast<int>(static_cast<int64_t>(p.stages) * (rank + 1) / p.split) - kb0;
  const int least = (count + kAccs - 1) / kAccs, chunk = least > kChunk ? least : kChunk;
  const int accs = (count + chunk - 1) / chunk;

  const auto weight = [&](int i, int s) {  // stage i of this CTA's, into stage s of the ring
    const int kb = kb0 + i;
    mbar_expect_tx(&s_full[s], kFused ? kW + kSfTile : kStage + 2 * kSfTile);
    tma_load_one(sm + s * kStage, &p.map_w, kb * kStageBytes, n0, &s_full[s]);
    bulk_load(sf + s * 2 * kSfTile, p.sfw + (static_cast<int64_t>(n0 / 128) * p.stages + kb) * kSfTile, kSfTile, &s_full[s]);
  };
  const int ahead = count < kStages ? count : kStages;
  if (warp == 0) {
    if (elect_one()) {
      s_fail = 0;
      for (int i = 0; i < kStages; ++i) { mbar_init(&s_full[i], kFused ? 1 + p.m : 1); mbar_init(&s_empty[i], 1); }
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
          tma_load_one(sm + ring.s * kStage + kW, &p.map_x, kb * kStageBytes, m0, &s_full[ring.s]);
          bulk_load(sf + ring.s * 2 * kSfTile + kSfTile, p.sfx + (static_cast<int64_t>(m0 / 128) * p.stages + kb) * kSfTile, kSfTile,
                    &s_full[ring.s]);
        }
      }
      __syncwarp();
    }
  } else if (warp == 1) {
    const bool one = elect_one();
    const uint32_t idesc = (1u << 7) | (1u << 10) | ((kBN / 8) << 17) | (1u << 23) | ((kTile / 128) << 27);
    const uint64_t dw0 = smem_desc(smem_u32(sm), 16, 1024, 2), dx0 = smem_desc(smem_u32(sm + kW), 16, 1024, 2);
    const uint64_t dsf0 = smem_desc(smem_u32(sf), 16, 128, 0);
    Ring<kStages> ring;
    uint32_t acc = tmem;
    int left = chunk;  // stages that this accumulator still takes
    for (int i = 0; i < count; ++i, ring.next()) {
      if (!mbar_wait(&s_full[ring.s], ring.phase, &s_fail)) break;
      asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
      if (one) {
        const uint64_t dw = dw0 + static_cast<uint32_t>(ring.s * (kStage / 16)), dx = dx0 + static_cast<uint32_t>(ring.s * (kStage / 16));
        const uint64_t d = dsf0 + static_cast<uint32_t>(ring.s * (2 * kSfTile / 16));
        // a set: the weight's two groups, A's two groups, four columns each
        const uint32_t tw = tmem + kFewSfCol + 16 * (i & 1);
#pragma unroll
        for (int h = 0; h < 4; ++h)
          asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(tw + 4 * h), "l"(d + static_cast<uint32_t>(h * (kSfGroup / 16))) : "memory");
#pragma unroll
        for (uint32_t q = 0; q < 4; ++q) {
          const uint32_t id = idesc + 2 * (q & 1) * ((1u << 4) | (1u << 29)), sfa = tw + 4 * (q >> 1);
          asm volatile("{\n .reg .pred p;\n setp.ne.b32 p, %6, 0;\n"
                       "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n}"
                       ::"r"(acc), "l"(dw + 2 * q), "l"(dx + 2 * q), "r"(id), "r"(sfa), "r"(sfa + 8),
                       "r"(static_cast<uint32_t>(left != chunk || q != 0)) : "memory");
        }
        commit_one(&s_empty[ring.s]);
      }
      __syncwarp();
      if (--left == 0) { left = chunk; acc += kBN; }
    }
    if (one) commit_one(&s_done);
  } else if constexpr (kFused) {
    // The eight warps take turns at units of a row of a stage, eight columns
    // to a lane, and have kAtOnce units' loads under way.  A unit's wait is for
    // the phase before its own, which cannot end before the unit does.
    wait_for_inputs();
    constexpr int kAtOnce = kT == kF32 ? 2 : 4;
    const int units = count * p.m;
    for (int u0 = warp - 2; u0 < units; u0 += kAtOnce * 8) {
      float v[kAtOnce][8];
#pragma unroll
      for (int h = 0; h < kAtOnce; ++h) {
        const int u = u0 + 8 * h, i = u / p.m, l = u - i * p.m;
        if (u < units) few_load<kT>(p, l, (kb0 + i) * kStageK + 8 * lane, v[h]);
      }
#pragma unroll
      for (int h = 0; h < kAtOnce; ++h) {
        const int u = u0 + 8 * h, i = u / p.m, l = u - i * p.m, s = i % kStages;
        if (u >= units) break;
        if (i >= kStages) mbar_wait(&s_empty[s], (i / kStages - 1) & 1, &s_fail);
        __syncwarp();
        uint32_t word;
        const uint32_t q = quantize8(v[h], lane, &word);
        // the 128-byte swizzle: 16-byte piece of row l at piece ^ (l mod 8)
        *reinterpret_cast<uint32_t*>(sm + s * kStage + kW + l * kStageBytes + (((lane >> 2) ^ (l & 7)) << 4) + (lane & 3) * 4) = q;
        if (lane % 16 == 0) *reinterpret_cast<uint32_t*>(sf + s * 2 * kSfTile + kSfTile + lane / 16 * kSfGroup + l * 16) = word;
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) mbar_arrive(&s_full[s]);
      }
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
fp4_fill_kernel(const void* __restrict__ bias, void* __restrict__ out, int64_t ldo, int64_t m, int64_t n) {
  const int64_t stride = static_cast<int64_t>(gridDim.x) * blockDim.x;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < m * n; i += stride)
    store1<kT>(out, i / n * ldo + i % n, bias ? load1<kT>(bias, i % n) : 0.0f);
}

// --------------------------------------------------------------------------
// host side

constexpr int64_t kMaxDim = int64_t{1} << 30;

bool valid_type(int t) { return t == BWD_F32 || t == BWD_BF16 || t == BWD_F16; }
int bytes_of(int t) { return t == BWD_F32 ? 4 : 2; }
int64_t tiles_of(int64_t n) { return (n + kTile - 1) / kTile; }
int64_t stages_of(int64_t k) { return (k + kStageK - 1) / kStageK; }

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

template <int kT>
cudaError_t opt_in_all() {
  const cudaError_t e[] = {opt_in(fp4_matmul_kernel<kT, 256, kT == kF32>, mm_smem<256>()), opt_in(fp4_matmul_kernel<kT, 128, kT == kF32>, mm_smem<128>()),
                           opt_in(fp4_matmul_few_kernel<kT, 16, false>, few_smem<16>()), opt_in(fp4_matmul_few_kernel<kT, 32, false>, few_smem<32>()),
                           opt_in(fp4_matmul_few_kernel<kT, 64, false>, few_smem<64>()), opt_in(fp4_matmul_few_kernel<kT, 128, false>, few_smem<128>()),
                           opt_in(fp4_matmul_few_kernel<kT, kFewest, true>, few_smem<kFewest>())};
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
  int smem = 0;
  e = cudaDeviceGetAttribute(&d.sms, cudaDevAttrMultiProcessorCount, dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&smem, cudaDevAttrMaxSharedMemoryPerMultiprocessor, dev);
  if (e != cudaSuccess) return cuda_fail(e, "cudaDeviceGetAttribute");
  if (e == cudaSuccess) e = opt_in_all<kF32>();
  if (e == cudaSuccess) e = opt_in_all<kBF16>();
  if (e == cudaSuccess) e = opt_in_all<kF16>();
  // so much shared memory that no SM takes two
  smem = smem / 2 > few_smem<128>() ? smem / 2 : few_smem<128>();
  if (e == cudaSuccess) e = opt_in(fp4_matmul_few_kernel<kBF16, 128, false>, smem);
  if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute(MaxDynamicSharedMemorySize)");
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cfg.blockDim = dim3(kThreads);
  cfg.gridDim = dim3(static_cast<unsigned>(d.sms / 2 * 2));
  cfg.dynamicSmemBytes = mm_smem<256>();
  attr[0].val.clusterDim = {2, 1, 1};
  e = cudaOccupancyMaxActiveClusters(&d.pairs, fp4_matmul_kernel<kBF16, 256, false>, &cfg);
  if (e != cudaSuccess) return cuda_fail(e, "cudaOccupancyMaxActiveClusters");
  if (d.pairs < 1) return fail(BWD_ERR_CUDA, "no room for a CTA pair of the matrix product");
  cfg.blockDim = dim3(kFewThreads);
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  d.clusters[1] = d.sms;
  for (int c = 2; c <= kMaxSplit; ++c) {
    cfg.gridDim = dim3(static_cast<unsigned>(d.sms / c * c));
    attr[0].val.clusterDim = {static_cast<unsigned>(c), 1, 1};
    e = cudaOccupancyMaxActiveClusters(&d.clusters[c], fp4_matmul_few_kernel<kBF16, 128, false>, &cfg);
    if (e != cudaSuccess) return cuda_fail(e, "cudaOccupancyMaxActiveClusters");
  }
  d.ctx = ctx;
  d.ready = true;
  return BWD_OK;
}

struct Operand {
  const uint8_t* codes;
  const uint8_t* scales;
  int64_t rows;
};

// out = A B^T + bias, k > 0.
struct Product {
  Operand a, b;
  int64_t k;
  const void* bias;
  void* out;
  int64_t ldo;
};

// The pitch's pad holds zero codes, and a map reaches over it: a box that ends
// inside 32 bytes is copied more slowly.
bwd_status code_map(CUtensorMap* map, const Operand& o, int64_t k, int box_rows) {
  return matrix_map(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, o.codes, o.rows, bwd_fp4_pitch(k), bwd_fp4_pitch(k), kStageBytes, box_rows,
                    CU_TENSOR_MAP_SWIZZLE_128B);
}
// One row for each tile of scales.
bwd_status scale_map(CUtensorMap* map, const Operand& o, int64_t k) {
  return matrix_map(map, CU_TENSOR_MAP_DATA_TYPE_UINT32, o.scales, tiles_of(o.rows) * stages_of(k), kSfTile / 4, kSfTile, kSfTile / 4, 1,
                    CU_TENSOR_MAP_SWIZZLE_NONE);
}

template <int kT, int kBN>
bwd_status launch_pairs(const MmArgs& p, int pairs, cudaStream_t st) {
  const dim3 grid(static_cast<unsigned>(2 * (p.items < pairs ? p.items : pairs)));
  return launch_ex(fp4_matmul_kernel<kT, kBN, kT == kF32>, grid, kThreads, 0, mm_smem<kBN>(), st, "fp4_matmul_kernel launch", p);
}

bwd_status by_pairs(const Product& q, bwd_dtype dtype, const DeviceState& d, cudaStream_t st) {
  const int eb = bytes_of(dtype);
  const int64_t m = q.a.rows, n = q.b.rows;
  const auto tiles_with = [&](int bn) { return (m + kBM - 1) / kBM * ((n + bn - 1) / bn); };
  const auto waves = [&](int bn) { return (tiles_with(bn) + d.pairs - 1) / d.pairs; };
  // a tile of 256 columns takes up to one and a half times as long as one of 128
  const int bn = 3 * waves(256) < 2 * waves(128) ? 256 : 128;
  const int64_t tiles = tiles_with(bn);
  if (tiles > 0x3fffffff || tiles_of(m) * stages_of(q.k) > 0x7fffffff || tiles_of(n) * stages_of(q.k) > 0x7fffffff)
    return fail(BWD_ERR_INVALID_ARG, "too many tiles");
  const int64_t last = tiles % d.pairs;
  const bool halves = bn == 256 && 2 * last <= d.pairs;
  MmArgs p{};
  p.bias = q.bias; p.out = q.out; p.ldo = q.ldo;
  p.m = static_cast<int>(m); p.n = static_cast<int>(n); p.stages = static_cast<int>(stages_of(q.k));
  p.tiles_n = static_cast<int>((n + bn - 1) / bn);
  p.whole = static_cast<int>(halves ? tiles - last : tiles);
  p.items = static_cast<int>(2 * tiles - p.whole);
  p.sf_rows_b = static_cast<int>(tiles_of(n));
  // A tensor store writes whole pieces of 16 bytes: where a row ends inside
  // one, the map covers whole groups of 128 bytes and the rest is stored
  // unit by unit.
  const int64_t mapped = n * eb % 16 == 0 ? n : n - n % (128 / eb);
  p.store = aligned16(q.out) && q.ldo * eb % 16 == 0 ? static_cast<int>(mapped) : 0;
  p.unit = unit_of(q.out, (q.ldo | n) * eb);
  bwd_status s;
  if ((s = code_map(&p.a, q.a, q.k, kBM / 2)) != BWD_OK) return s;
  if ((s = code_map(&p.b, q.b, q.k, bn / 2)) != BWD_OK) return s;
  if ((s = scale_map(&p.sfa, q.a, q.k)) != BWD_OK) return s;
  if ((s = scale_map(&p.sfb, q.b, q.k)) != BWD_OK) return s;
  if (p.store) {
    const CUtensorMapDataType type = dtype == BWD_F32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                     : dtype == BWD_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
    if ((s = matrix_map(&p.out_map, type, q.out, m, mapped, q.ldo * eb, 128 / eb, 32, CU_TENSOR_MAP_SWIZZLE_128B)) != BWD_OK) return s;
  }
  if (dtype == BWD_F32) return bn == 256 ? launch_pairs<kF32, 256>(p, d.pairs, st) : launch_pairs<kF32, 128>(p, d.pairs, st);
  if (dtype == BWD_BF16) return bn == 256 ? launch_pairs<kBF16, 256>(p, d.pairs, st) : launch_pairs<kBF16, 128>(p, d.pairs, st);
  return bn == 256 ? launch_pairs<kF16, 256>(p, d.pairs, st) : launch_pairs<kF16, 128>(p, d.pairs, st);
}

// Parts of the summed axis: as many as find an SM for each CTA.  Where up to
// 64 rows of A leave long parts, reading B takes the time, and two CTAs on an
// SM read faster.
int64_t few_split(int64_t tiles, int64_t stages, int64_t rows, const DeviceState& d) {
  const int64_t most = stages < kMaxSplit ? stages : kMaxSplit;
  int64_t split = most < 1 ? 1 : most;
  while (split > 1 && tiles > d.clusters[split]) --split;
  if (rows > 64 || (stages + split - 1) / split < 8) return split;
  const int64_t two = 2 * d.sms / tiles < most ? 2 * d.sms / tiles : most;
  return two > split ? two : split;
}

// A as it is, for the kernel that quantizes it.
struct Plain {
  const void* x;
  int64_t ld;
  int unit;
};

template <int kT, int kBN, bool kFused>
bwd_status launch_few(const Product& q, const Plain& plain, int b_ready, const DeviceState& d, cudaStream_t st) {
  FewArgs p{};
  bwd_status s;
  if ((s = code_map(&p.map_w, q.b, q.k, kTile)) != BWD_OK) return s;
  if (!kFused && (s = code_map(&p.map_x, q.a, q.k, kBN)) != BWD_OK) return s;
  p.x = plain.x; p.ldx = plain.ld; p.unit = plain.unit; p.k = static_cast<int>(q.k);
  p.sfw = q.b.scales; p.sfx = q.a.scales; p.bias = q.bias; p.out = q.out; p.ldo = q.ldo;
  p.m = static_cast<int>(q.a.rows); p.n = static_cast<int>(q.b.rows); p.stages = static_cast<int>(stages_of(q.k));
  const int64_t tiles = tiles_of(p.n) * ((p.m + kBN - 1) / kBN), part = few_accs<kBN>() * kChunk;
  const int64_t split = few_split(tiles, p.stages, p.m, d);
  // fp32 results: no accumulator may take more than kChunk stages
  p.split = static_cast<int>(kT == kF32 && split * part < p.stages ? (p.stages + part - 1) / part : split);
  p.tiles_n = static_cast<int>(tiles_of(p.n));
  p.b_ready = b_ready;
  return launch_ex(fp4_matmul_few_kernel<kT, kBN, kFused>, dim3(static_cast<unsigned>(tiles * p.split)), kFewThreads, p.split, few_smem<kBN>(), st,
                   "fp4_matmul_few_kernel launch", p);
}

template <int kT>
bwd_status few(const Product& q, const Plain& plain, int b_ready, const DeviceState& d, cudaStream_t st) {
  if (plain.x) return launch_few<kT, kFewest, true>(q, plain, b_ready, d, st);
  if (q.a.rows > 64) return launch_few<kT, 128, false>(q, plain, b_ready, d, st);
  if (q.a.rows > 32) return launch_few<kT, 64, false>(q, plain, b_ready, d, st);
  if (q.a.rows > 16) return launch_few<kT, 32, false>(q, plain, b_ready, d, st);
  return launch_few<kT, 16, false>(q, plain, b_ready, d, st);
}

bwd_status few(const Product& q, const Plain& plain, bwd_dtype dtype, int b_ready, const DeviceState& d, cudaStream_t st) {
  if (dtype == BWD_F32) return few<kF32>(q, plain, b_ready, d, st);
  return dtype == BWD_BF16 ? few<kBF16>(q, plain, b_ready, d, st) : few<kF16>(q, plain, b_ready, d, st);
}

// Whether a product goes to the kernel for few rows of A, or few tiles: for
// more than 64 rows where its parts' stages are much fewer than all of them.
bool use_few(const Product& q, bwd_dtype dtype, const DeviceState& d) {
  const int64_t stages = stages_of(q.k), tiles = tiles_of(q.b.rows) * tiles_of(q.a.rows);
  const int64_t split = few_split(tiles, stages, q.a.rows, d), part = (stages + split - 1) / split;
  // fp32 results: no accumulator may take more than kChunk stages, with as many parts as there can be
  const int64_t least = (stages + kMaxSplit - 1) / kMaxSplit;
  const int accs = q.a.rows > 64 ? few_accs<128>() : q.a.rows > 32 ? few_accs<64>() : q.a.rows > 16 ? few_accs<32>() : few_accs<16>();
  if (dtype == BWD_F32 && least > kChunk * accs) return false;
  return q.a.rows <= 64 || 3 * part + (2 * tiles * split <= d.sms ? 12 : 24) < 2 * stages;
}

// b_ready: a kernel that this call launched lies between whatever wrote B and
// this product.
bwd_status product(const Product& q, bwd_dtype dtype, int b_ready, cudaStream_t st) {
  const int64_t m = q.a.rows, n = q.b.rows;
  if (m == 0 || n == 0) return BWD_OK;
  if (q.k == 0) {
    const int64_t need = (m * n + 255) / 256;
    const unsigned grid = static_cast<unsigned>(need < 1216 ? need : 1216);
    if (dtype == BWD_F32) fp4_fill_kernel<kF32><<<grid, 256, 0, st>>>(q.bias, q.out, q.ldo, m, n);
    else if (dtype == BWD_BF16) fp4_fill_kernel<kBF16><<<grid, 256, 0, st>>>(q.bias, q.out, q.ldo, m, n);
    else fp4_fill_kernel<kF16><<<grid, 256, 0, st>>>(q.bias, q.out, q.ldo, m, n);
    return check_launch("fp4_fill_kernel launch");
  }
  const DeviceState* d = nullptr;
  const bwd_status s = ensure_device(&d);
  if (s != BWD_OK) return s;
  if (!use_few(q, dtype, *d)) return by_pairs(q, dtype, *d, st);
  return few(q, Plain{nullptr, 0, 0}, dtype, b_ready, *d, st);
}

bwd_status check_matrix(const void* x, bwd_dtype dtype, int64_t rows, int64_t cols, int64_t ld) {
  if (!valid_type(dtype)) return fail(BWD_ERR_UNSUPPORTED_DTYPE, "dtype %d", (int)dtype);
  if (rows < 0 || cols < 0 || rows > kMaxDim || cols > kMaxDim) return fail(BWD_ERR_INVALID_ARG, "bad size");
  if (rows > int64_t{65535} * kRows) return fail(BWD_ERR_INVALID_ARG, "more than 65535 * 32 rows");
  if (ld < cols) return fail(BWD_ERR_INVALID_ARG, "ld is less than cols");
  if (rows > 0 && cols > 0) {
    if (!x) return fail(BWD_ERR_INVALID_ARG, "NULL pointer");
    if (!aligned_to(x, bytes_of(dtype))) return fail(BWD_ERR_INVALID_ARG, "x is not aligned to its element size");
  }
  return BWD_OK;
}

// The largest of 16, 8, 4 and 2 bytes that divides an address and a row.
int unit16_of(const void* base, int64_t row_bytes) { return aligned16(base) && row_bytes % 16 == 0 ? 16 : unit_of(base, row_bytes); }

template <int kT>
bwd_status launch_quantize(const QuantArgs& a, cudaStream_t st) {
  const dim3 grid(static_cast<unsigned>(stages_of(a.cols)), static_cast<unsigned>((a.rows + kRows - 1) / kRows));
  const auto go = [&](auto unit) {
    return launch_ex(fp4_quantize_kernel<kT, decltype(unit)>, grid, 32 * kWarps, 0, 0, st, "fp4_quantize_kernel launch", a);
  };
  if (a.unit == 16) return go(uint4{});
  if (a.unit == 8) return go(uint2{});
  if constexpr (kT != kF32)
    if (a.unit == 2) return go(uint16_t{});
  return go(uint32_t{});
}

bwd_status quantize(const void* x, bwd_dtype dtype, int64_t rows, int64_t cols, int64_t ld, uint8_t* codes, uint8_t* scales, cudaStream_t st) {
  if (rows == 0 || cols == 0) return BWD_OK;
  const QuantArgs a{x, rows, cols, ld, bwd_fp4_pitch(cols), 2 * stages_of(cols), codes, scales, unit16_of(x, (ld | cols) * bytes_of(dtype))};
  if (dtype == BWD_F32) return launch_quantize<kF32>(a, st);
  return dtype == BWD_BF16 ? launch_quantize<kBF16>(a, st) : launch_quantize<kF16>(a, st);
}

template <int kT>
bwd_status launch_dequantize(const DequantArgs& a, int unit, cudaStream_t st) {
  const dim3 grid(static_cast<unsigned>(stages_of(a.cols)), static_cast<unsigned>((a.rows + kRows - 1) / kRows));
  const auto go = [&](auto u) {
    return launch_ex(fp4_dequantize_kernel<kT, decltype(u)>, grid, 32 * kWarps, 0, 0, st, "fp4_dequantize_kernel launch", a);
  };
  if (unit == 16) return go(uint4{});
  if (unit == 8) return go(uint2{});
  if constexpr (kT != kF32)
    if (unit == 2) return go(uint16_t{});
  return go(uint32_t{});
}

}  // namespace

namespace bwd {
namespace host {

bwd_status take_fp4_fault(unsigned int* fault) { return take_wait_fault(fault); }

}  // namespace host
}  // namespace bwd

extern "C" {

int64_t bwd_fp4_pitch(int64_t cols) {
  if (cols < 0 || cols > kMaxDim) return -1;
  // on 128-byte boundaries a stage's row of 128 bytes is one line of L2; rows
  // that would be padded to twice their length keep the 16 bytes that the
  // tensor maps need
  const int64_t bytes = (cols + 1) / 2;
  return bytes > 64 ? (bytes + 127) / 128 * 128 : (bytes + 15) / 16 * 16;
}

int64_t bwd_fp4_scale_bytes(int64_t rows, int64_t cols) {
  if (rows < 0 || cols < 0 || rows > kMaxDim || cols > kMaxDim) return -1;
  return tiles_of(rows) * stages_of(cols) * kSfTile;
}

bwd_status bwd_fp4_quantize(const void* x, bwd_dtype dtype, int64_t rows, int64_t cols, int64_t ld, uint8_t* codes, uint8_t* scales,
                            void* stream) {
  const bwd_status s = check_matrix(x, dtype, rows, cols, ld);
  if (s != BWD_OK) return s;
  if (rows == 0 || cols == 0) return BWD_OK;
  if (!codes || !scales) return fail(BWD_ERR_INVALID_ARG, "NULL pointer");
  if (!aligned16(codes) || !aligned16(scales)) return fail(BWD_ERR_INVALID_ARG, "codes and scales must be 16-byte aligned");
  return quantize(x, dtype, rows, cols, ld, codes, scales, static_cast<cudaStream_t>(stream));
}

bwd_status bwd_fp4_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t cols, void* out, bwd_dtype dtype,
                              void* stream) {
  const bwd_status s = check_matrix(out, dtype, rows, cols, cols);
  if (s != BWD_OK) return s;
  if (rows == 0 || cols == 0) return BWD_OK;
  if (!codes || !scales) return fail(BWD_ERR_INVALID_ARG, "NULL pointer");
  if (!aligned16(codes) || !aligned16(scales)) return fail(BWD_ERR_INVALID_ARG, "codes and scales must be 16-byte aligned");
  const DequantArgs a{codes, scales, rows, cols, bwd_fp4_pitch(cols), 2 * stages_of(cols), out};
  const int unit = unit16_of(out, cols * bytes_of(dtype));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (dtype == BWD_F32) return launch_dequantize<kF32>(a, unit, st);
  return dtype == BWD_BF16 ? launch_dequantize<kBF16>(a, unit, st) : launch_dequantize<kF16>(a, unit, st);
}

bwd_status bwd_fp4_matmul(int64_t m, int64_t n, int64_t k, const uint8_t* a, const uint8_t* a_scales, const uint8_t* b,
                          const uint8_t* b_scales, const void* bias, void* out, int64_t ldo, bwd_dtype dtype, void* stream) {
  if (!valid_type(dtype)) return fail(BWD_ERR_UNSUPPORTED_DTYPE, "dtype %d", (int)dtype);
  if (m < 0 || n < 0 || k < 0 || m > kMaxDim || n > kMaxDim || k > kMaxDim) return fail(BWD_ERR_INVALID_ARG, "bad size");
  if (ldo < n) return fail(BWD_ERR_INVALID_ARG, "ldo is less than n");
  if (m == 0 || n == 0) return BWD_OK;
  const int eb = bytes_of(dtype);
  if (!out || (k > 0 && (!a || !b || !a_scales || !b_scales))) return fail(BWD_ERR_INVALID_ARG, "NULL pointer");
  if (!aligned_to(out, eb) || !aligned_to(bias, eb)) return fail(BWD_ERR_INVALID_ARG, "out and bias must be aligned to their element size");
  if (k > 0 && (!aligned16(a) || !aligned16(b) || !aligned16(a_scales) || !aligned16(b_scales)))
    return fail(BWD_ERR_INVALID_ARG, "codes and scales must be 16-byte aligned");
  return product(Product{Operand{a, a_scales, m}, Operand{b, b_scales, n}, k, bias, out, ldo}, dtype, 0, static_cast<cudaStream_t>(stream));
}

int64_t bwd_fp4_linear_work_bytes(int64_t rows, int64_t cols) {
  if (rows < 0 || cols < 0 || rows > kMaxDim || cols > kMaxDim) return -1;
  if (rows <= kFuse && cols <= kFuseCols) return 0;
  Pieces w{nullptr};
  w.take(rows * bwd_fp4_pitch(cols));
  w.take(bwd_fp4_scale_bytes(rows, cols));
  return w.used;
}

bwd_status bwd_fp4_linear(const void* x, bwd_dtype dtype, int64_t rows, int64_t cols, int64_t ld, const uint8_t* w, const uint8_t* w_scales,
                          int64_t n, const void* bias, void* y, int64_t ldy, void* work, void* stream) {
  bwd_status s = check_matrix(x, dtype, rows, cols, ld);
  if (s != BWD_OK) return s;
  if (n < 0 || n > kMaxDim) return fail(BWD_ERR_INVALID_ARG, "bad size");
  if (ldy < n) return fail(BWD_ERR_INVALID_ARG, "ldy is less than n");
  if (rows == 0 || n == 0) return BWD_OK;
  const int eb = bytes_of(dtype);
  const bool fused = rows <= kFuse && (dtype != BWD_F32 || cols <= kFuseCols);
  if (!y || (cols > 0 && (!w || !w_scales || (!fused && !work)))) return fail(BWD_ERR_INVALID_ARG, "NULL pointer");
  if (!aligned_to(y, eb) || !aligned_to(bias, eb)) return fail(BWD_ERR_INVALID_ARG, "y and bias must be aligned to their element size");
  if (!aligned16(w) || !aligned16(w_scales) || !aligned16(work)) return fail(BWD_ERR_INVALID_ARG, "codes, scales and work must be 16-byte aligned");
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (fused && cols > 0) {
    const DeviceState* d = nullptr;
    if ((s = ensure_device(&d)) != BWD_OK) return s;
    return few(Product{Operand{nullptr, nullptr, rows}, Operand{w, w_scales, n}, cols, bias, y, ldy}, Plain{x, ld, unit16_of(x, (ld | cols) * eb)},
               dtype, 0, *d, st);
  }
  Pieces pieces{static_cast<uint8_t*>(work)};
  uint8_t* const codes = pieces.take(rows * bwd_fp4_pitch(cols));
  uint8_t* const scales = pieces.take(bwd_fp4_scale_bytes(rows, cols));
  s = quantize(x, dtype, rows, cols, ld, codes, scales, st);
  if (s != BWD_OK) return s;
  return product(Product{Operand{codes, scales, rows}, Operand{w, w_scales, n}, cols, bias, y, ldy}, dtype, 1, st);
}

}  // extern "C"
