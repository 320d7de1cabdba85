// Orthogonalised updates by Newton-Schulz steps, and the optimizer step that
// takes them (sm_103a).
//
//   X = G / (|G| + 1e-7)             Frobenius norm; G^T where G is tall
//   five times:  A = X X^T;  B = b A + c A A;  X = a X + B X
//
// which moves every singular value of G towards 1 by the odd polynomial a s +
// b s^3 + c s^5.  The steps are matrix products.  A and A A are symmetric:
// tiles on and below the diagonal are computed and stored twice.
//
// Operands are pairs of fp16 matrices, the value's nearest fp16 and what that
// leaves, both times 2^14 (22 bits in all).  A product of two such pairs takes
// three matrix instructions into one fp32 accumulator, high x low, low x high
// and high x high.  One 16-bit operand does not do: a gradient has a few
// strong directions, the steps raise the weak ones by up to 3.4 each, and with
// them the strong ones' roundings (measured in simulation, error of the result
// relative to its norm for rank 8 plus noise of 1/140: bf16 operands 0.23,
// fp16 0.028, pairs 5e-6; fp32 arithmetic has 2e-5).  The last step takes pairs
// too, whatever the result's type: high parts alone would save two of its three
// passes, and leave a bf16 result 2.0e-3 off in place of the 1.66e-3 that its
// rounding leaves (1024 x 1024).
//
// The last steps of a wide matrix (m rows, n = 2 m to 16 m columns) stay among
// m x m matrices, all of them polynomials of A, so that they commute and their
// products are symmetric:
//
//   P = a I + B;  Q = P Q;  A = P A P        and in the end X = Q X
//
// A step takes four symmetric products, 4 m m m operations, in place of m m n
// + m m m + 2 m m n.  What it costs is precision: rounding A moves its small
// eigenvalues, squares of the singular values, which a step raises by 11.8 as
// it raises those by 3.4; see squared_steps for how many steps that leaves.
// Of a bf16 gradient times a power of two X has no low part: its product with
// itself then takes one pass, and that with Q two.
#include "tensor.cuh"

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstring>
#include <vector>

namespace {

constexpr float kA = 3.4445f, kB = -4.7750f, kC = 2.0315f, kEps = 1e-7f;
// Largest magnitude that is stored: eigenvalues of B reach -2.8 (singular
// values stay below 1.21), and 2.8 * 2^14 is below fp16's 65504.
constexpr float kScale = 16384.0f;

constexpr int kBatch = 64;      // matrices of one launch
constexpr int kGroups = 8;      // shapes of one launch
constexpr int kSlots = 512;     // partial sums of a matrix's norm at most
constexpr int kThreads = 256;

struct Matrices {
  const void* g[kBatch];
  float* mom[kBatch];
  void* out[kBatch];     // the result, or the parameter
  uint8_t tall[kBatch];  // rows > columns: the steps run on the transposed matrix
};

// --------------------------------------------------------------------------
// momentum, norm and the first pair of operands

// Matrices of one shape, in either orientation.
struct PrepareGroup {
  __half* planes;           // [matrix][high, low][m][pitch]
  int64_t size;             // elements of a matrix
  int64_t chunk;            // of one CTA of the first kernel
  int chunks;
  int m, n, pitch;          // of the wide form
  int split_cols;           // columns of one CTA of the second kernel, a multiple of 64
  int first;                // its first matrix
  int norm_start, split_start;  // its first CTA of either kernel
};

struct PrepareArgs {
  Matrices x;
  double* slots;            // [matrix][kSlots]
  float* scale;             // [matrix] of exact planes: X = scale planes / kScale; null: pairs
  const float* grad_scale;  // or null: 1
  float momentum;
  int nesterov;
  int groups;
  PrepareGroup g[kGroups];
};

__device__ __forceinline__ bool finite(float s) { return fabsf(s) <= 3.402823466e38f; }

// mom = mu mom + s g; the update u is s g + mu mom, or mom.

// Eight consecutive values.
template <int kT>
__device__ __forceinline__ void load8(const void* x, int64_t i, float (&v)[8]) {
  if constexpr (kT == kF32) {
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const float4 f = __ldcs(reinterpret_cast<const float4*>(static_cast<const float*>(x) + i) + q);
      v[4 * q] = f.x; v[4 * q + 1] = f.y; v[4 * q + 2] = f.z; v[4 * q + 3] = f.w;
    }
  } else {
    const uint4 w = __ldcs(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(x) + i));
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t h = j % 2 ? (&w.x)[j / 2] >> 16 : (&w.x)[j / 2] & 0xffffu;
      v[j] = kT == kBF16 ? __uint_as_float(h << 16) : __half2float(__ushort_as_half(static_cast<unsigned short>(h)));
    }
  }
}
__device__ __forceinline__ bool on16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// The update's values i .. i + 7, zeros from `end` on; with kStep the new
// momentum is formed and written, else it is read.
template <int kT, bool kMomentum, bool kStep>
__device__ __forceinline__ void update8(const PrepareArgs& a, const void* g, float* mom, float s, bool vec, int64_t i, int64_t end, float (&u)[8]) {
  float m[8] = {};
  const bool whole = vec && i + 8 <= end;
  if (whole) {
    load8<kT>(g, i, u);
    if constexpr (kMomentum) load8<kF32>(mom, i, m);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      u[j] = i + j < end ? load1<kT>(g, i + j) : 0.0f;
      if constexpr (kMomentum) m[j] = i + j < end ? mom[i + j] : 0.0f;
    }
  }
  if constexpr (kMomentum && kStep) {
#pragma unroll
    for (int j = 0; j < 8; ++j) m[j] = __fmaf_rn(a.momentum, m[j], __fmul_rn(s, u[j]));
    if (!finite(s)) {
      // nothing is written
    } else if (whole) {
      reinterpret_cast<float4*>(mom + i)[0] = make_float4(m[0], m[1], m[2], m[3]);
      reinterpret_cast<float4*>(mom + i)[1] = make_float4(m[4], m[5], m[6], m[7]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (i + j < end) mom[i + j] = m[j];
    }
  }
  if constexpr (kMomentum) {
#pragma unroll
    for (int j = 0; j < 8; ++j) u[j] = a.nesterov ? __fmaf_rn(a.momentum, m[j], __fmul_rn(s, u[j])) : m[j];
  }
}

// One chunk of one matrix: the new momentum, and the update's sum of squares
// into its slot.  A thread adds in fp32, with what each addition loses carried
// along, a warp in fp32, and only the warps in binary64, of which the device
// does few (with all of it in binary64 33.5M bf16 values took 34 us).  Eight
// values whose squares fp32 does not hold in full are squared in binary64.
template <int kT, bool kMomentum>
__global__ void __launch_bounds__(kThreads)
ns_norm_kernel(const __grid_constant__ PrepareArgs a) {
  __shared__ double s_red[kThreads / 32];
  wait_for_inputs();
  let_next_begin();
  int gi = 0;
  while (gi + 1 < a.groups && static_cast<int>(blockIdx.x) >= a.g[gi + 1].norm_start) ++gi;
  const PrepareGroup& p = a.g[gi];
  const int local = static_cast<int>(blockIdx.x) - p.norm_start, z = p.first + local / p.chunks, chunk = local % p.chunks;
  const void* const g = a.x.g[z];
  float* const mom = a.x.mom[z];
  const float s = kMomentum && a.grad_scale ? *a.grad_scale : 1.0f;
  const bool vec = on16(g) && on16(mom);
  float sum = 0.0f, lost = 0.0f;
  double wide = 0.0;
  const int64_t end = min(p.size, (chunk + 1) * p.chunk);
#pragma unroll 4
  for (int64_t i = chunk * p.chunk + 8 * threadIdx.x; i < end; i += 8 * kThreads) {
    float u[8];
    update8<kT, kMomentum, true>(a, g, mom, s, vec, i, end, u);
    float part = 0.0f;
    uint32_t any = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      any |= __float_as_uint(u[j]);
      part = __fmaf_rn(u[j], u[j], part);
    }
    if ((any & 0x7fffffffu) != 0 && !(part >= 0x1p-120f && part <= 0x1p100f)) {
#pragma unroll
      for (int j = 0; j < 8; ++j) wide = __fma_rn(static_cast<double>(u[j]), static_cast<double>(u[j]), wide);
    } else {
      const float next = __fsub_rn(part, lost), all = __fadd_rn(sum, next);
      lost = __fsub_rn(__fsub_rn(all, sum), next);
      sum = all;
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (__any_sync(0xffffffffu, wide != 0.0)) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) wide += __shfl_xor_sync(0xffffffffu, wide, o);
  }
  wide += static_cast<double>(sum);
  if (threadIdx.x % 32 == 0) s_red[threadIdx.x / 32] = wide;
  __syncthreads();
  if (threadIdx.x != 0) return;
  for (int w = 1; w < kThreads / 32; ++w) wide += s_red[w];
  a.slots[z * kSlots + chunk] = wide;
}

// Two values as packed pairs of high and low parts.
__device__ __forceinline__ void split2(float v0, float v1, uint32_t& high, uint32_t& low) {
  const __half2 h = __floats2half2_rn(v0, v1);
  const float2 f = __half22float2(h);
  const __half2 l = __floats2half2_rn(__fsub_rn(v0, f.x), __fsub_rn(v1, f.y));
  high = *reinterpret_cast<const uint32_t*>(&h);
  low = *reinterpret_cast<const uint32_t*>(&l);
}

// X's pair from the update, 64 rows and split_cols columns of the wide form to a CTA.
// Of a 16-bit gradient, whose bits fp16 holds, the high part alone with a
// power of two for its factor, and what is left of the factor as a.scale.
// A tall matrix goes through shared memory, 64 x 64 elements at a time, so
// that both sides' rows are contiguous.  Columns up to the pitch are written,
// as zeros.
constexpr int kSplitRows = 64;

template <int kT, bool kMomentum>
__global__ void __launch_bounds__(kThreads)
ns_split_kernel(const __grid_constant__ PrepareArgs a) {
  __shared__ float s_x[64][65];
  __shared__ float s_inv[2];
  wait_for_inputs();
  let_next_begin();
  int gi = 0;
  while (gi + 1 < a.groups && static_cast<int>(blockIdx.x) >= a.g[gi + 1].split_start) ++gi;
  const PrepareGroup& p = a.g[gi];
  const int strips = (p.pitch + p.split_cols - 1) / p.split_cols, per = strips * ((p.m + kSplitRows - 1) / kSplitRows);
  const int local = static_cast<int>(blockIdx.x) - p.split_start, in_group = local / per, tile = local % per, z = p.first + in_group;
  if (threadIdx.x < 32) {
    double sum = 0.0;
    for (int i = threadIdx.x; i < p.chunks; i += 32) sum += a.slots[z * kSlots + i];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    // the norm may pass fp32's range, and its reciprocal what fp32 holds in full
    const double norm = sqrt(sum) + static_cast<double>(kEps);
    const bool large = norm > 0x1p64;
    if (threadIdx.x == 0) {
      s_inv[0] = large ? 0x1p-64f : 1.0f;
      const float inv = static_cast<float>((large ? 0x1p64 : 1.0) * static_cast<double>(kScale) / norm);
      const float power = __uint_as_float(__float_as_uint(inv) & 0x7f800000u);
      s_inv[1] = a.scale ? power : inv;
      if (a.scale && tile == 0) a.scale[z] = __fdiv_rn(inv, power);
    }
  }
  __syncthreads();
  const float first = s_inv[0], inv = s_inv[1];
  const void* const g = a.x.g[z];
  float* const mom = a.x.mom[z];
  const float s = kMomentum && a.grad_scale ? *a.grad_scale : 1.0f;
  const bool tall = a.x.tall[z];
  const int cols = tall ? p.m : p.n;  // as stored
  const bool vec = on16(g) && on16(mom) && cols % 8 == 0;
  __half* const high = p.planes + static_cast<int64_t>(in_group) * 2 * p.m * p.pitch;
  __half* const low = high + static_cast<int64_t>(p.m) * p.pitch;
  const int r0 = tile / strips * kSplitRows;
  const auto put = [&](int row, int col, const float (&x)[8]) {
    if (row >= p.m || col >= p.pitch) return;
    uint4 h, l;
#pragma unroll
    for (int j = 0; j < 4; ++j) split2(x[2 * j], x[2 * j + 1], (&h.x)[j], (&l.x)[j]);
    const int64_t at = static_cast<int64_t>(row) * p.pitch + col;
    *reinterpret_cast<uint4*>(high + at) = h;
    if (!a.scale) *reinterpret_cast<uint4*>(low + at) = l;
  };
  for (int c0 = tile % strips * p.split_cols, c1 = c0 + p.split_cols; c0 < c1; c0 += 64) {
    const int sr0 = tall ? c0 : r0, sc0 = tall ? r0 : c0, rows = tall ? p.n : p.m;
#pragma unroll
    for (int e = threadIdx.x; e < 64 * 8; e += kThreads) {
      const int r = e / 8, c = e % 8 * 8;
      float x[8] = {};
      if (sr0 + r < rows && sc0 + c < cols) {
        const int64_t at = static_cast<int64_t>(sr0 + r) * cols;
        update8<kT, kMomentum, false>(a, g, mom, s, vec, at + sc0 + c, at + cols, x);
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = __fmul_rn(__fmul_rn(x[j], first), inv);
      }
      if (tall) {
#pragma unroll
        for (int j = 0; j < 8; ++j) s_x[c + j][r] = x[j];
      } else {
        put(r0 + r, c0 + c, x);
      }
    }
    if (!tall) continue;
    __syncthreads();
#pragma unroll
    for (int e = threadIdx.x; e < 64 * 8; e += kThreads) {
      const int r = e / 8, c = e % 8 * 8;
      float x[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = s_x[r][c + j];
      put(r0 + r, c0 + c, x);
    }
    __syncthreads();
  }
}

// --------------------------------------------------------------------------
// the products
//
// A pair of CTAs (a cluster of two) works on a tile of 256 rows and kBN
// columns; pairs walk the tiles of all matrices with a grid stride.  Warp 0
// copies, warp 1 of the first CTA issues for both, and sixteen warps store the
// tile before from the other accumulator: each 32 rows of a quarter of the
// columns, whose sums its registers hold, 32 columns at a time through 4 KB of
// its own.  There the matrix that is added arrives by a tensor copy and the
// result replaces it, high and low parts in rows of 64 bytes.
constexpr int kBM = 256;
constexpr int kBK = 64;  // fp16 values of the summed axis in a stage: 128 bytes
constexpr int kStoreWarps = 16;
constexpr int kStoreWarp = 2;  // the first of them
constexpr int kMmThreads = 32 * (kStoreWarp + kStoreWarps);
constexpr uint32_t kTmemCols = 512;
constexpr int kPlaneBytes = 32 * 64;  // of a warp's 32 x 32 values, one plane

template <int kBN> __host__ __device__ constexpr int ns_stages() { return kBN == 256 ? 5 : 6; }
constexpr int kABytes = kBM / 2 * kBK * 2;
template <int kBN> __host__ __device__ constexpr int ns_b_bytes() { return kBN / 2 * kBK * 2; }
template <int kBN> __host__ __device__ constexpr int ns_smem() {
  return 1024 + ns_stages<kBN>() * (kABytes + ns_b_bytes<kBN>()) + kStoreWarps * 2 * kPlaneBytes;
}

enum Mode { kGram, kPoly, kApply, kFinal };

struct ProductArgs {
  CUtensorMap p, q;      // planes of the two operands
  CUtensorMap add, out;  // planes that alpha multiplies, and the result's, in boxes of 32 x 32
  const __half* add_at;  // the same planes' addresses; null: nothing is added
  __half* out_at;
  int m, n, pitch;       // the result's
  int kblocks;
  int passes;            // 3; 2: q's high part alone; 1: the high parts alone
  int tiles_m, tiles_n, tiles, items;
  int whole;             // the first items; the others are halves of a tile
  float alpha, beta;     // result = alpha add + beta product
  const float* scale;    // [matrix] of exact planes, or null; a factor of beta, its square for A
  const float* diagonal; // [matrix][m] of p, which has zeros there, or null: in place of alpha, times beta
};

// beta of one matrix.
template <int kMode>
__device__ __forceinline__ float beta_of(const ProductArgs& a, int z) {
  if ((kMode != kGram && kMode != kFinal) || !a.scale) return a.beta;
  const float s = a.scale[z];
  return __fmul_rn(a.beta, kMode == kGram ? __fmul_rn(s, s) : s);
}

struct FinalArgs {
  Matrices x;
  const float* grad_scale;  // or null: 1
  float decay;              // of the parameter
  float step[kGroups];      // of the update
  int first[kGroups];       // a group's first matrix
};

__device__ __forceinline__ void tma_load3(void* dst, const CUtensorMap* map, int x, int y, int z, uint32_t bar) {
  asm volatile("cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];"
               ::"r"(smem_u32(dst)), "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar) : "memory");
}

// 16 columns of this warp's 32 lanes.
__device__ __forceinline__ void tmem_load16(uint32_t addr, float (&r)[16]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
               : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7]),
                 "=f"(r[8]), "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]), "=f"(r[14]), "=f"(r[15])
               : "r"(addr));
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ void tma_load3_one(void* dst, const CUtensorMap* map, int x, int y, int z, uint64_t* bar) {
  asm volatile("cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];"
               ::"r"(smem_u32(dst)), "l"(map), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void tma_store3(const CUtensorMap* map, int x, int y, int z, const void* src) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3}], [%4];"
               ::"l"(map), "r"(x), "r"(y), "r"(z), "r"(smem_u32(src)) : "memory");
}

__device__ __forceinline__ uint4 shared_load16(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
  return v;
}
__device__ __forceinline__ void shared_store16(uint32_t at, const uint4& v) {
  asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(at), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
__device__ __forceinline__ void shared_store2(uint32_t at, uint32_t v) {
  asm volatile("st.shared.u16 [%0], %1;" ::"r"(at), "h"(static_cast<uint16_t>(v)) : "memory");
}

struct Tile {
  int z, m0, n0;
  bool mirror;  // also stored transposed
};
// Symmetric results: the tiles that reach the diagonal or lie below it, row
// by row, kRows / kCols more in each row of tiles than in the one before.
template <int kRows, int kCols, bool kSymmetric>
__device__ __forceinline__ Tile tile_of(const ProductArgs& a, int item) {
  const int z = item / a.tiles, t = item - z * a.tiles;
  if constexpr (!kSymmetric) {
    // eight rows of tiles at a time, down their columns: what the device works
    // on together has few rows and columns
    constexpr int kTogether = 8;
    const int strip = t / (kTogether * a.tiles_n), i0 = strip * kTogether, in = a.tiles_m - i0 < kTogether ? a.tiles_m - i0 : kTogether;
    const int u = t - i0 * a.tiles_n;
    return Tile{z, (i0 + u % in) * kRows, u / in * kCols, false};
  }
  constexpr int kPer = kRows / kCols;
  // rows of tiles before row i hold kPer i (i + 1) / 2
  int i = static_cast<int>((sqrtf(8.0f * (t / kPer) + 1.0f) - 1.0f) * 0.5f);
  while (kPer * (i + 1) * (i + 2) / 2 <= t) ++i;
  while (kPer * i * (i + 1) / 2 > t) --i;
  const int j = t - kPer * i * (i + 1) / 2;
  return Tile{z, i * kRows, j * kCols, j < kPer * i};
}

__device__ __forceinline__ float half_at(const uint4& w, int j) {
  const uint32_t q = (&w.x)[j / 2];
  return __half2float(__ushort_as_half(static_cast<unsigned short>(j % 2 ? q >> 16 : q & 0xffffu)));
}

// The matrix instruction adds into its fp32 accumulator with truncation, an
// error with a sign, which A's diagonal shows in full.  So sums leave it every
// kChunk stages of high x high, 128 products, and are added up in registers,
// rounded to nearest; what low parts add is 2^-11 of that and stays for all of
// their products.  (1000 x 1000, fp32: error 1.0e-6, 1.6 times as much with 256 products;
// 24 matrices of 1024 x 1024 and 48 of 1024 x 4096 1.7% slower than with 256.)
constexpr int kChunk = 2;

// Stages of a tile whose sums leave the accumulator together, from stage k on.
__device__ __forceinline__ int chunk_end(const ProductArgs& a, int k) {
  const int all = a.passes * a.kblocks, small = all - a.kblocks;
  if (k < small) return small;
  return k + kChunk < all ? k + kChunk : all;
}

// alpha of one row.
template <int kMode>
__device__ __forceinline__ float alpha_of(const ProductArgs& a, int z, int row) {
  if (kMode != kFinal || !a.diagonal) return a.alpha;
  return row < a.m ? __fmul_rn(a.beta, a.diagonal[static_cast<int64_t>(z) * a.m + row]) : 0.0f;
}

// What a pair works on: a tile, or half of its columns.  A last wave that less
// than half fills the device is cut into halves, which take half as long.
template <int kBN, bool kSymmetric>
__device__ __forceinline__ Tile item_of(const ProductArgs& a, int i, int* cols) {
  *cols = kBN;
  if (kBN == 128 || i < a.whole) return tile_of<kBM, kBN, kSymmetric>(a, i);
  Tile t = tile_of<kBM, kBN, kSymmetric>(a, a.whole + (i - a.whole) / 2);
  t.n0 += (i - a.whole) % 2 * 128;
  *cols = 128;
  return t;
}

// kT and kUpdate: of the last product, whose result has type kT, or updates a
// parameter of that type.
template <int kBN, int kMode, int kT, bool kUpdate>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kMmThreads, 1)
ns_product_kernel(const __grid_constant__ ProductArgs a, const __grid_constant__ std::conditional_t<kMode == kFinal, FinalArgs, int> f) {
  constexpr bool kSymmetric = kMode == kGram || kMode == kPoly, kAdd = kMode != kGram;
  constexpr bool kTrans = kMode == kApply || kMode == kFinal;  // q's summed axis is its rows
  constexpr int kStages = ns_stages<kBN>(), kB_ = ns_b_bytes<kBN>(), kStage = kABytes + kB_;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* const sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  __shared__ __align__(8) uint64_t s_full[kStages], s_empty[kStages], s_acc_full[2], s_acc_empty[2], s_add[kStoreWarps];
  __shared__ uint32_t s_tmem;
  __shared__ int s_fail;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  uint32_t rank;
  asm("mov.u32 %0, %cluster_ctarank;" : "=r"(rank));
  if (threadIdx.x == 0) {
    prefetch_map(&a.p);
    prefetch_map(&a.q);
    s_fail = 0;
    for (int i = 0; i < kStages; ++i) { mbar_init(&s_full[i], 1); mbar_init(&s_empty[i], 1); }
    for (int i = 0; i < 2; ++i) { mbar_init(&s_acc_full[i], 1); mbar_init(&s_acc_empty[i], 2 * kStoreWarps); }
    for (int i = 0; i < kStoreWarps; ++i) mbar_init(&s_add[i], 1);
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
    for (int t = first; ok && t < a.items; t += pairs) {
      int cols;
      const Tile tile = item_of<kBN, kSymmetric>(a, t, &cols);
      // of a half, the copies of Q bring as many lines as of a whole
      const int m0 = tile.m0 + static_cast<int>(rank) * (kBM / 2), n0 = tile.n0 + static_cast<int>(rank) * (cols / 2);
      for (int pass = 3 - a.passes; ok && pass < 3; ++pass) {
        const int zp = 2 * tile.z + (pass == 1), zq = 2 * tile.z + (pass == 0);
        for (int kb = 0; kb < a.kblocks; ++kb, ring.next()) {
          if (!(ok = mbar_wait(&s_empty[ring.s], ring.phase ^ 1u, &s_fail))) break;
          if (one) {
            const uint32_t bar = leader_addr(&s_full[ring.s]);
            if (rank == 0) mbar_expect_tx(&s_full[ring.s], 2 * kStage);
            uint8_t* const p = sm + ring.s * kStage;
            uint8_t* const q = p + kABytes;
            tma_load3(p, &a.p, kb * kBK, m0, zp, bar);
            if constexpr (!kTrans) {
              tma_load3(q, &a.q, kb * kBK, n0, zq, bar);
            } else {
#pragma unroll
              for (int h = 0; h < kBN / 128; ++h) tma_load3(q + h * (kBK * 128), &a.q, n0 + 64 * h, kb * kBK, zq, bar);
            }
          }
          __syncwarp();
        }
      }
    }
  } else if (warp == 1) {
    if (rank == 0) {
      const bool one = elect_one();
      // f16 x f16, fp32 accumulators; bit 16: q's lines are contiguous
      const uint32_t idesc_of = (1u << 4) | (kTrans ? 1u << 16 : 0u) | ((kBM / 16) << 24);
      const uint64_t dp0 = smem_desc(smem_u32(sm), 16, 1024, 2);
      const uint64_t dq0 = kTrans ? smem_desc(smem_u32(sm + kABytes), kBK * 128, 1024, 2) : smem_desc(smem_u32(sm + kABytes), 16, 1024, 2);
      constexpr uint32_t kStepP = 32 / 16, kStepQ = kTrans ? 2048 / 16 : 32 / 16;  // 16 of the summed axis
      Ring<kStages> ring;
      int use = 0;
      bool ok = true;
      const int blocks = a.passes * a.kblocks;
      for (int t = first; ok && t < a.items; t += pairs) {
        const uint32_t idesc = idesc_of | ((kBN == 128 || t < a.whole ? kBN / 8 : 128 / 8) << 17);
        for (int k0 = 0, k1; ok && k0 < blocks; k0 = k1, ++use) {
          k1 = chunk_end(a, k0);
          const int buf = use & 1;
          ok = mbar_wait(&s_acc_empty[buf], ((use >> 1) & 1) ^ 1, &s_fail);
          asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
          const uint32_t acc = tmem + buf * 256;
          for (int kb = k0; ok && kb < k1; ++kb, ring.next()) {
            if (!(ok = mbar_wait(&s_full[ring.s], ring.phase, &s_fail))) break;
            asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
            if (one) {
              const uint64_t dp = dp0 + static_cast<uint32_t>(ring.s * (kStage / 16)), dq = dq0 + static_cast<uint32_t>(ring.s * (kStage / 16));
#pragma unroll
              for (uint32_t q = 0; q < 4; ++q)
                asm volatile("{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
                             "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}"
                             ::"r"(acc), "l"(dp + q * kStepP), "l"(dq + q * kStepQ), "r"(idesc),
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
    wait_for_inputs();
    const int w = warp - kStoreWarp, quarter = warp & 3;
    constexpr int kOwn = kBN / 4, kGroups = kOwn / 32;  // columns of one warp
    const int own_col = w / 4 * kOwn;
    uint8_t* const buf = sm + kStages * kStage + w * 2 * kPlaneBytes;
    const uint32_t own = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + own_col;
    int use = 0;
    uint32_t adds = 0;  // parity of the next tensor copy
    const bool adds_some = kAdd && (kMode != kFinal || a.add_at);
    bool ok = true, writes = true;
    if constexpr (kMode == kFinal && kUpdate) writes = finite(f.grad_scale ? *f.grad_scale : 1.0f);
    const int blocks = a.passes * a.kblocks;
    const auto wait_full = [&] {
      ok = __all_sync(0xffffffffu, mbar_wait(&s_acc_full[use & 1], (use >> 1) & 1, &s_fail));
      asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
      return ok;
    };
    const auto done = [&] {
      asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
      __syncwarp();
      if (lane == 0) mbar_arrive_leader(&s_acc_empty[use & 1]);
      ++use;
    };
    // 16-byte piece q of this lane's row; the tensor maps swizzle rows of 64 bytes
    const uint32_t buf_at = smem_u32(buf), my_row = buf_at + lane * 64, swizzle = ((lane >> 1) & 3) << 4;
    const auto store_planes = [&](int x, int y, int z) {
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) {
        tma_store3(&a.out, x, y, 2 * z, buf);
        tma_store3(&a.out, x, y, 2 * z + 1, buf + kPlaneBytes);
        asm volatile("cp.async.bulk.commit_group;" ::: "memory");
      }
    };
    const auto wait_stored = [&] {
      if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
      __syncwarp();
    };
    for (int t = first; ok && t < a.items; t += pairs) {
      int cols;
      const Tile tile = item_of<kBN, kSymmetric>(a, t, &cols);
      const int row0 = tile.m0 + static_cast<int>(rank) * (kBM / 2) + quarter * 32, row = row0 + lane, col0 = tile.n0 + own_col;
      // (what lies past the matrix is not there to copy or to store, but for a
      // mirrored tile's rows up to the pitch: their zeros are the pad's columns)
      const bool some = row0 < (kSymmetric && tile.mirror ? a.pitch : a.m) && own_col < cols;
      const auto fetch = [&](int col) {
        if (!adds_some || !some || col >= a.pitch) return;
        wait_stored();
        if (lane == 0) {
          mbar_expect_tx(&s_add[w], 2 * kPlaneBytes);
          tma_load3_one(buf, &a.add, col, row0, 2 * tile.z, &s_add[w]);
          tma_load3_one(buf + kPlaneBytes, &a.add, col, row0, 2 * tile.z + 1, &s_add[w]);
        }
      };
      fetch(col0);
      float sum[kOwn];
#pragma unroll
      for (int j = 0; j < kOwn; ++j) sum[j] = 0.0f;
#pragma unroll 1
      for (int k0 = 0; k0 < blocks; k0 = chunk_end(a, k0)) {
        if (!wait_full()) break;
#pragma unroll
        for (int c = 0; c < kOwn; c += 16) {
          float r[16];
          tmem_load16(own + (use & 1) * 256 + c, r);
#pragma unroll
          for (int j = 0; j < 16; ++j) sum[c + j] = __fadd_rn(sum[c + j], r[j]);
        }
        done();
      }
      if (!ok) break;
      const float beta = beta_of<kMode>(a, tile.z), alpha = alpha_of<kMode>(a, tile.z, row);
#pragma unroll
      for (int g = 0; g < kGroups; ++g) {
        const int col = col0 + 32 * g;
        if (g > 0) fetch(col);
        float v[32];
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] = sum[32 * g + j];
        if (!some || col >= a.pitch) continue;
        if (adds_some) {
          ok = __all_sync(0xffffffffu, mbar_wait(&s_add[w], adds, &s_fail));
          adds ^= 1u;
          if (!ok) break;
        } else {
          wait_stored();
        }
        uint32_t h[16], l[16];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          uint4 ch{}, cl{};
          if (adds_some) {
            ch = shared_load16(my_row + (swizzle ^ (q << 4)));
            cl = shared_load16(my_row + (swizzle ^ (q << 4)) + kPlaneBytes);
          }
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            float& x = v[8 * q + j];
            x = __fmul_rn(beta, x);
            if constexpr (kAdd) x = __fmaf_rn(alpha, __fadd_rn(half_at(ch, j), half_at(cl, j)), x);
          }
          if constexpr (kMode != kFinal) {
#pragma unroll
            for (int j = 0; j < 4; ++j) split2(v[8 * q + 2 * j], v[8 * q + 2 * j + 1], h[4 * q + j], l[4 * q + j]);
            shared_store16(my_row + (swizzle ^ (q << 4)), make_uint4(h[4 * q], h[4 * q + 1], h[4 * q + 2], h[4 * q + 3]));
            shared_store16(my_row + (swizzle ^ (q << 4)) + kPlaneBytes, make_uint4(l[4 * q], l[4 * q + 1], l[4 * q + 2], l[4 * q + 3]));
          }
        }
        if constexpr (kMode != kFinal) {
          if (row0 < a.m) store_planes(col, row0, tile.z);
          // Columns left of the diagonal's tiles are all rows of the matrix.
          if (kSymmetric && tile.mirror) {
            wait_stored();
            // column j becomes a row: this lane's 2 bytes in piece lane / 8 of it
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              const uint32_t to = buf_at + ((((lane >> 3) ^ x) << 4) | (lane & 7) * 2);
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                const int j = i / 2 * 8 + 2 * x + i % 2;
                shared_store2(to + j * 64, j % 2 ? h[j / 2] >> 16 : h[j / 2]);
                shared_store2(to + j * 64 + kPlaneBytes, j % 2 ? l[j / 2] >> 16 : l[j / 2]);
              }
            }
            store_planes(row0, col, tile.z);
          }
        } else {
          if (!writes) continue;
          // 32 values of a line of the result that are far apart, neighbouring
          // lanes' side by side; several old parameters are read before any of
          // them is written
          const int z = f.first[0] + tile.z;
          const bool tall = f.x.tall[z];
          float* const stage = reinterpret_cast<float*>(buf);
          __syncwarp();
          if (!tall) {
#pragma unroll
            for (int j = 0; j < 32; ++j) stage[lane * 32 + (j ^ lane)] = v[j];
          }
          __syncwarp();
          const int64_t ld = tall ? a.m : a.n;
          int64_t at = tall ? static_cast<int64_t>(col) * ld + row : static_cast<int64_t>(row0) * ld + col + lane;
          const int count = tall ? (row < a.m ? a.n - col : 0) : col + lane < a.n ? a.m - row0 : 0;
          void* const out = f.x.out[z];
#pragma unroll
          for (int j0 = 0; j0 < 32; j0 += 8, at += 8 * ld) {
            float o[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) o[j] = tall ? v[j0 + j] : stage[(j0 + j) * 32 + (lane ^ (j0 + j))];
            if constexpr (kUpdate) {
              float p[8];
#pragma unroll
              for (int j = 0; j < 8; ++j) p[j] = j0 + j < count ? load1<kT>(out, at + j * ld) : 0.0f;
#pragma unroll
              for (int j = 0; j < 8; ++j) o[j] = __fmaf_rn(-f.step[0], o[j], __fmul_rn(p[j], f.decay));
            }
#pragma unroll
            for (int j = 0; j < 8; ++j)
              if (j0 + j < count) store1<kT>(out, at + j * ld, o[j]);
          }
          // the next tensor copy writes where `stage` was written
          if (adds_some) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();
        }
      }
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
// the products of small matrices
//
// Where the tiles above are too few for the device, what takes the time is
// latency: launch, first copy, each stage in turn, the store.  Here a tile is
// 128 x 64, and a cluster of `split` CTAs divides the summed axis, so that a
// CTA has a stage or two.  A stage holds both parts of both operands, 48 KB,
// for twelve instructions.  The low parts' products and every kChunk stages of
// high x high, 128 products, have accumulators of their own, three of which
// take turns: where a CTA has more stages than they hold, its storing warps add
// up one while the next two fill.  (One 1408 x 16384, fp32, whose sums of 5,504
// products stayed in one accumulator: error 1.6e-5 of the result, 1.9e-6 so;
// 1408 x 5632, 1,920 products, 1.0e-5 and 3.2e-6.)  A thread adds its accumulators,
// sends each unit of 8 columns to the CTA that gathers it over distributed
// shared memory, and that one adds the cluster's parts in the order of the
// ranks.
constexpr int kSmallRows = 128, kSmallCols = 64, kSmallStages = 2;
constexpr int kSmallStoreWarps = 8;
constexpr int kSmallThreads = 32 * (2 + kSmallStoreWarps);  // warp 0 copies, warp 1 issues, the others add up and store
constexpr int kSmallP = kSmallRows * kBK * 2, kSmallQ = kSmallCols * kBK * 2, kSmallStage = 2 * (kSmallP + kSmallQ);
constexpr int kSmallSmem = 1024 + kSmallStages * kSmallStage;
// Two CTAs fit an SM and its tensor memory, so that the next product's begin
// while this one's still run.
constexpr uint32_t kSmallTmem = kTmemCols / 2;
constexpr int kSmallAccs = static_cast<int>(kSmallTmem) / kSmallCols - 1;  // of high x high
constexpr int kMaxSplit = 8;
constexpr int kUnit = 8, kUnits = kSmallCols / kUnit;  // columns that move together
static_assert((kUnits + kMaxSplit - 1) * kSmallRows * kUnit * 4 <= kSmallStages * kSmallStage, "the gathered parts take the stages' place");

// Products of up to kGroups shapes, one CTA cluster for each tile.
struct SmallCall {
  int groups, split;
  int start[kGroups];  // a group's first tile
  ProductArgs g[kGroups];
};

// Eight neighbouring columns of this thread's row, of both planes.
struct Pair8 {
  uint4 h, l;
};

// kLong: a CTA has more stages than the accumulators hold (without it, which
// takes fewer registers, 777 x 301 99 us, 108 with it).
template <int kMode, int kT, bool kUpdate, bool kLong>
__global__ void __launch_bounds__(kSmallThreads, 2)
ns_small_kernel(const __grid_constant__ SmallCall call, const __grid_constant__ std::conditional_t<kMode == kFinal, FinalArgs, int> f) {
  constexpr bool kSymmetric = kMode == kGram || kMode == kPoly, kAdd = kMode != kGram;
  constexpr bool kTrans = kMode == kApply || kMode == kFinal;  // q's summed axis is its rows
  extern __shared__ uint8_t smem_raw[];
  uint8_t* const sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  float* const parts = reinterpret_cast<float*>(sm);  // [rank][unit of the share][half][row][4], once the stages are done with
  __shared__ __align__(8) uint64_t s_full[kSmallStages], s_empty[kSmallStages], s_done, s_acc_full[kSmallAccs], s_acc_empty[kSmallAccs];
  __shared__ uint32_t s_tmem;
  __shared__ int s_fail;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  uint32_t rank;
  asm("mov.u32 %0, %cluster_ctarank;" : "=r"(rank));
  const int item = static_cast<int>(blockIdx.x) / call.split;
  int gi = 0;
  while (gi + 1 < call.groups && item >= call.start[gi + 1]) ++gi;
  const ProductArgs& a = call.g[gi];
  const Tile tile = tile_of<kSmallRows, kSmallCols, kSymmetric>(a, item - call.start[gi]);
  const int kb0 = a.kblocks * static_cast<int>(rank) / call.split, count = a.kblocks * (static_cast<int>(rank) + 1) / call.split - kb0;
  // sums of high x high that leave an accumulator; all but the last kSmallAccs of them while the products go on
  const int chunks = (count + kChunk - 1) / kChunk, early = kLong && chunks > kSmallAccs ? chunks - kSmallAccs : 0;
  const bool p_low = a.passes >= 2, q_low = a.passes == 3;
  if (threadIdx.x == 0) {
    prefetch_map(&a.p);
    prefetch_map(&a.q);
    s_fail = 0;
    for (int i = 0; i < kSmallStages; ++i) { mbar_init(&s_full[i], 1); mbar_init(&s_empty[i], 1); }
    mbar_init(&s_done, 1);
    for (int i = 0; kLong && i < kSmallAccs; ++i) { mbar_init(&s_acc_full[i], 1); mbar_init(&s_acc_empty[i], kSmallStoreWarps); }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&s_tmem)), "r"(kSmallTmem) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  __syncwarp();
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  const uint32_t tmem = s_tmem;
  wait_for_inputs();
  let_next_begin();

  const int quarter = warp & 3, half = (warp - 2) / 4, row = quarter * 32 + lane, r = tile.m0 + row;
  const uint32_t share = (kUnits + call.split - 1) / call.split;
  const int64_t plane = static_cast<int64_t>(a.m) * a.pitch;
  // this thread's units of its CTA's share: the half-th and every second from there
  constexpr int kMine = kUnits / 2;
  const auto unit_col = [&](uint32_t u) { return tile.n0 + static_cast<int>(rank * share + u) * kUnit; };
  const auto unit_in = [&](uint32_t u) { return u < share && rank * share + u < kUnits && r < a.m && unit_col(u) < a.pitch; };
  Pair8 add[kAdd ? kMine : 1];
  if (warp == 0) {
    const bool one = elect_one();
    Ring<kSmallStages> ring;
    for (int i = 0; i < count; ++i, ring.next()) {
      if (!mbar_wait(&s_empty[ring.s], ring.phase ^ 1u, &s_fail)) break;
      if (one) {
        const int k = (kb0 + i) * kBK;
        uint64_t* const bar = &s_full[ring.s];
        uint8_t* const p = sm + ring.s * kSmallStage;
        mbar_expect_tx(bar, (p_low ? 2 : 1) * kSmallP + (q_low ? 2 : 1) * kSmallQ);
        for (int h = 0; h < (p_low ? 2 : 1); ++h) {
          tma_load3_one(p + h * kSmallP, &a.p, k, tile.m0, 2 * tile.z + h, bar);
          if (h == 0 || q_low) tma_load3_one(p + 2 * kSmallP + h * kSmallQ, &a.q, kTrans ? tile.n0 : k, kTrans ? k : tile.n0, 2 * tile.z + h, bar);
        }
      }
      __syncwarp();
    }
  } else if (warp == 1) {
    const bool one = elect_one();
    const uint32_t idesc = (1u << 4) | (kTrans ? 1u << 16 : 0u) | ((kSmallCols / 8) << 17) | ((kSmallRows / 16) << 24);
    const uint64_t dp0 = smem_desc(smem_u32(sm), 16, 1024, 2), dq0 = smem_desc(smem_u32(sm + 2 * kSmallP), kTrans ? kBK * 128 : 16, 1024, 2);
    constexpr uint32_t kStepP = 32 / 16, kStepQ = kTrans ? 2048 / 16 : 32 / 16;
    Ring<kSmallStages> ring;
    Ring<kSmallAccs> acc;
    for (int i = 0; i < count; ++i, ring.next()) {
      if (kLong && i % kChunk == 0 && !mbar_wait(&s_acc_empty[acc.s], acc.phase ^ 1u, &s_fail)) break;
      if (!mbar_wait(&s_full[ring.s], ring.phase, &s_fail)) break;
      asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
      if (one) {
        const uint64_t dp = dp0 + static_cast<uint32_t>(ring.s * (kSmallStage / 16)), dq = dq0 + static_cast<uint32_t>(ring.s * (kSmallStage / 16));
        const auto issue = [&](uint32_t acc, uint64_t p, uint64_t q, bool fresh) {
#pragma unroll
          for (uint32_t s = 0; s < 4; ++s)
            asm volatile("{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
                         "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}"
                         ::"r"(acc), "l"(p + s * kStepP), "l"(q + s * kStepQ), "r"(idesc), "r"(static_cast<uint32_t>(!fresh || s != 0)) : "memory");
        };
        if (p_low) issue(tmem, dp + kSmallP / 16, dq, i == 0);
        if (q_low) issue(tmem, dp, dq + kSmallQ / 16, false);
        issue(tmem + kSmallCols * (1 + (kLong ? acc.s : i / kChunk)), dp, dq, i % kChunk == 0);
        commit_one(&s_empty[ring.s]);
        if (kLong && i % kChunk == kChunk - 1) commit_one(&s_acc_full[acc.s]);
      }
      __syncwarp();
      if (kLong && i % kChunk == kChunk - 1) acc.next();
    }
    if (one) commit_one(&s_done);
  } else if constexpr (kAdd) {
    // under way while the products are
#pragma unroll
    for (int i = 0; i < kMine; ++i) {
      const uint32_t u = 2 * i + half;
      if (!unit_in(u)) continue;
      if (kMode == kFinal && !a.add_at) {
        add[i] = Pair8{};
        continue;
      }
      const __half* const from = a.add_at + 2 * tile.z * plane + static_cast<int64_t>(r) * a.pitch + unit_col(u);
      // (not loads for constant data: the kernel ahead may have written these after this one began)
      add[i] = Pair8{*reinterpret_cast<const uint4*>(from), *reinterpret_cast<const uint4*>(from + plane)};
    }
  }
  __syncwarp();
  bool ok = true;
  const uint32_t own = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + 16 * half;
  const auto add_up = [&](float (&sum)[16], uint32_t column) {
    float v[16];
    tmem_load16(own + column, v);
#pragma unroll
    for (int j = 0; j < 16; ++j) sum[j] = __fadd_rn(sum[j], v[j]);
  };
  float sums[kLong ? kSmallCols / 32 : 1][16] = {};
  Ring<kSmallAccs> acc;
  if (warp >= 2) {
    if constexpr (kLong) {
#pragma unroll 1
      for (int i = 0; ok && i < early; ++i, acc.next()) {
        ok = __all_sync(0xffffffffu, mbar_wait(&s_acc_full[acc.s], acc.phase, &s_fail));
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
#pragma unroll
        for (int c = 0; c < kSmallCols; c += 32) add_up(sums[c / 32], (1 + acc.s) * kSmallCols + c);
        asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
        __syncwarp();
        if (lane == 0) mbar_arrive(&s_acc_empty[acc.s]);
      }
    }
    ok = __all_sync(0xffffffffu, ok && mbar_wait(&s_done, 0, &s_fail));
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  }
  if (s_fail && lane == 0 && warp < 2) let_copies_land();
  __syncwarp();
  cluster_sync();  // every CTA is done with its stages: the parts may take their place
  if (warp >= 2) {
#pragma unroll
    for (int c = 0; c < kSmallCols; c += 32) {
      const int c0 = c + 16 * half;  // the two halves' warps take turns at 16 columns
      float (&sum)[16] = sums[kLong ? c / 32 : 0];
      if constexpr (kLong) {
        if (p_low && count > 0) add_up(sum, c);
        Ring<kSmallAccs> from = acc;
        for (int i = early; i < chunks; ++i, from.next()) add_up(sum, (1 + from.s) * kSmallCols + c);
      } else {
#pragma unroll
        for (int j = 0; j < 16; ++j) sum[j] = 0.0f;
        for (int i = p_low ? 0 : 1; i <= chunks && count > 0; ++i) add_up(sum, i * kSmallCols + c);
      }
#pragma unroll
      for (int j = 0; j < 16; j += kUnit) {
        const uint32_t unit = (c0 + j) / kUnit, to = unit / share, at = ((rank * share + unit - to * share) * 2 * kSmallRows + row) * 4;
        uint32_t dst;
        asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(dst) : "r"(smem_u32(parts + at)), "r"(to));
#pragma unroll
        for (int q = 0; q < kUnit; q += 4)
          asm volatile("st.shared::cluster.v4.f32 [%0], {%1,%2,%3,%4};"
                       ::"r"(dst + 4 * q * kSmallRows), "f"(sum[j + q]), "f"(sum[j + q + 1]), "f"(sum[j + q + 2]), "f"(sum[j + q + 3]) : "memory");
      }
    }
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  }
  __syncwarp();
  cluster_sync();
  if (warp >= 2 && ok) {
    bool writes = true;
    if constexpr (kMode == kFinal && kUpdate) writes = finite(f.grad_scale ? *f.grad_scale : 1.0f);
    const float beta = beta_of<kMode>(a, tile.z), alpha = alpha_of<kMode>(a, tile.z, r);
#pragma unroll
    for (int i = 0; i < kMine; ++i) {
      const uint32_t u = 2 * i + half;
      // rows past the matrix hold zeros, which a mirrored tile's pad needs
      const bool pad = kSymmetric && tile.mirror && u < share && rank * share + u < kUnits && r >= a.m && r < a.pitch && unit_col(u) < a.pitch;
      if (!unit_in(u) && !pad) continue;
      const int col = unit_col(u);
      float v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = 0.0f;
      for (int q = 0; q < call.split; ++q) {
        const float4* const from = reinterpret_cast<const float4*>(parts) + (q * share + u) * 2 * kSmallRows + row;
        const float4 x = from[0], y = from[kSmallRows];
        v[0] = __fadd_rn(v[0], x.x); v[1] = __fadd_rn(v[1], x.y); v[2] = __fadd_rn(v[2], x.z); v[3] = __fadd_rn(v[3], x.w);
        v[4] = __fadd_rn(v[4], y.x); v[5] = __fadd_rn(v[5], y.y); v[6] = __fadd_rn(v[6], y.z); v[7] = __fadd_rn(v[7], y.w);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        v[j] = __fmul_rn(beta, v[j]);
        if constexpr (kAdd) v[j] = pad ? 0.0f : __fmaf_rn(alpha, __fadd_rn(half_at(add[i].h, j), half_at(add[i].l, j)), v[j]);
      }
      if constexpr (kMode != kFinal) {
        Pair8 o;
#pragma unroll
        for (int j = 0; j < 4; ++j) split2(v[2 * j], v[2 * j + 1], (&o.h.x)[j], (&o.l.x)[j]);
        __half* const base = a.out_at + 2 * tile.z * plane;
        if (!pad) {
          __half* const to = base + static_cast<int64_t>(r) * a.pitch + col;
          *reinterpret_cast<uint4*>(to) = o.h;
          *reinterpret_cast<uint4*>(to + plane) = o.l;
        }
        if (kSymmetric && tile.mirror && r < a.pitch) {
          uint16_t* to = reinterpret_cast<uint16_t*>(base) + static_cast<int64_t>(col) * a.pitch + r;
#pragma unroll
          for (int j = 0; j < 8; ++j, to += a.pitch) {
            to[0] = static_cast<uint16_t>(j % 2 ? (&o.h.x)[j / 2] >> 16 : (&o.h.x)[j / 2] & 0xffffu);
            to[plane] = static_cast<uint16_t>(j % 2 ? (&o.l.x)[j / 2] >> 16 : (&o.l.x)[j / 2] & 0xffffu);
          }
        }
      } else if (writes) {
        const int z = f.first[gi] + tile.z;
        const bool tall = f.x.tall[z];
        const int64_t at = tall ? static_cast<int64_t>(col) * a.m + r : static_cast<int64_t>(r) * a.n + col, step = tall ? a.m : 1;
        void* const out = f.x.out[z];
        if constexpr (kUpdate) {
          float p[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) p[j] = col + j < a.n ? load1<kT>(out, at + j * step) : 0.0f;
#pragma unroll
          for (int j = 0; j < 8; ++j) v[j] = __fmaf_rn(-f.step[gi], v[j], __fmul_rn(p[j], f.decay));
        }
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (col + j < a.n) store1<kT>(out, at + j * step, v[j]);
      }
    }
  }
  if (warp == 1) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kSmallTmem));
}

// Diagonals of `all` rows: P = a I + B, or (with `out`) taken out of Q, which
// has zeros there from then on.
__global__ void __launch_bounds__(kThreads)
ns_diagonal_kernel(__half* planes, int64_t m, int64_t pitch, int64_t all, float* out) {
  wait_for_inputs();
  let_next_begin();
  const int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  if (i >= all) return;
  __half* const high = planes + i / m * 2 * m * pitch + i % m * (pitch + 1);
  __half* const low = high + m * pitch;
  float x = __fadd_rn(__half2float(*high), __half2float(*low));
  if (out) {
    out[i] = x;
    x = 0.0f;
  } else {
    x = __fmaf_rn(kA, kScale, x);
  }
  uint32_t h, l;
  split2(x, 0.0f, h, l);
  *high = __ushort_as_half(static_cast<unsigned short>(h & 0xffffu));
  *low = __ushort_as_half(static_cast<unsigned short>(l & 0xffffu));
}

// --------------------------------------------------------------------------
// host side

bool valid_type(int t) { return t == BWD_F32 || t == BWD_BF16 || t == BWD_F16; }
uintptr_t bytes_of(int t) { return t == BWD_F32 ? 4 : 2; }
int64_t up(int64_t n, int64_t to) { return (n + to - 1) / to * to; }

constexpr int64_t kMaxSide = 65536;
constexpr int kMaxSteps = 100;
// Bytes of a batch of more than one matrix, where the caller names no other
// number.  (48 matrices of 1024 x 4096, 50 MB each, and 24 of 1024 x 1024: 9.45
// ms with 1 GB, 9.20 with 2, 8.88 with 4, of which they take 2.4.)
constexpr int64_t kWorkMost = int64_t{4} << 30;

struct Shape {
  int64_t m, n;
  int64_t x_bytes() const { return 4 * m * up(n, 64); }  // a pair of planes
  int64_t a_bytes() const { return 4 * m * up(m, 64); }
  bool wide() const { return n >= 2 * m && n <= 16 * m; }  // steps among the squares
  bool operator<(const Shape& o) const { return m != o.m ? m < o.m : n < o.n; }
};
Shape shape_of(int64_t rows, int64_t cols) { return rows > cols ? Shape{cols, rows} : Shape{rows, cols}; }

// Tiles of a product, of so many rows and columns each.
int64_t tiles_of(const Shape& result, int rows, int cols, bool symmetric) {
  const int64_t tm = (result.m + rows - 1) / rows;
  return symmetric ? rows / cols * tm * (tm + 1) / 2 : tm * ((result.n + cols - 1) / cols);
}

// Matrices that are worked on together: of up to kGroups shapes whose products
// have few tiles, or of one shape.
struct Group {
  Shape s;
  int64_t first, count;  // in the order of shapes
};
struct Set {
  Group g[kGroups];
  int groups;
  bool small;  // few tiles: all groups' products in one launch
  int64_t count() const { return g[groups - 1].first + g[groups - 1].count - g[0].first; }
  int64_t bytes() const {
    int64_t n = 0;
    for (int i = 0; i < groups; ++i) {
      const bool squares = !small && g[i].s.wide();
      n += 2 * up(g[i].s.x_bytes() * g[i].count, 256) + (squares ? 4 : 2) * up(g[i].s.a_bytes() * g[i].count, 256) +
           (squares ? up(4 * g[i].s.m * g[i].count, 256) + up(4 * g[i].count, 256) : 0);
    }
    return n + 8 * kSlots * count();
  }
};

constexpr int kMaxDevices = 64;
struct DeviceState {
  bool ready = false;
  unsigned long long ctx = 0;
  int pairs = 0;  // CTA pairs that are resident at a time
  int clusters[kMaxSplit + 1] = {};  // clusters of so many CTAs of the small products'
};
std::mutex g_mu;
DeviceState g_dev[kMaxDevices];

template <int kBN, int kMode, int kT, bool kUpdate>
constexpr auto kernel_of() { return ns_product_kernel<kBN, kMode, kT, kUpdate>; }

template <int kBN, int kMode, int kT, bool kUpdate>
cudaError_t opt_in_one() { return opt_in(kernel_of<kBN, kMode, kT, kUpdate>(), ns_smem<kBN>()); }

template <int kBN>
cudaError_t opt_in_all() {
  const cudaError_t e[] = {opt_in_one<kBN, kGram, kF32, false>(), opt_in_one<kBN, kPoly, kF32, false>(), opt_in_one<kBN, kApply, kF32, false>(),
                           opt_in_one<kBN, kFinal, kF32, false>(), opt_in_one<kBN, kFinal, kBF16, false>(), opt_in_one<kBN, kFinal, kF16, false>(),
                           opt_in_one<kBN, kFinal, kF32, true>(), opt_in_one<kBN, kFinal, kBF16, true>(), opt_in_one<kBN, kFinal, kF16, true>()};
  for (const cudaError_t x : e)
    if (x != cudaSuccess) return x;
  return cudaSuccess;
}

template <int kMode, int kT, bool kUpdate>
cudaError_t opt_in_small() {
  const cudaError_t e = opt_in(ns_small_kernel<kMode, kT, kUpdate, false>, kSmallSmem);
  return e == cudaSuccess ? opt_in(ns_small_kernel<kMode, kT, kUpdate, true>, kSmallSmem) : e;
}

cudaError_t opt_in_all_small() {
  const cudaError_t e[] = {opt_in_small<kGram, kF32, false>(), opt_in_small<kPoly, kF32, false>(), opt_in_small<kApply, kF32, false>(),
                           opt_in_small<kFinal, kF32, false>(), opt_in_small<kFinal, kBF16, false>(), opt_in_small<kFinal, kF16, false>(),
                           opt_in_small<kFinal, kF32, true>(), opt_in_small<kFinal, kBF16, true>(), opt_in_small<kFinal, kF16, true>()};
  for (const cudaError_t x : e)
    if (x != cudaSuccess) return x;
  return cudaSuccess;
}

bwd_status ensure_device(DeviceState* out) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
  if (dev < 0 || dev >= kMaxDevices) return fail(BWD_ERR_CUDA, "device ordinal %d unsupported", dev);
  unsigned long long ctx = 0;
  const bwd_status s = bwd::host::current_context_id(&ctx);
  if (s != BWD_OK) return s;
  std::lock_guard<std::mutex> lock(g_mu);
  DeviceState& d = g_dev[dev];
  if (!d.ready || d.ctx != ctx) {
    int sms = 0;
    e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e == cudaSuccess) e = opt_in_all<256>();
    if (e == cudaSuccess) e = opt_in_all<128>();
    if (e == cudaSuccess) e = opt_in_all_small();
    if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute(MaxDynamicSharedMemorySize)");
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(sms / 2 * 2));
    cfg.blockDim = dim3(kMmThreads);
    cfg.dynamicSmemBytes = ns_smem<256>();
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim = {2, 1, 1};
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaOccupancyMaxActiveClusters(&d.pairs, kernel_of<256, kApply, kF32, false>(), &cfg);
    if (e != cudaSuccess) return cuda_fail(e, "cudaOccupancyMaxActiveClusters");
    if (d.pairs < 1) return fail(BWD_ERR_CUDA, "no room for a CTA pair of the matrix product");
    // with so much shared memory that no SM takes two
    int smem = 0;
    e = cudaDeviceGetAttribute(&smem, cudaDevAttrMaxSharedMemoryPerMultiprocessor, dev);
    smem = std::max(smem / 2, kSmallSmem);
    if (e == cudaSuccess) e = opt_in(ns_small_kernel<kApply, kF32, false, false>, smem);
    if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute(MaxDynamicSharedMemorySize)");
    cfg.blockDim = dim3(kSmallThreads);
    cfg.dynamicSmemBytes = static_cast<size_t>(smem);
    d.clusters[1] = sms;
    for (int c = 2; c <= kMaxSplit; ++c) {
      cfg.gridDim = dim3(static_cast<unsigned>(sms / c * c));
      attr[0].val.clusterDim = {static_cast<unsigned>(c), 1, 1};
      e = cudaOccupancyMaxActiveClusters(&d.clusters[c], ns_small_kernel<kApply, kF32, false, false>, &cfg);
      if (e != cudaSuccess) return cuda_fail(e, "cudaOccupancyMaxActiveClusters");
    }
    d.ctx = ctx;
    d.ready = true;
  }
  *out = d;
  return BWD_OK;
}

// Map of `planes` planes of m rows and `pitch` columns.
bwd_status plane_map(CUtensorMap* map, const __half* base, int64_t m, int64_t pitch, int64_t planes, int box_cols, int box_rows) {
  const CUtensorMapSwizzle swizzle = box_cols == 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B;  // a box's whole row
  EncodeFn encode = nullptr;
  const bwd_status s = encode_fn(&encode);
  if (s != BWD_OK) return s;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(pitch), static_cast<cuuint64_t>(m), static_cast<cuuint64_t>(planes)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(pitch * 2), static_cast<cuuint64_t>(m * pitch * 2)};
  const cuuint32_t box[3] = {static_cast<cuuint32_t>(box_cols), static_cast<cuuint32_t>(box_rows), 1}, step[3] = {1, 1, 1};
  const CUresult r = encode(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<__half*>(base), dims, strides, box, step,
                            CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(BWD_ERR_CUDA, "cuTensorMapEncodeTiled: error %d", static_cast<int>(r));
  return BWD_OK;
}

struct Step {
  const float* grad_scale;
  float momentum, decay;
  double step;  // times the root of a matrix's longer side
  int nesterov, steps;
  bool has_momentum, update;
  bwd_dtype g_type, out_type;
  int64_t work_most;  // bytes of a batch of more than one matrix
};

// How many of the last steps work on the squares (see the top), at n = r m.  In
// passes of the matrix instruction, times m m m, a result takes 45 r + 15
// without them, 9 r + 51 with five (5 r + 51 from exact planes) and 27 r + 33
// with three.  An error of A in a weak direction is raised by 11.8 a step, so
// only bf16 results take five, which leave 3e-5 to 9e-5 of the result beside
// the rounding's 1.66e-3 (at most 4e-4 in simulation, whatever the spectrum);
// the direct steps, and three, leave 2e-6 to 2e-5.  Below two columns to a row
// that buys nothing or little: in ms, bf16, with five and without, 1600 x 2048
// 0.48 and 0.44, 1320 x 1650 0.37 and 0.39, 1100 x 2100 0.34 and 0.36; 2048 x
// 5632 0.65 and 1.01, 11008 x 4096 2.98 and 6.45 (three: 5.11).  Above sixteen
// a row of X is known far better than A, whose error the steps raise: fp32,
// error against 64 bits with three, without, and in fp32 arithmetic, 64 x 65536
// 1.2e-5, 1.7e-6 and 1.0e-6 (0.37 and 0.51 ms), 512 x 16384 3.7e-6, 0.9e-6 and
// 1.9e-6 (0.31 and 0.40 ms); 512 x 8192 3.6e-6, 0.8e-6 and 3.1e-6.
int squared_steps(const Shape& s, const Step& st) {
  return s.wide() ? std::min(st.steps, st.out_type == BWD_BF16 ? 5 : 3) : 0;
}

template <int kBN, int kMode>
bwd_status launch_product(const ProductArgs& a, const FinalArgs* f, const Step& st, int pairs, cudaStream_t stream) {
  const dim3 grid(static_cast<unsigned>(2 * (a.items < pairs ? a.items : pairs)));
  const auto go = [&](auto kernel, const auto& last) {
    return launch_ex(kernel, grid, kMmThreads, 0, ns_smem<kBN>(), stream, "ns_product_kernel launch", a, last);
  };
  if constexpr (kMode != kFinal) {
    return go(kernel_of<kBN, kMode, kF32, false>(), 0);
  } else if (st.update) {
    if (st.out_type == BWD_F32) return go(kernel_of<kBN, kMode, kF32, true>(), *f);
    return st.out_type == BWD_BF16 ? go(kernel_of<kBN, kMode, kBF16, true>(), *f) : go(kernel_of<kBN, kMode, kF16, true>(), *f);
  } else {
    if (st.out_type == BWD_F32) return go(kernel_of<kBN, kMode, kF32, false>(), *f);
    return st.out_type == BWD_BF16 ? go(kernel_of<kBN, kMode, kBF16, false>(), *f) : go(kernel_of<kBN, kMode, kF16, false>(), *f);
  }
}

template <int kMode, bool kLong>
bwd_status launch_small(const SmallCall& c, int tiles, const FinalArgs* f, const Step& st, cudaStream_t stream) {
  const auto go = [&](auto kernel, const auto& last) {
    return launch_ex(kernel, dim3(static_cast<unsigned>(tiles * c.split)), kSmallThreads, c.split, kSmallSmem, stream, "ns_small_kernel launch",
                     c, last);
  };
  if constexpr (kMode != kFinal) {
    return go(ns_small_kernel<kMode, kF32, false, kLong>, 0);
  } else if (st.update) {
    if (st.out_type == BWD_F32) return go(ns_small_kernel<kMode, kF32, true, kLong>, *f);
    return st.out_type == BWD_BF16 ? go(ns_small_kernel<kMode, kBF16, true, kLong>, *f) : go(ns_small_kernel<kMode, kF16, true, kLong>, *f);
  } else {
    if (st.out_type == BWD_F32) return go(ns_small_kernel<kMode, kF32, false, kLong>, *f);
    return st.out_type == BWD_BF16 ? go(ns_small_kernel<kMode, kBF16, false, kLong>, *f) : go(ns_small_kernel<kMode, kF16, false, kLong>, *f);
  }
}

// A group's product: result = alpha add + beta P Q^T (or P Q).
struct Operation {
  Shape result;
  int64_t k, count;
  const __half *p, *q, *add;
  __half* out;
  const float *scale = nullptr, *diagonal = nullptr;
};
struct Factors {
  int passes;
  float alpha, beta;
};

// The kernels' arguments, for tiles of so many rows and columns, of which a
// CTA copies lines_p of P's lines and lines_q of Q's.
template <int kMode>
bwd_status fill_args(ProductArgs& a, const Operation& o, int rows, int cols, int lines_p, int lines_q, const Factors& x) {
  constexpr bool kSymmetric = kMode == kGram || kMode == kPoly;
  a.add_at = o.add; a.out_at = o.out;
  a.m = static_cast<int>(o.result.m); a.n = static_cast<int>(o.result.n); a.pitch = static_cast<int>(up(o.result.n, 64));
  a.kblocks = static_cast<int>((o.k + kBK - 1) / kBK);
  a.passes = x.passes; a.scale = o.scale; a.diagonal = o.diagonal;
  a.tiles_m = static_cast<int>((o.result.m + rows - 1) / rows); a.tiles_n = static_cast<int>((o.result.n + cols - 1) / cols);
  const int64_t tiles = tiles_of(o.result, rows, cols, kSymmetric);
  if (tiles * o.count > 0x3fffffff) return fail(BWD_ERR_INVALID_ARG, "too many tiles");
  a.tiles = static_cast<int>(tiles); a.items = a.whole = static_cast<int>(tiles * o.count);
  a.alpha = x.alpha; a.beta = x.beta;
  // P: lines along k; Q: its lines along k, or its rows along the result's columns
  const bwd_status s = plane_map(&a.p, o.p, o.result.m, up(o.k, 64), 2 * o.count, kBK, lines_p);
  if (s != BWD_OK) return s;
  return kSymmetric ? plane_map(&a.q, o.q, o.result.m, up(o.k, 64), 2 * o.count, kBK, lines_q)
                    : plane_map(&a.q, o.q, o.k, up(o.result.n, 64), 2 * o.count, 64, kBK);
}

// CTAs that divide the summed axis of small products: as many as find an SM.
// (Timestamps in the kernel, 301 x 777: from the inputs to the last product
// 1.4 us with one or two stages to a CTA and 3.3 with five; the exchange of the
// parts costs less than that, and divides the storing too.)
int small_split(int64_t tiles, int64_t kblocks, const DeviceState& d) {
  int split = static_cast<int>(kblocks < kMaxSplit ? kblocks : kMaxSplit);
  while (split > 1 && tiles > d.clusters[split]) --split;
  return split;
}

template <int kMode>
bwd_status products(const Operation* o, int groups, const Factors& x, const FinalArgs* f, const Step& st,
                    const DeviceState& d, cudaStream_t stream) {
  static thread_local SmallCall c;
  c.groups = groups;
  int64_t tiles = 0, kblocks = 1;
  for (int i = 0; i < groups; ++i) {
    const bwd_status s = fill_args<kMode>(c.g[i], o[i], kSmallRows, kSmallCols, kSmallRows, kSmallCols, x);
    if (s != BWD_OK) return s;
    c.start[i] = static_cast<int>(tiles);
    tiles += c.g[i].items;
    kblocks = std::max<int64_t>(kblocks, c.g[i].kblocks);
  }
  c.split = small_split(tiles, kblocks, d);
  const bool longer = (kblocks + c.split - 1) / c.split > kSmallAccs * kChunk;
  return longer ? launch_small<kMode, true>(c, static_cast<int>(tiles), f, st, stream)
                : launch_small<kMode, false>(c, static_cast<int>(tiles), f, st, stream);
}

// One group's product, by whichever kernel takes less time.
template <int kMode>
bwd_status product(const Operation& o, const Factors& x, const FinalArgs* f, const Step& st, const DeviceState& d,
                   cudaStream_t stream) {
  constexpr bool kSymmetric = kMode == kGram || kMode == kPoly;
  // (the last wave of 256 columns counts half where its tiles are cut into halves)
  const int64_t items = o.count * tiles_of(o.result, kBM, 256, kSymmetric), left = items % d.pairs;
  const bool halves = 2 * left <= d.pairs;
  const double waves256 = static_cast<double>(items / d.pairs) + (left == 0 ? 0.0 : halves ? 0.5 : 1.0);
  const double waves128 = static_cast<double>((o.count * tiles_of(o.result, kBM, 128, kSymmetric) + d.pairs - 1) / d.pairs);
  const int64_t kblocks = (o.k + kBK - 1) / kBK, small = o.count * tiles_of(o.result, kSmallRows, kSmallCols, kSymmetric);
  const int split = small_split(small, kblocks, d);
  // Small tiles where they take less time than the large ones.  In us: a stage
  // of a small tile 0.2, and 0.5 where all SMs read (48 KB each, 14.6 TB/s from
  // L2); of a large one, a third of that work for four or eight times the tile,
  // 0.24 with 128 columns and 0.36 with 256; beside its stages a wave of small
  // tiles takes some 5, a launch of large ones 8.  (777 x 301 and five such:
  // 159 us with large tiles, 119 with small ones; A of 4096 x 11008, 1,056
  // small tiles, 600 us against 342 the other way.)
  const int64_t at_once = d.clusters[split] * split, small_waves = (small * split + at_once - 1) / at_once;
  const double full = std::min(1.0, static_cast<double>(small * split) / static_cast<double>(at_once));
  const double stage = (0.2 + 0.3 * full) * (x.passes > 1 ? 1.0 : 0.5);
  const double small_time = static_cast<double>(small_waves) * (5.0 + stage * static_cast<double>((kblocks + split - 1) / split));
  const double large_time = 8.0 + std::min(0.24 * waves128, 0.36 * waves256) * static_cast<double>(x.passes * kblocks);
  if (small_time < large_time) return products<kMode>(&o, 1, x, f, st, d, stream);
  // (eight matrices of 1024 x 4096, A: 133 us with 128 columns, three waves, and 120 with 256, one and a half)
  const int bn = 0.36 * waves256 < 0.24 * waves128 ? 256 : 128;
  ProductArgs a{};
  // of a pair's tile each CTA copies half of either operand's lines
  bwd_status s = fill_args<kMode>(a, o, kBM, bn, kBM / 2, bn / 2, x);
  if (s == BWD_OK && o.add) s = plane_map(&a.add, o.add, o.result.m, a.pitch, 2 * o.count, 32, 32);
  if (s == BWD_OK && o.out) s = plane_map(&a.out, o.out, o.result.m, a.pitch, 2 * o.count, 32, 32);
  if (s != BWD_OK) return s;
  if (bn == 256 && halves) {
    a.whole = a.items - static_cast<int>(left);
    a.items += static_cast<int>(left);
  }
  return bn == 256 ? launch_product<256, kMode>(a, f, st, d.pairs, stream) : launch_product<128, kMode>(a, f, st, d.pairs, stream);
}

template <bool kMomentum>
bwd_status prepare(const PrepareArgs& a, int norm_ctas, int split_ctas, int type, cudaStream_t st) {
  const auto go = [&](auto norm, auto split) {
    const bwd_status s = launch_ex(norm, dim3(static_cast<unsigned>(norm_ctas)), kThreads, 0, 0, st, "ns_norm_kernel launch", a);
    return s == BWD_OK ? launch_ex(split, dim3(static_cast<unsigned>(split_ctas)), kThreads, 0, 0, st, "ns_split_kernel launch", a) : s;
  };
  if (type == BWD_F32) return go(ns_norm_kernel<kF32, kMomentum>, ns_split_kernel<kF32, kMomentum>);
  if (type == BWD_BF16) return go(ns_norm_kernel<kBF16, kMomentum>, ns_split_kernel<kBF16, kMomentum>);
  return go(ns_norm_kernel<kF16, kMomentum>, ns_split_kernel<kF16, kMomentum>);
}

bwd_status run_set(const Matrices& x, const Set& set, const Step& st, uint8_t* work, const DeviceState& d, cudaStream_t stream) {
  static thread_local PrepareArgs a;
  static thread_local FinalArgs f;
  a.x = f.x = x;
  a.grad_scale = f.grad_scale = st.grad_scale;
  a.momentum = st.momentum; a.nesterov = st.nesterov;
  a.groups = set.groups;
  f.decay = st.decay;
  Pieces pieces{work};
  a.slots = reinterpret_cast<double*>(pieces.take(8 * kSlots * set.count()));
  const int squares = set.small ? 0 : squared_steps(set.g[0].s, st);
  float* const scale = reinterpret_cast<float*>(pieces.take(squares > 0 ? 4 * set.count() : 0));
  float* const diagonal = reinterpret_cast<float*>(pieces.take(squares > 0 ? 4 * set.g[0].s.m * set.count() : 0));
  a.scale = squares > 0 && squares == st.steps && !st.has_momentum && st.g_type == BWD_BF16 ? scale : nullptr;
  struct Planes {
    __half *x[2], *a, *p, *q[2];
  } planes[kGroups];
  int64_t norm_ctas = 0, split_ctas = 0;
  for (int i = 0; i < set.groups; ++i) {
    const Group& g = set.g[i];
    const Shape& s = g.s;
    for (__half** at : {&planes[i].x[0], &planes[i].x[1]}) *at = reinterpret_cast<__half*>(pieces.take(s.x_bytes() * g.count));
    for (__half** at : {&planes[i].a, &planes[i].p}) *at = reinterpret_cast<__half*>(pieces.take(s.a_bytes() * g.count));
    if (squares > 0)
      for (__half*& at : planes[i].q) at = reinterpret_cast<__half*>(pieces.take(s.a_bytes() * g.count));
    PrepareGroup& p = a.g[i];
    p.planes = planes[i].x[0];
    p.size = s.m * s.n;
    p.chunk = up((p.size + kSlots - 1) / kSlots, 8 * kThreads);
    p.chunks = static_cast<int>((p.size + p.chunk - 1) / p.chunk);
    p.m = static_cast<int>(s.m); p.n = static_cast<int>(s.n); p.pitch = static_cast<int>(up(s.n, 64));
    // each CTA adds up the norm's parts: four tiles share that where there are many
    p.split_cols = g.count * ((s.m + 63) / 64) * ((s.n + 63) / 64) > 2048 ? 256 : 64;
    p.first = f.first[i] = static_cast<int>(g.first - set.g[0].first);
    p.norm_start = static_cast<int>(norm_ctas); p.split_start = static_cast<int>(split_ctas);
    norm_ctas += g.count * p.chunks;
    split_ctas += g.count * ((p.pitch + p.split_cols - 1) / p.split_cols) * ((s.m + kSplitRows - 1) / kSplitRows);
    f.step[i] = static_cast<float>(st.step * std::sqrt(static_cast<double>(s.n)));
  }
  if (split_ctas > 0x7fffffff) return fail(BWD_ERR_INVALID_ARG, "too many tiles");
  bwd_status e = st.has_momentum ? prepare<true>(a, static_cast<int>(norm_ctas), static_cast<int>(split_ctas), st.g_type, stream)
                                 : prepare<false>(a, static_cast<int>(norm_ctas), static_cast<int>(split_ctas), st.g_type, stream);
  const auto run = [&](auto mode, const Operation* o, const Factors& x) {
    constexpr int kMode = decltype(mode)::value;
    if (e != BWD_OK) return;
    e = set.small ? products<kMode>(o, set.groups, x, &f, st, d, stream) : product<kMode>(o[0], x, &f, st, d, stream);
  };
  constexpr std::integral_constant<int, kGram> to_square{};  // a symmetric product, of A or of two that commute
  constexpr std::integral_constant<int, kPoly> to_poly{};
  constexpr std::integral_constant<int, kApply> to_x{};
  constexpr std::integral_constant<int, kFinal> to_result{};
  const int before = st.steps - squares;
  for (int i = 0; i < before; ++i) {
    const bool last = i + 1 == st.steps;
    Operation gram[kGroups], poly[kGroups], apply[kGroups];
    for (int j = 0; j < set.groups; ++j) {
      const Shape& s = set.g[j].s;
      const Shape square{s.m, s.m};
      const Planes& p = planes[j];
      const __half* const from = p.x[i % 2];
      gram[j] = Operation{square, s.n, set.g[j].count, from, from, nullptr, p.a};
      poly[j] = Operation{square, s.m, set.g[j].count, p.a, p.a, p.a, p.p};
      apply[j] = Operation{s, s.m, set.g[j].count, p.p, from, from, last ? nullptr : p.x[(i + 1) % 2]};
    }
    run(to_square, gram, Factors{3, 0.0f, 1.0f / kScale});
    run(to_poly, poly, Factors{3, kB, kC / kScale});
    if (last) run(to_result, apply, Factors{3, kA / kScale, 1.0f / (kScale * kScale)});
    else run(to_x, apply, Factors{3, kA, 1.0f / kScale});
  }
  if (squares == 0) return e;
  const Group& g = set.g[0];
  const Shape square{g.s.m, g.s.m};
  const __half* const from = planes[0].x[before % 2];
  __half *const at_a = planes[0].a, *const at_p = planes[0].p, *q = planes[0].q[0], *c = planes[0].q[1];
  const auto diagonals = [&](float* out) {
    const int64_t all = g.count * g.s.m;
    if (e == BWD_OK)
      e = launch_ex(ns_diagonal_kernel, dim3(static_cast<unsigned>((all + kThreads - 1) / kThreads)), kThreads, 0, 0, stream,
                    "ns_diagonal_kernel launch", q, g.s.m, up(g.s.m, 64), all, out);
  };
  // a Y + B Y, which is P Y
  const auto times = [&](const __half* b, const __half* y, __half* out, float factor) {
    const Operation o{square, g.s.m, g.count, b, y, y, out};
    run(to_poly, &o, Factors{3, kA * factor, factor / kScale});
  };
  const Operation gram{square, g.s.n, g.count, from, from, nullptr, at_a, a.scale};
  run(to_square, &gram, Factors{a.scale ? 1 : 3, 0.0f, 1.0f / kScale});
  float level = 1.0f;  // Q is stored divided by this
  for (int i = 0; i < squares; ++i) {
    const bool last = i + 1 == squares;
    __half* const b = i == 0 ? q : at_p;
    const Operation poly{square, g.s.m, g.count, at_a, at_a, at_a, b};
    run(to_poly, &poly, Factors{3, kB, kC / kScale});
    if (i > 0) {
      times(b, q, c, 0.25f);
      std::swap(q, c);
      level *= 4.0f;
    }
    if (!last) {
      times(b, at_a, c, 1.0f);
      times(b, c, at_a, 1.0f);
    }
    if (i == 0) diagonals(nullptr);  // the first P is Q
  }
  Operation last{g.s, g.s.m, g.count, q, from, nullptr, nullptr, a.scale};
  if (st.out_type != BWD_BF16) {
    // Q's diagonal outweighs its rows; in the sums each addition would be cut
    // off at its 24th bit (1024 x 4096: 4e-7 of the result)
    diagonals(diagonal);
    last.add = from;
    last.diagonal = diagonal;
  }
  run(to_result, &last, Factors{a.scale ? 2 : 3, 0.0f, level / (kScale * kScale)});
  return e;
}

bool empty(int64_t rows, int64_t cols) { return rows == 0 || cols == 0; }

// Matrices in an order that puts those of one shape together.
bwd_status order(int32_t count, const int64_t* rows, const int64_t* cols, std::vector<int32_t>* out) {
  out->clear();
  for (int32_t i = 0; i < count; ++i) {
    if (rows[i] < 0 || cols[i] < 0 || rows[i] > kMaxSide || cols[i] > kMaxSide) return fail(BWD_ERR_INVALID_ARG, "matrix %d: bad size", i);
    if (!empty(rows[i], cols[i])) out->push_back(i);
  }
  std::stable_sort(out->begin(), out->end(), [&](int32_t a, int32_t b) { return shape_of(rows[a], cols[a]) < shape_of(rows[b], cols[b]); });
  return BWD_OK;
}

// Calls f(set) for matrices in that order, set by set.  Shapes with few tiles
// share sets of up to kBatch matrices and kGroups shapes; the others have sets
// of their own, of equal numbers.  A set of more than one matrix has `work_most`
// bytes at most.
template <typename F>
bwd_status each_set(const std::vector<int32_t>& at, const int64_t* rows, const int64_t* cols, int64_t work_most, F f) {
  constexpr int64_t kFewTiles = 256;
  Set few{};
  few.small = true;
  const auto flush = [&] {
    const bwd_status e = few.groups ? f(few) : BWD_OK;
    few.groups = 0;
    return e;
  };
  const int64_t all = static_cast<int64_t>(at.size());
  for (int64_t i = 0, j; i < all; i = j) {
    const Shape s = shape_of(rows[at[i]], cols[at[i]]);
    for (j = i; j < all && !(s < shape_of(rows[at[j]], cols[at[j]]));) ++j;
    const int64_t number = j - i;
    Set one{};
    one.groups = 1;
    one.g[0] = Group{s, i, number};
    one.small = number <= kBatch && number * tiles_of(s, kSmallRows, kSmallCols, false) <= kFewTiles;
    if (one.small && (number == 1 || one.bytes() <= work_most)) {
      // a set's matrices follow one another
      if (few.groups && (few.groups == kGroups || few.count() + number > kBatch || few.bytes() + one.bytes() > work_most ||
                         few.g[few.groups - 1].first + few.g[few.groups - 1].count != i))
        if (const bwd_status e = flush()) return e;
      few.g[few.groups++] = one.g[0];
      continue;
    }
    one.small = false;
    one.g[0].count = 1;
    int64_t most = work_most / one.bytes();
    most = most < 1 ? 1 : most > kBatch ? kBatch : most;
    const int64_t sets = (number + most - 1) / most, each = (number + sets - 1) / sets;
    for (int64_t b = i; b < j; b += each) {
      one.g[0].first = b;
      one.g[0].count = std::min(each, j - b);
      if (const bwd_status e = f(one)) return e;
    }
  }
  return flush();
}

bwd_status run(int32_t count, const void* const* g, float* const* mom, void* const* out, const int64_t* rows, const int64_t* cols,
               const Step& st, void* work, void* stream) try {
  if (count < 0) return fail(BWD_ERR_INVALID_ARG, "count < 0");
  if (!valid_type(st.g_type)) return fail(BWD_ERR_UNSUPPORTED_DTYPE, "gradient dtype %d", (int)st.g_type);
  if (!valid_type(st.out_type)) return fail(BWD_ERR_UNSUPPORTED_DTYPE, "dtype %d", (int)st.out_type);
  if (st.steps < 1 || st.steps > kMaxSteps) return fail(BWD_ERR_INVALID_ARG, "steps must be 1 to %d", kMaxSteps);
  if (count == 0) return BWD_OK;
  if (!g || !out || !rows || !cols || (st.has_momentum && !mom)) return fail(BWD_ERR_INVALID_ARG, "NULL array");
  if (!aligned_to(st.grad_scale, 4)) return fail(BWD_ERR_INVALID_ARG, "grad_scale is not 4-byte aligned");
  std::vector<int32_t> at;
  bwd_status s = order(count, rows, cols, &at);
  if (s != BWD_OK) return s;
  if (at.empty()) return BWD_OK;
  for (const int32_t i : at) {
    if (!g[i] || !out[i] || (st.has_momentum && !mom[i])) return fail(BWD_ERR_INVALID_ARG, "matrix %d: NULL pointer", i);
    if (!aligned_to(g[i], bytes_of(st.g_type)) || !aligned_to(out[i], bytes_of(st.out_type)) || (st.has_momentum && !aligned_to(mom[i], 4)))
      return fail(BWD_ERR_INVALID_ARG, "matrix %d: pointer not aligned to its element size", i);
  }
  if (!work || !aligned_to(work, 256)) return fail(BWD_ERR_INVALID_ARG, "work must be 256-byte aligned");
  DeviceState d;
  if ((s = ensure_device(&d)) != BWD_OK) return s;
  static thread_local Matrices x;
  return each_set(at, rows, cols, st.work_most, [&](const Set& set) {
    for (int64_t z = 0; z < set.count(); ++z) {
      const int32_t i = at[static_cast<size_t>(set.g[0].first + z)];
      x.g[z] = g[i];
      x.mom[z] = st.has_momentum ? mom[i] : nullptr;
      x.out[z] = out[i];
      x.tall[z] = rows[i] > cols[i];
    }
    return run_set(x, set, st, static_cast<uint8_t*>(work), d, static_cast<cudaStream_t>(stream));
  });
} catch (const std::bad_alloc&) {
  return fail(BWD_ERR_INVALID_ARG, "out of host memory");
}

}  // namespace

namespace bwd {
namespace host {

bwd_status take_muon_fault(unsigned int* fault) { return take_wait_fault(fault); }

}  // namespace host
}  // namespace bwd

extern "C" {

int64_t bwd_orthogonalize_work_bytes(int32_t count, const int64_t* rows, const int64_t* cols) {
  return bwd_muon_work_bytes(count, rows, cols, 0);
}

int64_t bwd_muon_work_bytes(int32_t count, const int64_t* rows, const int64_t* cols, int64_t work_most) try {
  std::vector<int32_t> at;
  if (count < 0 || work_most < 0 || (count > 0 && (!rows || !cols)) || order(count, rows, cols, &at) != BWD_OK) return -1;
  int64_t most = 0;
  each_set(at, rows, cols, work_most > 0 ? work_most : kWorkMost, [&](const Set& set) {
    most = std::max(most, set.bytes());
    return BWD_OK;
  });
  return most;
} catch (const std::bad_alloc&) {
  return -1;
}

bwd_status bwd_orthogonalize(int32_t count, const void* const* g, bwd_dtype dtype, const int64_t* rows, const int64_t* cols, int32_t steps,
                             void* const* out, void* work, void* stream) {
  return run(count, g, nullptr, out, rows, cols, Step{nullptr, 0.0f, 1.0f, 0.0, 0, steps, false, false, dtype, dtype, kWorkMost}, work, stream);
}

bwd_status bwd_muon_step(int32_t count, void* const* p, bwd_dtype p_dtype, const void* const* g, bwd_dtype g_dtype, float* const* mom,
                         const int64_t* rows, const int64_t* cols, const float* grad_scale, const bwd_muon_hparams* hp, void* work,
                         void* stream) {
  if (!hp) return fail(BWD_ERR_INVALID_ARG, "hparams is NULL");
  if (!(hp->lr >= 0.0) || !std::isfinite(hp->lr) || !(hp->momentum >= 0.0 && hp->momentum < 1.0) || !(hp->weight_decay >= 0.0) ||
      !std::isfinite(hp->weight_decay))
    return fail(BWD_ERR_INVALID_ARG, "lr and weight_decay must be finite and >= 0, momentum in [0, 1)");
  if (!(hp->rms >= 0.0) || !std::isfinite(hp->rms)) return fail(BWD_ERR_INVALID_ARG, "rms must be finite and >= 0");
  if (hp->work_most < 0) return fail(BWD_ERR_INVALID_ARG, "work_most must be >= 0");
  const Step st{grad_scale, static_cast<float>(hp->momentum), static_cast<float>(1.0 - hp->lr * hp->weight_decay), hp->lr * hp->rms,
                hp->nesterov != 0, hp->steps, true, true, g_dtype, p_dtype, hp->work_most > 0 ? hp->work_most : kWorkMost};
  return run(count, g, mom, reinterpret_cast<void* const*>(p), rows, cols, st, work, stream);
}

}  // extern "C"
