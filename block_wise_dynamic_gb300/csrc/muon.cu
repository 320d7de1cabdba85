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
// fp16 0.028, pairs 5e-6; fp32 arithmetic has 2e-5).  By the last step the
// spectrum is level and an operand's rounding counts once: for bf16 results,
// whose own rounding is 1.7e-3, that step takes the high parts alone (4e-4 to
// 7e-4 more).
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

struct PrepareArgs {
  Matrices x;
  double* slots;            // [matrix][kSlots]
  const float* grad_scale;  // or null: 1
  __half* planes;           // [matrix][high, low][m][pitch]
  int64_t size;             // elements of a matrix
  int64_t chunk;            // of one CTA of the first kernel
  int chunks;
  int m, n, pitch;          // of the wide form
  float momentum;
  int nesterov;
};

__device__ __forceinline__ bool finite(float s) { return fabsf(s) <= 3.402823466e38f; }

// mom = mu mom + s g; the update u is s g + mu mom, or mom.
__device__ __forceinline__ float new_momentum(const PrepareArgs& a, float s, float g, float mom) {
  return __fmaf_rn(a.momentum, mom, __fmul_rn(s, g));
}
__device__ __forceinline__ float update_of(const PrepareArgs& a, float s, float g, float mom) {
  return a.nesterov ? __fmaf_rn(a.momentum, mom, __fmul_rn(s, g)) : mom;
}

// One chunk of one matrix: the new momentum, and the update's sum of squares
// into its slot (in fp32 for a thread's eight elements, in binary64 beyond
// them, or from the start where fp32 does not hold the squares).
template <int kT, bool kMomentum>
__global__ void __launch_bounds__(kThreads)
ns_norm_kernel(const __grid_constant__ PrepareArgs a) {
  constexpr int kEach = 8;
  __shared__ double s_red[kThreads / 32];
  wait_for_inputs();
  let_next_begin();
  const int z = blockIdx.y;
  const void* const g = a.x.g[z];
  float* const mom = a.x.mom[z];
  const float s = kMomentum && a.grad_scale ? *a.grad_scale : 1.0f;
  double sum = 0.0;
  const int64_t end = min(a.size, (blockIdx.x + 1) * a.chunk);
  for (int64_t i0 = blockIdx.x * a.chunk + threadIdx.x; i0 < end; i0 += kEach * kThreads) {
    float u[kEach], old[kEach];
#pragma unroll
    for (int j = 0; j < kEach; ++j) {
      const int64_t i = i0 + j * kThreads;
      u[j] = i < end ? load1<kT>(g, i) : 0.0f;
      if constexpr (kMomentum) old[j] = i < end ? mom[i] : 0.0f;
    }
    float part = 0.0f;
    uint32_t any = 0;
#pragma unroll
    for (int j = 0; j < kEach; ++j) {
      const int64_t i = i0 + j * kThreads;
      if constexpr (kMomentum) {
        const float next = new_momentum(a, s, u[j], old[j]);
        if (i < end && finite(s)) mom[i] = next;
        u[j] = update_of(a, s, u[j], next);
      }
      any |= __float_as_uint(u[j]);
      part = __fmaf_rn(u[j], u[j], part);
    }
    if ((any & 0x7fffffffu) != 0 && !(part >= 0x1p-120f && part <= 3.402823466e38f)) {
#pragma unroll
      for (int j = 0; j < kEach; ++j) sum = __fma_rn(static_cast<double>(u[j]), static_cast<double>(u[j]), sum);
    } else {
      sum += static_cast<double>(part);
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (threadIdx.x % 32 == 0) s_red[threadIdx.x / 32] = sum;
  __syncthreads();
  if (threadIdx.x != 0) return;
  for (int w = 1; w < kThreads / 32; ++w) sum += s_red[w];
  a.slots[z * kSlots + blockIdx.x] = sum;
}

// Two values as packed pairs of high and low parts.
__device__ __forceinline__ void split2(float v0, float v1, uint32_t& high, uint32_t& low) {
  const __half2 h = __floats2half2_rn(v0, v1);
  const float2 f = __half22float2(h);
  const __half2 l = __floats2half2_rn(__fsub_rn(v0, f.x), __fsub_rn(v1, f.y));
  high = *reinterpret_cast<const uint32_t*>(&h);
  low = *reinterpret_cast<const uint32_t*>(&l);
}

// X's pair from the update, 64 x 64 elements of the wide form to a CTA, which
// go through shared memory so that both sides' rows are contiguous for either
// orientation.  Columns up to the pitch are written, as zeros.
template <int kT, bool kMomentum>
__global__ void __launch_bounds__(kThreads)
ns_split_kernel(const __grid_constant__ PrepareArgs a) {
  __shared__ float s_x[64][65];
  __shared__ double s_red[kThreads / 32];
  __shared__ float s_inv[2];
  wait_for_inputs();
  let_next_begin();
  const int z = blockIdx.z;
  double sum = 0.0;
  for (int i = threadIdx.x; i < a.chunks; i += kThreads) sum += a.slots[z * kSlots + i];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (threadIdx.x % 32 == 0) s_red[threadIdx.x / 32] = sum;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < kThreads / 32; ++w) sum += s_red[w];
    // the norm may pass fp32's range, and its reciprocal what fp32 holds in full
    const double norm = sqrt(sum) + static_cast<double>(kEps);
    const bool large = norm > 0x1p64;
    s_inv[0] = large ? 0x1p-64f : 1.0f;
    s_inv[1] = static_cast<float>((large ? 0x1p64 : 1.0) * static_cast<double>(kScale) / norm);
  }
  __syncthreads();
  const float first = s_inv[0], inv = s_inv[1];
  const void* const g = a.x.g[z];
  const float* const mom = a.x.mom[z];
  const float s = kMomentum && a.grad_scale ? *a.grad_scale : 1.0f;
  const bool tall = a.x.tall[z];
  const int r0 = blockIdx.y * 64, c0 = blockIdx.x * 64;
  // as stored: rows of the wide form, or its columns
  const int rows = tall ? a.n : a.m, cols = tall ? a.m : a.n, sr0 = tall ? c0 : r0, sc0 = tall ? r0 : c0;
#pragma unroll 4
  for (int e = threadIdx.x; e < 64 * 64; e += kThreads) {
    const int r = e / 64, c = e % 64;
    float x = 0.0f;
    if (sr0 + r < rows && sc0 + c < cols) {
      const int64_t i = static_cast<int64_t>(sr0 + r) * cols + sc0 + c;
      x = load1<kT>(g, i);
      if constexpr (kMomentum) x = update_of(a, s, x, mom[i]);
      x = __fmul_rn(__fmul_rn(x, first), inv);
    }
    if (tall) s_x[c][r] = x;
    else s_x[r][c] = x;
  }
  __syncthreads();
  __half* const high = a.planes + static_cast<int64_t>(z) * 2 * a.m * a.pitch;
  __half* const low = high + static_cast<int64_t>(a.m) * a.pitch;
  for (int e = threadIdx.x; e < 64 * 8; e += kThreads) {
    const int r = e / 8, c = e % 8 * 8;
    if (r0 + r >= a.m || c0 + c >= a.pitch) continue;
    uint4 h, l;
#pragma unroll
    for (int j = 0; j < 4; ++j) split2(s_x[r][c + 2 * j], s_x[r][c + 2 * j + 1], (&h.x)[j], (&l.x)[j]);
    const int64_t at = static_cast<int64_t>(r0 + r) * a.pitch + c0 + c;
    *reinterpret_cast<uint4*>(high + at) = h;
    *reinterpret_cast<uint4*>(low + at) = l;
  }
}

// --------------------------------------------------------------------------
// the products
//
// A pair of CTAs (a cluster of two) works on a tile of 256 rows and kBN
// columns; pairs walk the tiles of all matrices with a grid stride.  Warp 0
// copies, warp 1 of the first CTA issues for both, and eight warps store the
// tile before from the other accumulator.
constexpr int kBM = 256;
constexpr int kBK = 64;  // fp16 values of the summed axis in a stage: 128 bytes
constexpr int kMmThreads = 320;
constexpr uint32_t kTmemCols = 512;
constexpr int kPad = 33;  // words of a staged row of 32

template <int kBN> __host__ __device__ constexpr int ns_stages() { return kBN == 256 ? 5 : 6; }
constexpr int kABytes = kBM / 2 * kBK * 2;
template <int kBN> __host__ __device__ constexpr int ns_b_bytes() { return kBN / 2 * kBK * 2; }
template <int kBN> __host__ __device__ constexpr int ns_smem() {
  return 1024 + ns_stages<kBN>() * (kABytes + ns_b_bytes<kBN>()) + 8 * 32 * kPad * 4;
}

enum Mode { kGram, kPoly, kApply, kFinal };

struct ProductArgs {
  CUtensorMap p, q;      // planes of the two operands
  const __half* add;     // planes that alpha multiplies, of the result's shape
  __half* out;           // the result's planes
  int m, n, pitch;       // the result's
  int kblocks;
  int passes;            // 3, or 1: the high parts alone
  int tiles_m, tiles_n, tiles, items;
  float alpha, beta;     // result = alpha add + beta product
};

struct FinalArgs {
  Matrices x;
  const float* grad_scale;  // or null: 1
  float decay, step;        // of the parameter and of the update
};

__device__ __forceinline__ void tma_load3(void* dst, const CUtensorMap* map, int x, int y, int z, uint32_t bar) {
  asm volatile("cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];"
               ::"r"(smem_u32(dst)), "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar) : "memory");
}

struct Tile {
  int z, m0, n0;
  bool mirror;  // also stored transposed
};
// Symmetric results: the tiles that reach the diagonal or lie below it, row
// by row, kBM / kBN more in each row of tiles than in the one before.
template <int kBN, bool kSymmetric>
__device__ __forceinline__ Tile tile_of(const ProductArgs& a, int item) {
  const int z = item / a.tiles, t = item - z * a.tiles;
  if constexpr (!kSymmetric) return Tile{z, t / a.tiles_n * kBM, t % a.tiles_n * kBN, false};
  constexpr int kPer = kBM / kBN;
  // rows of tiles before row i hold kPer i (i + 1) / 2
  int i = static_cast<int>((sqrtf(8.0f * (t / kPer) + 1.0f) - 1.0f) * 0.5f);
  while (kPer * (i + 1) * (i + 2) / 2 <= t) ++i;
  while (kPer * i * (i + 1) / 2 > t) --i;
  const int j = t - kPer * i * (i + 1) / 2;
  return Tile{z, i * kBM, j * kBN, j < kPer * i};
}

__device__ __forceinline__ float half_at(const uint4& w, int j) {
  const uint32_t q = (&w.x)[j / 2];
  return __half2float(__ushort_as_half(static_cast<unsigned short>(j % 2 ? q >> 16 : q & 0xffffu)));
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
  __shared__ __align__(8) uint64_t s_full[kStages], s_empty[kStages], s_acc_full[2], s_acc_empty[2];
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
    for (int i = 0; i < 2; ++i) { mbar_init(&s_acc_full[i], 1); mbar_init(&s_acc_empty[i], 16); }
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
      const Tile tile = tile_of<kBN, kSymmetric>(a, t);
      const int m0 = tile.m0 + static_cast<int>(rank) * (kBM / 2), n0 = tile.n0 + static_cast<int>(rank) * (kBN / 2);
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
      const uint32_t idesc = (1u << 4) | (kTrans ? 1u << 16 : 0u) | ((kBN / 8) << 17) | ((kBM / 16) << 24);
      const uint64_t dp0 = smem_desc(smem_u32(sm), 16, 1024, 2);
      const uint64_t dq0 = kTrans ? smem_desc(smem_u32(sm + kABytes), kBK * 128, 1024, 2) : smem_desc(smem_u32(sm + kABytes), 16, 1024, 2);
      constexpr uint32_t kStepP = 32 / 16, kStepQ = kTrans ? 2048 / 16 : 32 / 16;  // 16 of the summed axis
      Ring<kStages> ring;
      int use = 0;
      bool ok = true;
      const int blocks = a.passes * a.kblocks;
      for (int t = first; ok && t < a.items; t += pairs, ++use) {
        const int buf = use & 1;
        ok = mbar_wait(&s_acc_empty[buf], ((use >> 1) & 1) ^ 1, &s_fail);
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        const uint32_t acc = tmem + buf * 256;
        for (int kb = 0; ok && kb < blocks; ++kb, ring.next()) {
          if (!(ok = mbar_wait(&s_full[ring.s], ring.phase, &s_fail))) break;
          asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
          if (one) {
            const uint64_t dp = dp0 + static_cast<uint32_t>(ring.s * (kStage / 16)), dq = dq0 + static_cast<uint32_t>(ring.s * (kStage / 16));
#pragma unroll
            for (uint32_t q = 0; q < 4; ++q)
              asm volatile("{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
                           "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}"
                           ::"r"(acc), "l"(dp + q * kStepP), "l"(dq + q * kStepQ), "r"(idesc),
                           "r"(static_cast<uint32_t>(kb != 0 || q != 0)) : "memory");
            commit_pair(&s_empty[ring.s]);
          }
          __syncwarp();
        }
        if (one) commit_pair(&s_acc_full[buf]);
        __syncwarp();
      }
    }
  } else {
    wait_for_inputs();
    const int quarter = warp & 3, half = (warp - 2) / 4;
    constexpr int kHalf = kBN / 2;  // columns of one warp
    float* const stage = reinterpret_cast<float*>(sm + kStages * kStage) + (warp - 2) * 32 * kPad;
    const uint32_t own = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + half * kHalf;
    int use = 0;
    bool ok = true, writes = true;
    if constexpr (kMode == kFinal && kUpdate) writes = finite(f.grad_scale ? *f.grad_scale : 1.0f);
    for (int t = first; ok && t < a.items; t += pairs, ++use) {
      const Tile tile = tile_of<kBN, kSymmetric>(a, t);
      const int buf = use & 1, row0 = tile.m0 + static_cast<int>(rank) * (kBM / 2) + quarter * 32, row = row0 + lane;
      const bool in = row < a.m;
      ok = __all_sync(0xffffffffu, mbar_wait(&s_acc_full[buf], (use >> 1) & 1, &s_fail));
      if (!ok) break;
      asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
      const int64_t plane = static_cast<int64_t>(a.m) * a.pitch, at_row = 2 * tile.z * plane + static_cast<int64_t>(in ? row : 0) * a.pitch;
#pragma unroll 1
      for (int g = 0; g < kHalf / 32; ++g) {
        const int col = tile.n0 + half * kHalf + 32 * g;
        uint4 ch[4], cl[4];
        if constexpr (kAdd) {
          if (col < a.pitch) {
            const uint4* const from = reinterpret_cast<const uint4*>(a.add + at_row + col);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              ch[q] = __ldg(from + q);
              cl[q] = __ldg(from + plane / 8 + q);
            }
          }
        }
        uint32_t r[32];
        tmem_load32(own + buf * 256 + 32 * g, r);
        asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
        if (g == kHalf / 32 - 1) {
          asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
          __syncwarp();
          if (lane == 0) mbar_arrive_leader(&s_acc_empty[buf]);
        }
        if (col >= a.pitch) continue;
        float v[32];
#pragma unroll
        for (int j = 0; j < 32; ++j) {
          v[j] = __fmul_rn(a.beta, __uint_as_float(r[j]));
          if constexpr (kAdd) v[j] = __fmaf_rn(a.alpha, __fadd_rn(half_at(ch[j / 8], j % 8), half_at(cl[j / 8], j % 8)), v[j]);
          if constexpr (kSymmetric) v[j] = in ? v[j] : 0.0f;
        }
        if constexpr (kMode != kFinal) {
          uint32_t h[16], l[16];
#pragma unroll
          for (int j = 0; j < 16; ++j) split2(v[2 * j], v[2 * j + 1], h[j], l[j]);
          if (in) {
            uint4* const to = reinterpret_cast<uint4*>(a.out + at_row + col);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              to[q] = make_uint4(h[4 * q], h[4 * q + 1], h[4 * q + 2], h[4 * q + 3]);
              to[plane / 8 + q] = make_uint4(l[4 * q], l[4 * q + 1], l[4 * q + 2], l[4 * q + 3]);
            }
          }
          // Columns left of the diagonal's tiles are all rows of the matrix.
          // As rows they have their zeros up to the pitch from here.
          if (kSymmetric && tile.mirror && row < a.pitch) {
            uint16_t* const to = reinterpret_cast<uint16_t*>(a.out) + 2 * tile.z * plane + static_cast<int64_t>(col) * a.pitch + row;
#pragma unroll
            for (int j = 0; j < 32; ++j) {
              to[static_cast<int64_t>(j) * a.pitch] = static_cast<uint16_t>(j % 2 ? h[j / 2] >> 16 : h[j / 2] & 0xffffu);
              to[plane + static_cast<int64_t>(j) * a.pitch] = static_cast<uint16_t>(j % 2 ? l[j / 2] >> 16 : l[j / 2] & 0xffffu);
            }
          }
        } else {
          void* const out = f.x.out[tile.z];
          const auto emit = [&](int64_t i, float o) {
            if constexpr (kUpdate) store1<kT>(out, i, __fmaf_rn(-f.step, o, __fmul_rn(load1<kT>(out, i), f.decay)));
            else store1<kT>(out, i, o);
          };
          if (!writes) continue;
          if (f.x.tall[tile.z]) {
            if (in) {
#pragma unroll
              for (int j = 0; j < 32; ++j)
                if (col + j < a.n) emit(static_cast<int64_t>(col + j) * a.m + row, v[j]);
            }
          } else {
            __syncwarp();
#pragma unroll
            for (int j = 0; j < 32; ++j) stage[lane * kPad + j] = v[j];
            __syncwarp();
            if (col + lane < a.n) {
              const int rows = a.m - row0 < 32 ? a.m - row0 : 32;
#pragma unroll 8
              for (int q = 0; q < rows; ++q) emit(static_cast<int64_t>(row0 + q) * a.n + col + lane, stage[q * kPad + lane]);
            }
          }
        }
      }
    }
  }
  if (s_fail && lane == 0 && warp < 2) let_copies_land();
  __syncwarp();
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  cluster_sync();
  if (warp == 1) asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols));
}

// --------------------------------------------------------------------------
// host side

bool valid_type(int t) { return t == BWD_F32 || t == BWD_BF16 || t == BWD_F16; }
uintptr_t bytes_of(int t) { return t == BWD_F32 ? 4 : 2; }
int64_t up(int64_t n, int64_t to) { return (n + to - 1) / to * to; }

constexpr int64_t kMaxSide = 65536;
constexpr int kMaxSteps = 100;
constexpr int64_t kWorkMost = int64_t{2} << 30;  // bytes of a batch of more than one matrix

struct Shape {
  int64_t m, n;
  int64_t x_bytes() const { return 4 * m * up(n, 64); }  // a pair of planes
  int64_t a_bytes() const { return 4 * m * up(m, 64); }
  int64_t bytes() const { return 2 * x_bytes() + 2 * a_bytes() + 8 * kSlots + 256; }
  bool operator<(const Shape& o) const { return m != o.m ? m < o.m : n < o.n; }
};
Shape shape_of(int64_t rows, int64_t cols) { return rows > cols ? Shape{cols, rows} : Shape{rows, cols}; }

// Matrices of one shape that are worked on together.
int64_t batch_of(const Shape& s, int64_t count) {
  int64_t most = kWorkMost / s.bytes();
  most = most < 1 ? 1 : most > kBatch ? kBatch : most;
  const int64_t launches = (count + most - 1) / most;
  return (count + launches - 1) / launches;
}

constexpr int kMaxDevices = 64;
struct DeviceState {
  bool ready = false;
  unsigned long long ctx = 0;
  int pairs = 0;
};
std::mutex g_mu;
DeviceState g_dev[kMaxDevices];

template <int kBN, int kMode, int kT, bool kUpdate>
cudaError_t opt_in_one() { return opt_in(ns_product_kernel<kBN, kMode, kT, kUpdate>, ns_smem<kBN>()); }

template <int kBN>
cudaError_t opt_in_all() {
  const cudaError_t e[] = {opt_in_one<kBN, kGram, kF32, false>(), opt_in_one<kBN, kPoly, kF32, false>(), opt_in_one<kBN, kApply, kF32, false>(),
                           opt_in_one<kBN, kFinal, kF32, false>(), opt_in_one<kBN, kFinal, kBF16, false>(), opt_in_one<kBN, kFinal, kF16, false>(),
                           opt_in_one<kBN, kFinal, kF32, true>(), opt_in_one<kBN, kFinal, kBF16, true>(), opt_in_one<kBN, kFinal, kF16, true>()};
  for (const cudaError_t x : e)
    if (x != cudaSuccess) return x;
  return cudaSuccess;
}

bwd_status ensure_device(int* pairs) {
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
    e = cudaOccupancyMaxActiveClusters(&d.pairs, ns_product_kernel<256, kApply, kF32, false>, &cfg);
    if (e != cudaSuccess) return cuda_fail(e, "cudaOccupancyMaxActiveClusters");
    if (d.pairs < 1) return fail(BWD_ERR_CUDA, "no room for a CTA pair of the matrix product");
    d.ctx = ctx;
    d.ready = true;
  }
  *pairs = d.pairs;
  return BWD_OK;
}

// Map of `planes` planes of m rows and `pitch` columns.
bwd_status plane_map(CUtensorMap* map, const __half* base, int64_t m, int64_t pitch, int64_t planes, int box_cols, int box_rows) {
  EncodeFn encode = nullptr;
  const bwd_status s = encode_fn(&encode);
  if (s != BWD_OK) return s;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(pitch), static_cast<cuuint64_t>(m), static_cast<cuuint64_t>(planes)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(pitch * 2), static_cast<cuuint64_t>(m * pitch * 2)};
  const cuuint32_t box[3] = {static_cast<cuuint32_t>(box_cols), static_cast<cuuint32_t>(box_rows), 1}, step[3] = {1, 1, 1};
  const CUresult r = encode(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<__half*>(base), dims, strides, box, step,
                            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
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
};

// Tiles of a product with kBN columns each.
int64_t tiles_of(const Shape& result, int bn, bool symmetric) {
  const int64_t tm = (result.m + kBM - 1) / kBM;
  return symmetric ? kBM / bn * tm * (tm + 1) / 2 : tm * ((result.n + bn - 1) / bn);
}

template <int kBN, int kMode>
bwd_status launch_product(const ProductArgs& a, const FinalArgs* f, const Step& st, int pairs, cudaStream_t stream) {
  const dim3 grid(static_cast<unsigned>(2 * (a.items < pairs ? a.items : pairs)));
  const auto go = [&](auto kernel, const auto& last) {
    return launch_ex(kernel, grid, kMmThreads, 0, ns_smem<kBN>(), stream, "ns_product_kernel launch", a, last);
  };
  if constexpr (kMode != kFinal) {
    return go(ns_product_kernel<kBN, kMode, kF32, false>, 0);
  } else if (st.update) {
    if (st.out_type == BWD_F32) return go(ns_product_kernel<kBN, kMode, kF32, true>, *f);
    return st.out_type == BWD_BF16 ? go(ns_product_kernel<kBN, kMode, kBF16, true>, *f) : go(ns_product_kernel<kBN, kMode, kF16, true>, *f);
  } else {
    if (st.out_type == BWD_F32) return go(ns_product_kernel<kBN, kMode, kF32, false>, *f);
    return st.out_type == BWD_BF16 ? go(ns_product_kernel<kBN, kMode, kBF16, false>, *f) : go(ns_product_kernel<kBN, kMode, kF16, false>, *f);
  }
}

// result = alpha add + beta P Q^T (or P Q), `count` matrices.
template <int kMode>
bwd_status product(const Shape& result, int64_t k, int64_t count, const __half* p, const __half* q, const __half* add, __half* out,
                   float alpha, float beta, int passes, const FinalArgs* f, const Step& st, int pairs, cudaStream_t stream) {
  constexpr bool kSymmetric = kMode == kGram || kMode == kPoly;
  const auto waves = [&](int bn) { return (count * tiles_of(result, bn, kSymmetric) + pairs - 1) / pairs; };
  // a tile of 256 columns takes up to one and a half times as long as one of 128
  const int bn = 3 * waves(256) < 2 * waves(128) ? 256 : 128;
  ProductArgs a{};
  a.add = add; a.out = out;
  a.m = static_cast<int>(result.m); a.n = static_cast<int>(result.n); a.pitch = static_cast<int>(up(result.n, 64));
  a.kblocks = static_cast<int>((k + kBK - 1) / kBK);
  a.passes = passes;
  a.tiles_m = static_cast<int>((result.m + kBM - 1) / kBM); a.tiles_n = static_cast<int>((result.n + bn - 1) / bn);
  const int64_t tiles = tiles_of(result, bn, kSymmetric);
  if (tiles * count > 0x3fffffff) return fail(BWD_ERR_INVALID_ARG, "too many tiles");
  a.tiles = static_cast<int>(tiles); a.items = static_cast<int>(tiles * count);
  a.alpha = alpha; a.beta = beta;
  // P: `m` lines along k; Q: its lines along k, or its rows along the result's columns
  bwd_status s = plane_map(&a.p, p, result.m, up(k, 64), 2 * count, kBK, kBM / 2);
  if (s != BWD_OK) return s;
  s = kSymmetric ? plane_map(&a.q, q, result.m, up(k, 64), 2 * count, kBK, bn / 2) : plane_map(&a.q, q, k, up(result.n, 64), 2 * count, 64, kBK);
  if (s != BWD_OK) return s;
  return bn == 256 ? launch_product<256, kMode>(a, f, st, pairs, stream) : launch_product<128, kMode>(a, f, st, pairs, stream);
}

template <bool kMomentum>
bwd_status prepare(const PrepareArgs& a, int64_t count, int type, cudaStream_t st) {
  const dim3 by_chunk(static_cast<unsigned>(a.chunks), static_cast<unsigned>(count));
  const dim3 by_tile(static_cast<unsigned>((a.pitch + 63) / 64), static_cast<unsigned>((a.m + 63) / 64), static_cast<unsigned>(count));
  const auto go = [&](auto norm, auto split) {
    const bwd_status s = launch_ex(norm, by_chunk, kThreads, 0, 0, st, "ns_norm_kernel launch", a);
    return s == BWD_OK ? launch_ex(split, by_tile, kThreads, 0, 0, st, "ns_split_kernel launch", a) : s;
  };
  if (type == BWD_F32) return go(ns_norm_kernel<kF32, kMomentum>, ns_split_kernel<kF32, kMomentum>);
  if (type == BWD_BF16) return go(ns_norm_kernel<kBF16, kMomentum>, ns_split_kernel<kBF16, kMomentum>);
  return go(ns_norm_kernel<kF16, kMomentum>, ns_split_kernel<kF16, kMomentum>);
}

// All of one batch: matrices of one shape, in either orientation.
bwd_status run_batch(const Matrices& x, int64_t count, const Shape& s, const Step& st, uint8_t* work, int pairs, cudaStream_t stream) {
  Pieces pieces{work};
  double* const slots = reinterpret_cast<double*>(pieces.take(8 * kSlots * count));
  __half* xs[2] = {reinterpret_cast<__half*>(pieces.take(s.x_bytes() * count)), reinterpret_cast<__half*>(pieces.take(s.x_bytes() * count))};
  __half* const gram = reinterpret_cast<__half*>(pieces.take(s.a_bytes() * count));
  __half* const poly = reinterpret_cast<__half*>(pieces.take(s.a_bytes() * count));
  static thread_local PrepareArgs a;
  static thread_local FinalArgs f;
  a.x = x; a.slots = slots; a.grad_scale = st.grad_scale; a.planes = xs[0];
  a.size = s.m * s.n;
  a.chunk = up((a.size + kSlots - 1) / kSlots, 8 * kThreads);
  a.chunks = static_cast<int>((a.size + a.chunk - 1) / a.chunk);
  a.m = static_cast<int>(s.m); a.n = static_cast<int>(s.n); a.pitch = static_cast<int>(up(s.n, 64));
  a.momentum = st.momentum; a.nesterov = st.nesterov;
  bwd_status e = st.has_momentum ? prepare<true>(a, count, st.g_type, stream) : prepare<false>(a, count, st.g_type, stream);
  f.x = x; f.grad_scale = st.grad_scale; f.decay = st.decay;
  f.step = static_cast<float>(st.step * std::sqrt(static_cast<double>(s.n)));
  const Shape square{s.m, s.m};
  for (int i = 0; e == BWD_OK && i < st.steps; ++i) {
    const bool last = i + 1 == st.steps;
    const int passes = last && st.out_type == BWD_BF16 ? 1 : 3;
    const __half* const from = xs[i % 2];
    e = product<kGram>(square, s.n, count, from, from, nullptr, gram, 0.0f, 1.0f / kScale, passes, nullptr, st, pairs, stream);
    if (e == BWD_OK)
      e = product<kPoly>(square, s.m, count, gram, gram, gram, poly, kB, kC / kScale, passes, nullptr, st, pairs, stream);
    if (e != BWD_OK) break;
    e = last ? product<kFinal>(s, s.m, count, poly, from, from, nullptr, kA / kScale, 1.0f / (kScale * kScale), passes, &f, st, pairs, stream)
             : product<kApply>(s, s.m, count, poly, from, from, xs[(i + 1) % 2], kA, 1.0f / kScale, passes, nullptr, st, pairs, stream);
  }
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

// Calls f(first, number, shape, matrices of one batch) for each group.
template <typename F>
bwd_status each_group(const std::vector<int32_t>& at, const int64_t* rows, const int64_t* cols, F f) {
  for (size_t i = 0; i < at.size();) {
    const Shape s = shape_of(rows[at[i]], cols[at[i]]);
    size_t j = i;
    while (j < at.size() && !(s < shape_of(rows[at[j]], cols[at[j]]))) ++j;
    const bwd_status e = f(i, static_cast<int64_t>(j - i), s);
    if (e != BWD_OK) return e;
    i = j;
  }
  return BWD_OK;
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
  int pairs = 0;
  if ((s = ensure_device(&pairs)) != BWD_OK) return s;
  static thread_local Matrices x;
  return each_group(at, rows, cols, [&](size_t first, int64_t number, const Shape& shape) {
    const int64_t batch = batch_of(shape, number);
    for (int64_t b = 0; b < number; b += batch) {
      const int64_t n = number - b < batch ? number - b : batch;
      for (int64_t z = 0; z < n; ++z) {
        const int32_t i = at[first + b + z];
        x.g[z] = g[i];
        x.mom[z] = st.has_momentum ? mom[i] : nullptr;
        x.out[z] = out[i];
        x.tall[z] = rows[i] > cols[i];
      }
      const bwd_status e = run_batch(x, n, shape, st, static_cast<uint8_t*>(work), pairs, static_cast<cudaStream_t>(stream));
      if (e != BWD_OK) return e;
    }
    return BWD_OK;
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

int64_t bwd_orthogonalize_work_bytes(int32_t count, const int64_t* rows, const int64_t* cols) try {
  std::vector<int32_t> at;
  if (count < 0 || (count > 0 && (!rows || !cols)) || order(count, rows, cols, &at) != BWD_OK) return -1;
  int64_t most = 0;
  each_group(at, rows, cols, [&](size_t, int64_t number, const Shape& s) {
    const int64_t batch = batch_of(s, number);
    Pieces pieces{nullptr};
    pieces.take(8 * kSlots * batch);
    for (int i = 0; i < 2; ++i) pieces.take(s.x_bytes() * batch);
    for (int i = 0; i < 2; ++i) pieces.take(s.a_bytes() * batch);
    if (pieces.used > most) most = pieces.used;
    return BWD_OK;
  });
  return most;
} catch (const std::bad_alloc&) {
  return -1;
}

bwd_status bwd_orthogonalize(int32_t count, const void* const* g, bwd_dtype dtype, const int64_t* rows, const int64_t* cols, int32_t steps,
                             void* const* out, void* work, void* stream) {
  return run(count, g, nullptr, out, rows, cols, Step{nullptr, 0.0f, 1.0f, 0.0, 0, steps, false, false, dtype, dtype}, work, stream);
}

bwd_status bwd_muon_step(int32_t count, void* const* p, bwd_dtype p_dtype, const void* const* g, bwd_dtype g_dtype, float* const* mom,
                         const int64_t* rows, const int64_t* cols, const float* grad_scale, const bwd_muon_hparams* hp, void* work,
                         void* stream) {
  if (!hp) return fail(BWD_ERR_INVALID_ARG, "hparams is NULL");
  if (!(hp->lr >= 0.0) || !std::isfinite(hp->lr) || !(hp->momentum >= 0.0 && hp->momentum < 1.0) || !(hp->weight_decay >= 0.0) ||
      !std::isfinite(hp->weight_decay))
    return fail(BWD_ERR_INVALID_ARG, "lr and weight_decay must be finite and >= 0, momentum in [0, 1)");
  if (!(hp->rms >= 0.0) || !std::isfinite(hp->rms)) return fail(BWD_ERR_INVALID_ARG, "rms must be finite and >= 0");
  const Step st{grad_scale, static_cast<float>(hp->momentum), static_cast<float>(1.0 - hp->lr * hp->weight_decay), hp->lr * hp->rms,
                hp->nesterov != 0, hp->steps, true, true, g_dtype, p_dtype};
  return run(count, g, mom, reinterpret_cast<void* const*>(p), rows, cols, st, work, stream);
}

}  // extern "C"
