// Layer normalisation over the rows of a matrix, forward and backward
// (sm_103a).
//
//   mean = sum x / D;  var = sum (x - mean)^2 / D;  rstd = (var + eps)^-1/2
//   xh = (x - mean) rstd;  y = xh gamma + beta
//   h = dy gamma;  dx = rstd (h - sum h / D - xh sum(h xh) / D)
//   dgamma = sum over rows of dy xh;  dbeta = sum over rows of dy
//
// Each row is read once: a group of threads (a warp, or a CTA) holds it in
// registers as it was stored, forms the sums and writes the result.  The
// variance is summed from the centred values, so a row's offset costs no
// accuracy.  A group walks rows with a grid stride and has the next row's
// loads under way while it works on one; a thread's columns are the same in
// every row, so gamma and beta, and in the backward pass its columns' sums of
// dy xh and dy, stay with it.  Those sums go to a workspace, a row for each
// CTA, and a second kernel adds them in a fixed order: results do not depend
// on the schedule.
#include "tensor.cuh"

#include <algorithm>
#include <atomic>

namespace {

constexpr int kMaxWidth = 16384;
constexpr int kWarpWidth = 512;   // widest row that a warp takes
constexpr int kWarps = 8;         // rows of such a CTA
constexpr int kThreadValues = 16; // values of a row that a thread holds
constexpr int kMaxThreads = kMaxWidth / kThreadValues;

template <int kBytes> struct UnitOf;
template <> struct UnitOf<16> { using T = uint4; };
template <> struct UnitOf<8> { using T = uint2; };
template <> struct UnitOf<4> { using T = uint32_t; };
template <> struct UnitOf<2> { using T = uint16_t; };

// A thread's part of a row: units of kVals consecutive values, a group's
// threads side by side.
template <int kT, int kVals>
struct Part {
  static constexpr int kUnits = kThreadValues / kVals;
  using Unit = typename UnitOf<kVals * elem_bytes<kT>()>::T;
  Unit u[kUnits];

  __device__ __forceinline__ void load(const void* row, int width, int t, int threads) {
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
      const int c = (i * threads + t) * kVals;
      u[i] = c < width ? __ldcs(reinterpret_cast<const Unit*>(static_cast<const char*>(row) + static_cast<int64_t>(c) * elem_bytes<kT>())) : Unit{};
    }
  }
  __device__ __forceinline__ void load_shared(const uint8_t* row, int width, int t, int threads) {
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
      const int c = (i * threads + t) * kVals;
      u[i] = c < width ? *reinterpret_cast<const Unit*>(row + c * elem_bytes<kT>()) : Unit{};
    }
  }
  // 32-bit word k of unit i
  __device__ __forceinline__ uint32_t word(int i, int k) const {
    if constexpr (sizeof(Unit) <= 4) return u[i];
    else return (&u[i].x)[k];
  }
  __device__ __forceinline__ float value(int i, int j) const {
    if constexpr (kT == kF32) {
      return __uint_as_float(word(i, j));
    } else {
      const uint32_t w = word(i, j / 2);
      if constexpr (kT == kBF16) return __uint_as_float(j % 2 ? w & 0xffff0000u : w << 16);
      else return __half2float(__ushort_as_half(static_cast<unsigned short>(j % 2 ? w >> 16 : w & 0xffffu)));
    }
  }
  // values 2 k and 2 k + 1
  __device__ __forceinline__ float2 two(int i, int k) const {
    if constexpr (kT == kF16) {
      const uint32_t w = word(i, k);
      return __half22float2(*reinterpret_cast<const __half2*>(&w));
    } else {
      return make_float2(value(i, 2 * k), value(i, 2 * k + 1));
    }
  }
};

template <int kT, int kVals>
__device__ __forceinline__ void store_unit(void* row, int c, const float* v) {
  using Unit = typename UnitOf<kVals * elem_bytes<kT>()>::T;
  Unit u;
  if constexpr (kT == kF32) {
#pragma unroll
    for (int j = 0; j < kVals; ++j) reinterpret_cast<float*>(&u)[j] = v[j];
  } else if constexpr (kVals == 1) {
    u = static_cast<uint16_t>(pack16<kT>(v[0], 0.0f));
  } else {
#pragma unroll
    for (int j = 0; j < kVals; j += 2) reinterpret_cast<uint32_t*>(&u)[j / 2] = pack16<kT>(v[j], v[j + 1]);
  }
  *reinterpret_cast<Unit*>(static_cast<char*>(row) + static_cast<int64_t>(c) * elem_bytes<kT>()) = u;
}

struct VectorArg {
  const void* p;  // or null
  int f32;        // fp32, else of x's type
};
template <int kT>
__device__ __forceinline__ float vector_at(const VectorArg& a, int c, float otherwise) {
  if (!a.p) return otherwise;
  return a.f32 ? static_cast<const float*>(a.p)[c] : load1<kT>(a.p, c);
}

// Sums of a group's values, the same in each of its threads.  Two buffers in
// turn: a thread writes to one again only after all have passed the barrier
// of the sum between, behind which none reads it.
template <bool kWarp, int kN>
struct GroupSum {
  float (*red)[2][32];  // [2 turns][kN <= 2][warps]
  int turn = 0;
  __device__ __forceinline__ void operator()(float (&s)[kN]) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
      for (int n = 0; n < kN; ++n) s[n] += __shfl_xor_sync(0xffffffffu, s[n], o);
    if constexpr (!kWarp) {
      const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, warps = blockDim.x / 32;
      if (warps == 1) return;
      if (lane == 0)
#pragma unroll
        for (int n = 0; n < kN; ++n) red[turn][n][warp] = s[n];
      __syncthreads();
#pragma unroll
      for (int n = 0; n < kN; ++n) s[n] = lane < warps ? red[turn][n][lane] : 0.0f;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1)
#pragma unroll
        for (int n = 0; n < kN; ++n) s[n] += __shfl_xor_sync(0xffffffffu, s[n], o);
      turn ^= 1;
    }
  }
};

struct ForwardArgs {
  const void* x;
  int64_t ldx;  // elements between rows
  VectorArg gamma, beta;
  void* y;
  float* mean;  // or null
  float* rstd;  // or null
  int64_t rows;
  int width;
  float eps;
};

// kMax: threads of a CTA at most.  Up to half of kMaxThreads gamma and beta
// stay in registers; wider rows read them again each time.
template <int kT, int kVals, bool kWarp, int kMax>
__global__ void __launch_bounds__(kMax)
norm_forward_kernel(const ForwardArgs a) {
  constexpr int kUnits = kThreadValues / kVals;
  constexpr bool kKeep = kMax <= kMaxThreads / 2;
  __shared__ float s_red[2][2][32];
  const int threads = kWarp ? 32 : blockDim.x, t = kWarp ? threadIdx.x % 32 : threadIdx.x;
  const int64_t groups = kWarp ? static_cast<int64_t>(gridDim.x) * kWarps : gridDim.x;
  int64_t row = kWarp ? static_cast<int64_t>(blockIdx.x) * kWarps + threadIdx.x / 32 : blockIdx.x;
  GroupSum<kWarp, 1> sum{s_red};
  const auto x_row = [&](int64_t r) { return static_cast<const char*>(a.x) + r * a.ldx * elem_bytes<kT>(); };
  wait_for_inputs();
  let_next_begin();
  Part<kT, kVals> next;
  if (row < a.rows) next.load(x_row(row), a.width, t, threads);
  float g[kKeep ? kThreadValues : 1], b[kKeep ? kThreadValues : 1];
  if constexpr (kKeep) {
#pragma unroll
    for (int i = 0; i < kUnits; ++i)
#pragma unroll
      for (int j = 0; j < kVals; ++j) {
        const int c = (i * threads + t) * kVals;
        g[i * kVals + j] = c < a.width ? vector_at<kT>(a.gamma, c + j, 1.0f) : 0.0f;
        b[i * kVals + j] = c < a.width ? vector_at<kT>(a.beta, c + j, 0.0f) : 0.0f;
      }
  }
  const float width = static_cast<float>(a.width);
  for (; row < a.rows; row += groups) {
    float v[kThreadValues];
    float s[1] = {0.0f};
#pragma unroll
    for (int i = 0; i < kUnits; ++i)
#pragma unroll
      for (int j = 0; j < kVals; ++j) s[0] += v[i * kVals + j] = next.value(i, j);
    if (row + groups < a.rows) next.load(x_row(row + groups), a.width, t, threads);
    sum(s);
    const float mean = __fdiv_rn(s[0], width);
    s[0] = 0.0f;
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
      const bool in = (i * threads + t) * kVals < a.width;
#pragma unroll
      for (int j = 0; j < kVals; ++j) {
        float& d = v[i * kVals + j];
        d = in ? __fsub_rn(d, mean) : 0.0f;
        s[0] = __fmaf_rn(d, d, s[0]);
      }
    }
    sum(s);
    const float rstd = __fdiv_rn(1.0f, __fsqrt_rn(__fadd_rn(__fdiv_rn(s[0], width), a.eps)));
    if (t == 0) {
      if (a.mean) a.mean[row] = mean;
      if (a.rstd) a.rstd[row] = rstd;
    }
    char* const y = static_cast<char*>(a.y) + row * a.width * elem_bytes<kT>();
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
      const int c = (i * threads + t) * kVals;
      if (c >= a.width) continue;
      float out[kVals];
#pragma unroll
      for (int j = 0; j < kVals; ++j) {
        const int e = i * kVals + j;
        out[j] = __fmaf_rn(__fmul_rn(v[e], rstd), kKeep ? g[kKeep ? e : 0] : vector_at<kT>(a.gamma, c + j, 1.0f),
                           kKeep ? b[kKeep ? e : 0] : vector_at<kT>(a.beta, c + j, 0.0f));
      }
      store_unit<kT, kVals>(y, c, out);
    }
  }
}

struct BackwardArgs {
  const void* dy;
  const void* x;
  int64_t lddy, ldx;
  VectorArg gamma;
  const float* mean;
  const float* rstd;
  void* dx;        // or null
  float* partial;  // [2][CTAs][width]: sums of dy xh and of dy; or null
  int64_t rows;
  int width;
};

// The columns' sums are kept in registers for CTAs of up to half of
// kMaxThreads, in shared memory for wider ones.
template <int kT, int kVals, bool kWarp, int kMax>
__global__ void __launch_bounds__(kMax)
norm_backward_kernel(const BackwardArgs a) {
  constexpr int kUnits = kThreadValues / kVals;
  constexpr bool kKeep = kMax <= kMaxThreads / 2;
  extern __shared__ __align__(128) uint8_t s_raw[];
  float* const s_sums = reinterpret_cast<float*>(s_raw);  // [2][width]: of wide rows, or of a CTA's warps
  __shared__ float s_red[2][2][32];
  const int threads = kWarp ? 32 : blockDim.x, t = kWarp ? threadIdx.x % 32 : threadIdx.x;
  const int64_t groups = kWarp ? static_cast<int64_t>(gridDim.x) * kWarps : gridDim.x;
  int64_t row = kWarp ? static_cast<int64_t>(blockIdx.x) * kWarps + threadIdx.x / 32 : blockIdx.x;
  GroupSum<kWarp, 2> sum{s_red};
  const auto x_row = [&](int64_t r) { return static_cast<const char*>(a.x) + r * a.ldx * elem_bytes<kT>(); };
  const auto dy_row = [&](int64_t r) { return static_cast<const char*>(a.dy) + r * a.lddy * elem_bytes<kT>(); };
  wait_for_inputs();
  let_next_begin();
  Part<kT, kVals> next_x, next_dy;
  float next_mean = 0.0f, next_rstd = 0.0f;
  const auto fetch = [&](int64_t r) {
    next_x.load(x_row(r), a.width, t, threads);
    next_dy.load(dy_row(r), a.width, t, threads);
    next_mean = a.mean[r];
    next_rstd = a.rstd[r];
  };
  if (row < a.rows) fetch(row);
  float g[kKeep ? kThreadValues : 1], dg[kKeep ? kThreadValues : 1], db[kKeep ? kThreadValues : 1];
  if constexpr (kKeep) {
#pragma unroll
    for (int i = 0; i < kUnits; ++i)
#pragma unroll
      for (int j = 0; j < kVals; ++j) {
        const int c = (i * threads + t) * kVals, e = i * kVals + j;
        g[e] = c < a.width ? vector_at<kT>(a.gamma, c + j, 1.0f) : 0.0f;
        dg[e] = db[e] = 0.0f;
      }
  } else if (a.partial) {
    // each thread's own columns: no barrier is needed
    for (int i = 0; i < kUnits; ++i)
      for (int j = 0; j < kVals; ++j) {
        const int c = (i * threads + t) * kVals + j;
        if (c < a.width) s_sums[c] = s_sums[a.width + c] = 0.0f;
      }
  }
  const float width = static_cast<float>(a.width);
  for (; row < a.rows; row += groups) {
    const Part<kT, kVals> x = next_x, dy = next_dy;
    const float mean = next_mean, rstd = next_rstd;
    if (row + groups < a.rows) fetch(row + groups);
    float s[2] = {0.0f, 0.0f};
    const auto xh_of = [&](int i, int j) { return __fmul_rn(__fsub_rn(x.value(i, j), mean), rstd); };
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
      const int c = (i * threads + t) * kVals;
      if (c >= a.width) continue;
#pragma unroll
      for (int j = 0; j < kVals; ++j) {
        const int e = i * kVals + j;
        const float d = dy.value(i, j), xh = xh_of(i, j);
        float gamma;
        if constexpr (kKeep) {
          gamma = g[e];
          dg[e] = __fmaf_rn(d, xh, dg[e]);
          db[e] = __fadd_rn(db[e], d);
        } else {
          gamma = vector_at<kT>(a.gamma, c + j, 1.0f);
          if (a.partial) {
            s_sums[c + j] = __fmaf_rn(d, xh, s_sums[c + j]);
            s_sums[a.width + c + j] = __fadd_rn(s_sums[a.width + c + j], d);
          }
        }
        const float h = __fmul_rn(d, gamma);
        s[0] += h;
        s[1] = __fmaf_rn(h, xh, s[1]);
      }
    }
    if (!a.dx) continue;
    sum(s);
    const float mean_h = __fdiv_rn(s[0], width), mean_hx = __fdiv_rn(s[1], width);
    char* const dx = static_cast<char*>(a.dx) + row * a.width * elem_bytes<kT>();
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
      const int c = (i * threads + t) * kVals;
      if (c >= a.width) continue;
      float out[kVals];
#pragma unroll
      for (int j = 0; j < kVals; ++j) {
        const float h = __fmul_rn(dy.value(i, j), kKeep ? g[kKeep ? i * kVals + j : 0] : vector_at<kT>(a.gamma, c + j, 1.0f));
        out[j] = __fmul_rn(rstd, __fmaf_rn(-xh_of(i, j), mean_hx, __fsub_rn(h, mean_h)));
      }
      store_unit<kT, kVals>(dx, c, out);
    }
  }
  if (!a.partial) return;
  float* const to_gamma = a.partial + static_cast<int64_t>(blockIdx.x) * a.width;
  float* const to_beta = to_gamma + static_cast<int64_t>(gridDim.x) * a.width;
  if constexpr (kWarp) {
    // the CTA's warps one after the other
    for (int w = 0; w < kWarps; ++w) {
      if (threadIdx.x / 32 == w) {
#pragma unroll
        for (int i = 0; i < kUnits; ++i)
#pragma unroll
          for (int j = 0; j < kVals; ++j) {
            const int c = (i * 32 + t) * kVals + j, e = i * kVals + j;
            if (c < a.width) {
              s_sums[c] = w ? __fadd_rn(s_sums[c], dg[kKeep ? e : 0]) : dg[kKeep ? e : 0];
              s_sums[a.width + c] = w ? __fadd_rn(s_sums[a.width + c], db[kKeep ? e : 0]) : db[kKeep ? e : 0];
            }
          }
      }
      __syncthreads();
    }
    for (int c = threadIdx.x; c < a.width; c += 32 * kWarps) {
      to_gamma[c] = s_sums[c];
      to_beta[c] = s_sums[a.width + c];
    }
  } else {
#pragma unroll
    for (int i = 0; i < kUnits; ++i)
#pragma unroll
      for (int j = 0; j < kVals; ++j) {
        const int c = (i * threads + t) * kVals + j;
        if (c >= a.width) continue;
        to_gamma[c] = kKeep ? dg[kKeep ? i * kVals + j : 0] : s_sums[c];
        to_beta[c] = kKeep ? db[kKeep ? i * kVals + j : 0] : s_sums[a.width + c];
      }
  }
}

// --------------------------------------------------------------------------
// rows of whole 16-byte pieces, many of them

// Two operations in one instruction, each rounded by itself.
__device__ __forceinline__ uint64_t bits2(float2 a) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a.x), "f"(a.y));
  return r;
}
__device__ __forceinline__ float2 from2(uint64_t a) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a));
  return r;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(bits2(a)), "l"(bits2(b)));
  return from2(r);
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(bits2(a)), "l"(bits2(b)));
  return from2(r);
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(bits2(a)), "l"(bits2(b)), "l"(bits2(c)));
  return from2(r);
}
__device__ __forceinline__ float2 both(float a) { return make_float2(a, a); }
//
// A CTA takes kR rows at a time: what a row costs beside its bytes is the
// latency of its sums over the CTA, which kR rows share.  Rows come into
// shared memory by bulk copies, a set of kR ahead, and are read from there by
// each pass over them; the registers hold gamma, beta and the columns' sums.
// (16384 x 4096 bf16, forward and backward, with a row at a time in registers:
// 58 and 97 us; from shared memory, a row at a time, 56 and 100, and these sets
// with one operation to an instruction 58 and 89, bound by instructions.)

constexpr int kSets = 2;  // of rows, at most one of them being read

template <int kR, int kArrays>
struct RowRing {
  uint64_t* bars;
  uint8_t* rows;  // [kSets][kR][kArrays][row_bytes]
  int row_bytes;
  int s = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ const uint8_t* row(int r, int array) const { return rows + ((s * kR + r) * kArrays + array) * row_bytes; }
  __device__ __forceinline__ void init() {
    if (threadIdx.x == 0) {
      for (int i = 0; i < kSets; ++i) mbar_init(&bars[i], 1);
      asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncthreads();
  }
  // By one thread: rows first .. first + count - 1 of each array, `ld` bytes apart.
  __device__ __forceinline__ void fill(int set, int count, const char* x, int64_t ldx, const char* y, int64_t ldy) {
    mbar_expect_tx(&bars[set], count * kArrays * row_bytes);
    for (int r = 0; r < count; ++r) {
      uint8_t* const to = rows + (set * kR + r) * kArrays * row_bytes;
      bulk_load(to, x + r * ldx, row_bytes, &bars[set]);
      if constexpr (kArrays == 2) bulk_load(to + row_bytes, y + r * ldy, row_bytes, &bars[set]);
    }
  }
  // Waits for the current set.  Where a wait gives up, the CTA goes on over
  // whatever there is, with no wait any more, so that its barriers still meet.
  __device__ __forceinline__ void wait(volatile int* fail) { mbar_wait(&bars[s], phase, fail); }
  __device__ __forceinline__ void next() {
    if (++s == kSets) { s = 0; phase ^= 1u; }
  }
};

// Sums of kN values over a CTA, the same in each of its threads; two buffers
// in turn, as for GroupSum.
template <int kN>
__device__ __forceinline__ void cta_sum(float (&s)[kN], float (*red)[32][kN], int& turn) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
#pragma unroll
    for (int n = 0; n < kN; ++n) s[n] += __shfl_xor_sync(0xffffffffu, s[n], o);
  const int warp = threadIdx.x / 32, warps = blockDim.x / 32;
  if (threadIdx.x % 32 == 0)
#pragma unroll
    for (int n = 0; n < kN; ++n) red[turn][warp][n] = s[n];
  __syncthreads();
#pragma unroll
  for (int n = 0; n < kN; ++n) s[n] = 0.0f;
#pragma unroll 4
  for (int w = 0; w < warps; ++w)
#pragma unroll
    for (int n = 0; n < kN; ++n) s[n] += red[turn][w][n];
  turn ^= 1;
}

template <int kT, int kMax, int kR>
__global__ void __launch_bounds__(kMax)
norm_forward_ring_kernel(const ForwardArgs a, int row_bytes) {
  constexpr int kVals = 16 / elem_bytes<kT>(), kUnits = kThreadValues / kVals;
  constexpr bool kKeep = kMax <= kMaxThreads / 2;
  extern __shared__ __align__(128) uint8_t s_rows[];
  __shared__ __align__(8) uint64_t s_bars[kSets];
  __shared__ __align__(16) float s_red[2][32][kR];
  __shared__ int s_fail;
  const int threads = blockDim.x, t = threadIdx.x;
  const int64_t step = static_cast<int64_t>(gridDim.x) * kR, ld = a.ldx * elem_bytes<kT>();
  RowRing<kR, 1> ring{s_bars, s_rows, row_bytes};
  const auto fill = [&](int set, int64_t r) {
    if (t == 0 && r < a.rows)
      ring.fill(set, a.rows - r < kR ? static_cast<int>(a.rows - r) : kR, static_cast<const char*>(a.x) + r * ld, ld, nullptr, 0);
  };
  s_fail = 0;
  ring.init();
  wait_for_inputs();
  let_next_begin();
  int64_t row = static_cast<int64_t>(blockIdx.x) * kR;
  fill(0, row);
  const auto gamma_at = [&](int c) { return make_float2(vector_at<kT>(a.gamma, c, 1.0f), vector_at<kT>(a.gamma, c + 1, 1.0f)); };
  const auto beta_at = [&](int c) { return make_float2(vector_at<kT>(a.beta, c, 0.0f), vector_at<kT>(a.beta, c + 1, 0.0f)); };
  float2 g[kKeep ? kThreadValues / 2 : 1], b[kKeep ? kThreadValues / 2 : 1];
  if constexpr (kKeep) {
#pragma unroll
    for (int i = 0; i < kUnits; ++i)
#pragma unroll
      for (int k = 0; k < kVals / 2; ++k) {
        const int c = (i * threads + t) * kVals, e = i * kVals / 2 + k;
        g[e] = c < a.width ? gamma_at(c + 2 * k) : both(0.0f);
        b[e] = c < a.width ? beta_at(c + 2 * k) : both(0.0f);
      }
  }
  const float width = static_cast<float>(a.width);
  int turn = 0;
  for (; row < a.rows; row += step) {
    ring.wait(&s_fail);
    float mean[kR], s[kR];
#pragma unroll
    for (int r = 0; r < kR; ++r) {
      Part<kT, kVals> x;
      x.load_shared(ring.row(r, 0), a.width, t, threads);
      float2 sum = both(0.0f);
#pragma unroll
      for (int i = 0; i < kUnits; ++i)
#pragma unroll
        for (int k = 0; k < kVals / 2; ++k) sum = add2(sum, x.two(i, k));
      s[r] = __fadd_rn(sum.x, sum.y);
    }
    cta_sum<kR>(s, s_red, turn);
    fill(ring.s ^ 1, row + step);  // behind the barrier all threads are done with the set before
#pragma unroll
    for (int r = 0; r < kR; ++r) {
      mean[r] = __fdiv_rn(s[r], width);
      const float2 less = both(-mean[r]);
      float2 sum = both(0.0f);
      Part<kT, kVals> x;
      x.load_shared(ring.row(r, 0), a.width, t, threads);
#pragma unroll
      for (int i = 0; i < kUnits; ++i) {
        if ((i * threads + t) * kVals >= a.width) continue;
#pragma unroll
        for (int k = 0; k < kVals / 2; ++k) {
          const float2 d = add2(x.two(i, k), less);
          sum = fma2(d, d, sum);
        }
      }
      s[r] = __fadd_rn(sum.x, sum.y);
    }
    cta_sum<kR>(s, s_red, turn);
#pragma unroll
    for (int r = 0; r < kR; ++r) {
      if (row + r >= a.rows) break;
      const float rstd = __fdiv_rn(1.0f, __fsqrt_rn(__fadd_rn(__fdiv_rn(s[r], width), a.eps)));
      if (t == 0) {
        if (a.mean) a.mean[row + r] = mean[r];
        if (a.rstd) a.rstd[row + r] = rstd;
      }
      char* const y = static_cast<char*>(a.y) + (row + r) * row_bytes;
      Part<kT, kVals> x;
      x.load_shared(ring.row(r, 0), a.width, t, threads);
#pragma unroll
      for (int i = 0; i < kUnits; ++i) {
        const int c = (i * threads + t) * kVals;
        if (c >= a.width) continue;
        float out[kVals];
#pragma unroll
        for (int k = 0; k < kVals / 2; ++k) {
          const int e = i * kVals / 2 + k;
          const float2 xh = mul2(add2(x.two(i, k), both(-mean[r])), both(rstd));
          const float2 o = fma2(xh, kKeep ? g[kKeep ? e : 0] : gamma_at(c + 2 * k), kKeep ? b[kKeep ? e : 0] : beta_at(c + 2 * k));
          out[2 * k] = o.x;
          out[2 * k + 1] = o.y;
        }
        store_unit<kT, kVals>(y, c, out);
      }
    }
    ring.next();
  }
  if (s_fail) let_copies_land();
}

template <int kT, int kMax, int kR>
__global__ void __launch_bounds__(kMax)
norm_backward_ring_kernel(const BackwardArgs a, int row_bytes) {
  constexpr int kVals = 16 / elem_bytes<kT>(), kUnits = kThreadValues / kVals;
  extern __shared__ __align__(128) uint8_t s_rows[];
  __shared__ __align__(8) uint64_t s_bars[kSets];
  __shared__ __align__(16) float s_red[2][32][2 * kR];
  __shared__ int s_fail;
  const int threads = blockDim.x, t = threadIdx.x;
  const int64_t step = static_cast<int64_t>(gridDim.x) * kR, ldx = a.ldx * elem_bytes<kT>(), lddy = a.lddy * elem_bytes<kT>();
  RowRing<kR, 2> ring{s_bars, s_rows, row_bytes};
  const auto fill = [&](int set, int64_t r) {
    if (t == 0 && r < a.rows)
      ring.fill(set, a.rows - r < kR ? static_cast<int>(a.rows - r) : kR, static_cast<const char*>(a.x) + r * ldx, ldx,
                static_cast<const char*>(a.dy) + r * lddy, lddy);
  };
  s_fail = 0;
  ring.init();
  wait_for_inputs();
  let_next_begin();
  int64_t row = static_cast<int64_t>(blockIdx.x) * kR;
  fill(0, row);
  float next_mean[kR], next_rstd[kR];
  const auto statistics = [&](int64_t first) {
#pragma unroll
    for (int r = 0; r < kR; ++r) {
      const bool in = first + r < a.rows;
      next_mean[r] = in ? a.mean[first + r] : 0.0f;
      next_rstd[r] = in ? a.rstd[first + r] : 0.0f;
    }
  };
  statistics(row);
  float2 g[kThreadValues / 2], dg[kThreadValues / 2], db[kThreadValues / 2];
#pragma unroll
  for (int i = 0; i < kUnits; ++i)
#pragma unroll
    for (int k = 0; k < kVals / 2; ++k) {
      const int c = (i * threads + t) * kVals + 2 * k, e = i * kVals / 2 + k;
      g[e] = c < a.width ? make_float2(vector_at<kT>(a.gamma, c, 1.0f), vector_at<kT>(a.gamma, c + 1, 1.0f)) : both(0.0f);
      dg[e] = db[e] = both(0.0f);
    }
  const float width = static_cast<float>(a.width);
  int turn = 0;
  for (; row < a.rows; row += step) {
    float mean[kR], rstd[kR], s[2 * kR];
#pragma unroll
    for (int r = 0; r < kR; ++r) { mean[r] = next_mean[r]; rstd[r] = next_rstd[r]; }
    statistics(row + step);
    ring.wait(&s_fail);
#pragma unroll
    for (int r = 0; r < kR; ++r) {
      s[2 * r] = s[2 * r + 1] = 0.0f;
      if (row + r >= a.rows) continue;
      const float2 less = both(-mean[r]), scale = both(rstd[r]);
      float2 s0 = both(0.0f), s1 = both(0.0f);
      Part<kT, kVals> x, dy;
      x.load_shared(ring.row(r, 0), a.width, t, threads);
      dy.load_shared(ring.row(r, 1), a.width, t, threads);
#pragma unroll
      for (int i = 0; i < kUnits; ++i) {
        if ((i * threads + t) * kVals >= a.width) continue;
#pragma unroll
        for (int k = 0; k < kVals / 2; ++k) {
          const int e = i * kVals / 2 + k;
          const float2 d = dy.two(i, k), xh = mul2(add2(x.two(i, k), less), scale), h = mul2(d, g[e]);
          dg[e] = fma2(d, xh, dg[e]);
          db[e] = add2(db[e], d);
          s0 = add2(s0, h);
          s1 = fma2(h, xh, s1);
        }
      }
      s[2 * r] = __fadd_rn(s0.x, s0.y);
      s[2 * r + 1] = __fadd_rn(s1.x, s1.y);
    }
    cta_sum<2 * kR>(s, s_red, turn);
    fill(ring.s ^ 1, row + step);  // behind the barrier all threads are done with the set before
#pragma unroll
    for (int r = 0; r < kR; ++r) {
      if (!a.dx || row + r >= a.rows) break;
      const float mean_h = __fdiv_rn(s[2 * r], width), mean_hx = __fdiv_rn(s[2 * r + 1], width);
      char* const dx = static_cast<char*>(a.dx) + (row + r) * row_bytes;
      Part<kT, kVals> x, dy;
      x.load_shared(ring.row(r, 0), a.width, t, threads);
      dy.load_shared(ring.row(r, 1), a.width, t, threads);
#pragma unroll
      for (int i = 0; i < kUnits; ++i) {
        const int c = (i * threads + t) * kVals;
        if (c >= a.width) continue;
        float out[kVals];
#pragma unroll
        for (int k = 0; k < kVals / 2; ++k) {
          const float2 xh = mul2(add2(x.two(i, k), both(-mean[r])), both(rstd[r])), h = mul2(dy.two(i, k), g[i * kVals / 2 + k]);
          const float2 o = mul2(both(rstd[r]), fma2(xh, both(-mean_hx), add2(h, both(-mean_h))));
          out[2 * k] = o.x;
          out[2 * k + 1] = o.y;
        }
        store_unit<kT, kVals>(dx, c, out);
      }
    }
    ring.next();
  }
  if (s_fail) let_copies_land();
  if (!a.partial) return;
  float* const to_gamma = a.partial + static_cast<int64_t>(blockIdx.x) * a.width;
  float* const to_beta = to_gamma + static_cast<int64_t>(gridDim.x) * a.width;
#pragma unroll
  for (int i = 0; i < kUnits; ++i)
#pragma unroll
    for (int j = 0; j < kVals; j += 4) {
      const int c = (i * threads + t) * kVals + j, e = (i * kVals + j) / 2;
      if (c >= a.width) continue;
      *reinterpret_cast<float4*>(to_gamma + c) = make_float4(dg[e].x, dg[e].y, dg[e + 1].x, dg[e + 1].y);
      *reinterpret_cast<float4*>(to_beta + c) = make_float4(db[e].x, db[e].y, db[e + 1].x, db[e + 1].y);
    }
}

// Sums of the CTAs' rows: sixteen warps of a CTA each add every sixteenth of
// 32 columns' rows, in order, and the first then adds the sixteen.
constexpr int kSumWarps = 16;

struct SumArgs {
  const float* partial;
  int64_t parts;
  int width;
  void* out[2];  // dgamma and dbeta, or null
  int type[2];
};

__global__ void __launch_bounds__(32 * kSumWarps)
norm_sums_kernel(const SumArgs a) {
  __shared__ float s_part[kSumWarps][32];
  wait_for_inputs();
  let_next_begin();
  void* const out = a.out[blockIdx.y];
  if (!out) return;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, c = blockIdx.x * 32 + lane;
  const float* const from = a.partial + blockIdx.y * a.parts * a.width;
  float s = 0.0f;
  if (c < a.width) {
#pragma unroll 16
    for (int64_t p = warp; p < a.parts; p += kSumWarps) s += from[p * a.width + c];
  }
  s_part[warp][lane] = s;
  __syncthreads();
  if (warp != 0 || c >= a.width) return;
#pragma unroll
  for (int w = 1; w < kSumWarps; ++w) s += s_part[w][lane];
  const int type = a.type[blockIdx.y];
  if (type == kF32) store1<kF32>(out, c, s);
  else if (type == kBF16) store1<kBF16>(out, c, s);
  else store1<kF16>(out, c, s);
}

// --------------------------------------------------------------------------
// host side

bool valid_type(int t) { return t == BWD_F32 || t == BWD_BF16 || t == BWD_F16; }
int bytes_of(int t) { return t == BWD_F32 ? 4 : 2; }

constexpr int kSms = 160;  // at least as many as the device has

int threads_of(int width) { return (width + 32 * kThreadValues - 1) / (32 * kThreadValues) * 32; }

// CTAs of the backward pass, and so rows of its workspace, at most: as many as
// are resident (some 100 registers to a thread), each with two rows or more,
// since every one adds a row of sums.
int64_t backward_ctas(int64_t rows, int width, int sms) {
  const bool warp = width <= kWarpWidth;
  const int threads = warp ? 32 * kWarps : threads_of(width);
  const int64_t most = static_cast<int64_t>(sms) * std::max(1, std::min(512 / threads, 8));
  const int64_t each = 2 * (warp ? kWarps : 1), need = (rows + each - 1) / each;
  return std::min(need, most);
}

// Rows that a CTA of the ring kernels takes at a time, of so many bytes in
// all arrays, where `ctas` share an SM's shared memory: at most `most`, no more
// than gives each CTA several sets; 0 where not even one row fits twice.
int rows_at_a_time(int64_t row_bytes, int ctas, int64_t rows_each, int most) {
  for (int r = most; r >= 1; r /= 2)
    if (kSets * r * row_bytes * ctas <= 200 << 10 && rows_each >= 2 * r) return r;
  return 0;
}

template <typename... Params, typename... Args>
bwd_status launch_ring(void (*kernel)(Params...), int64_t ctas, int threads, int smem, cudaStream_t st, const char* what, const Args&... args) {
  if (smem > 48 * 1024) {
    const cudaError_t e = opt_in(kernel, 200 << 10);
    if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute(MaxDynamicSharedMemorySize)");
  }
  return launch_ex(kernel, dim3(static_cast<unsigned>(ctas)), threads, 0, smem, st, what, args...);
}

bwd_status sm_count(int* out) {
  static std::atomic<int> known[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess && dev >= 0 && dev < 64 && (*out = known[dev].load(std::memory_order_relaxed)) > 0) return BWD_OK;
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(out, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return cuda_fail(e, "cudaDeviceGetAttribute");
  if (*out > kSms) *out = kSms;
  if (dev >= 0 && dev < 64) known[dev].store(*out, std::memory_order_relaxed);
  return BWD_OK;
}

// Values of the largest unit that all of a call's rows consist of and start on.
int unit_values(int eb, uintptr_t addresses, int64_t row_bytes) {
  const uintptr_t all = addresses | static_cast<uintptr_t>(row_bytes);
  const int bytes = all % 16 == 0 ? 16 : all % 8 == 0 ? 8 : all % 4 == 0 ? 4 : 2;
  return bytes / eb;
}

template <template <int, int, bool, int> class Launch, typename Args, typename... More>
bwd_status by_type(int type, int values, int width, const Args& a, More... more) {
  const auto sized = [&](auto t, auto v) {
    constexpr int kT = decltype(t)::value, kVals = decltype(v)::value;
    if (width <= kWarpWidth) return Launch<kT, kVals, true, 32 * kWarps>::go(a, more...);
    const int threads = threads_of(width);
    if (threads <= kMaxThreads / 4) return Launch<kT, kVals, false, kMaxThreads / 4>::go(a, more...);
    if (threads <= kMaxThreads / 2) return Launch<kT, kVals, false, kMaxThreads / 2>::go(a, more...);
    return Launch<kT, kVals, false, kMaxThreads>::go(a, more...);
  };
  const auto typed = [&](auto t) {
    constexpr int kT = decltype(t)::value;
    if constexpr (kT != kF32)
      if (values == 8) return sized(t, std::integral_constant<int, 8>{});
    if (values == 4) return sized(t, std::integral_constant<int, 4>{});
    if (values == 2) return sized(t, std::integral_constant<int, 2>{});
    return sized(t, std::integral_constant<int, 1>{});
  };
  if (type == BWD_F32) return typed(std::integral_constant<int, kF32>{});
  if (type == BWD_BF16) return typed(std::integral_constant<int, kBF16>{});
  return typed(std::integral_constant<int, kF16>{});
}

template <int kT, int kVals, bool kWarp, int kMax>
struct LaunchForward {
  static bwd_status go(const ForwardArgs& a, int sms, cudaStream_t st) {
    constexpr bool kPieces = kVals * elem_bytes<kT>() == 16 && !kWarp;
    const int threads = kWarp ? 32 * kWarps : threads_of(a.width), per_sm = std::max(1, std::min(768 / threads, 8));
    const int64_t most = static_cast<int64_t>(sms) * per_sm, need = kWarp ? (a.rows + kWarps - 1) / kWarps : a.rows;
    const int64_t ctas = std::min(need, most);
    if constexpr (kPieces) {
      const int row_bytes = a.width * elem_bytes<kT>(), r = rows_at_a_time(row_bytes, per_sm, a.rows / ctas, 4);
      const auto go = [&](auto* kernel) {
        return launch_ring(kernel, ctas, threads, kSets * r * row_bytes, st, "norm_forward_ring_kernel launch", a, row_bytes);
      };
      if (r == 4) return go(norm_forward_ring_kernel<kT, kMax, 4>);
      if (r == 2) return go(norm_forward_ring_kernel<kT, kMax, 2>);
      if (r == 1) return go(norm_forward_ring_kernel<kT, kMax, 1>);
    }
    return launch_ex(norm_forward_kernel<kT, kVals, kWarp, kMax>, dim3(static_cast<unsigned>(ctas)), threads, 0, 0, st,
                     "norm_forward_kernel launch", a);
  }
};

template <int kT, int kVals, bool kWarp, int kMax>
struct LaunchBackward {
  static bwd_status go(const BackwardArgs& a, int64_t ctas, cudaStream_t st) {
    constexpr bool kKeep = kMax <= kMaxThreads / 2, kPieces = kVals * elem_bytes<kT>() == 16 && !kWarp && kKeep;
    const int threads = kWarp ? 32 * kWarps : threads_of(a.width), per_sm = std::max(1, std::min(512 / threads, 8));
    if constexpr (kPieces) {
      // (the partial sums go out in pieces of 16 bytes too)
      const int row_bytes = a.width * elem_bytes<kT>(), r = aligned16(a.partial) ? rows_at_a_time(2 * row_bytes, per_sm, a.rows / ctas, 2) : 0;
      const auto go = [&](auto* kernel) {
        return launch_ring(kernel, ctas, threads, kSets * r * 2 * row_bytes, st, "norm_backward_ring_kernel launch", a, row_bytes);
      };
      if (r == 2) return go(norm_backward_ring_kernel<kT, kMax, 2>);
      if (r == 1) return go(norm_backward_ring_kernel<kT, kMax, 1>);
    }
    const int smem = a.partial && (kWarp || !kKeep) ? 8 * a.width : 0;
    return launch_ring(norm_backward_kernel<kT, kVals, kWarp, kMax>, ctas, threads, smem, st, "norm_backward_kernel launch", a);
  }
};

constexpr int64_t kMaxRows = int64_t{1} << 31;

bwd_status check_size(int64_t rows, int64_t width, bwd_dtype dtype, bwd_dtype vector_dtype) {
  if (!valid_type(dtype)) return fail(BWD_ERR_UNSUPPORTED_DTYPE, "dtype %d", (int)dtype);
  if (vector_dtype != BWD_F32 && vector_dtype != dtype) return fail(BWD_ERR_UNSUPPORTED_DTYPE, "gamma and beta are fp32 or of x's type");
  if (rows < 0 || rows > kMaxRows || width < 1 || width > kMaxWidth)
    return fail(BWD_ERR_INVALID_ARG, "bad size: a row has 1 to %d elements", kMaxWidth);
  return BWD_OK;
}

}  // namespace

namespace bwd {
namespace host {

bwd_status take_norm_fault(unsigned int* fault) { return take_wait_fault(fault); }

}  // namespace host
}  // namespace bwd

extern "C" {

bwd_status bwd_norm_forward(const void* x, bwd_dtype dtype, int64_t rows, int64_t width, int64_t ldx, const void* gamma, const void* beta,
                            bwd_dtype vector_dtype, float eps, void* y, float* mean, float* rstd, void* stream) {
  bwd_status s = check_size(rows, width, dtype, vector_dtype);
  if (s != BWD_OK) return s;
  if (ldx < width) return fail(BWD_ERR_INVALID_ARG, "ldx is less than width");
  if (!(eps >= 0.0f)) return fail(BWD_ERR_INVALID_ARG, "eps must be >= 0");
  if (rows == 0) return BWD_OK;
  const int eb = bytes_of(dtype), vb = bytes_of(vector_dtype);
  if (!x || !y) return fail(BWD_ERR_INVALID_ARG, "NULL pointer");
  if (!aligned_to(x, eb) || !aligned_to(y, eb) || !aligned_to(gamma, vb) || !aligned_to(beta, vb) || !aligned_to(mean, 4) || !aligned_to(rstd, 4))
    return fail(BWD_ERR_INVALID_ARG, "pointer not aligned to its element size");
  int sms = 0;
  if ((s = sm_count(&sms)) != BWD_OK) return s;
  const int f32 = vector_dtype == BWD_F32;
  const ForwardArgs a{x, ldx, {gamma, f32}, {beta, f32}, y, mean, rstd, rows, static_cast<int>(width), eps};
  const int values = unit_values(eb, reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(y), (ldx | width) * eb);
  return by_type<LaunchForward>(dtype, values, a.width, a, sms, static_cast<cudaStream_t>(stream));
}

int64_t bwd_norm_backward_work_bytes(int64_t rows, int64_t width) {
  if (rows < 0 || rows > kMaxRows || width < 1 || width > kMaxWidth) return -1;
  return 8 * backward_ctas(rows, static_cast<int>(width), kSms) * width;
}

bwd_status bwd_norm_backward(const void* dy, const void* x, bwd_dtype dtype, int64_t rows, int64_t width, int64_t lddy, int64_t ldx,
                             const void* gamma, bwd_dtype vector_dtype, const float* mean, const float* rstd, void* dx, void* dgamma,
                             void* dbeta, void* work, void* stream) {
  bwd_status s = check_size(rows, width, dtype, vector_dtype);
  if (s != BWD_OK) return s;
  if (lddy < width || ldx < width) return fail(BWD_ERR_INVALID_ARG, "lddy or ldx is less than width");
  const int eb = bytes_of(dtype), vb = bytes_of(vector_dtype);
  if (!aligned_to(dy, eb) || !aligned_to(x, eb) || !aligned_to(dx, eb) || !aligned_to(gamma, vb) || !aligned_to(dgamma, vb) ||
      !aligned_to(dbeta, vb) || !aligned_to(mean, 4) || !aligned_to(rstd, 4) || !aligned_to(work, 4))
    return fail(BWD_ERR_INVALID_ARG, "pointer not aligned to its element size");
  const bool sums = dgamma || dbeta;
  if (rows > 0 && (dx || sums) && (!dy || !x || !mean || !rstd || (sums && !work))) return fail(BWD_ERR_INVALID_ARG, "NULL pointer");
  if (!dx && !sums) return BWD_OK;
  int sms = 0;
  if ((s = sm_count(&sms)) != BWD_OK) return s;
  const int64_t ctas = backward_ctas(rows, static_cast<int>(width), sms);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (rows > 0) {
    const BackwardArgs a{dy, x, lddy, ldx, {gamma, vector_dtype == BWD_F32}, mean, rstd, dx, sums ? static_cast<float*>(work) : nullptr, rows,
                         static_cast<int>(width)};
    const int values = unit_values(eb, reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(dy) | reinterpret_cast<uintptr_t>(dx),
                                   (ldx | lddy | width) * eb);
    if ((s = by_type<LaunchBackward>(dtype, values, a.width, a, ctas, st)) != BWD_OK) return s;
  }
  if (!sums) return BWD_OK;
  const SumArgs a{static_cast<const float*>(work), rows > 0 ? ctas : 0, static_cast<int>(width), {dgamma, dbeta}, {vector_dtype, vector_dtype}};
  return launch_ex(norm_sums_kernel, dim3(static_cast<unsigned>((width + 31) / 32), 2), 32 * kSumWarps, 0, 0, st, "norm_sums_kernel launch", a);
}

}  // extern "C"
