// Layer normalisation over the rows of a matrix, forward and backward
// (sm_103a).
//
//   mean = sum x / D;  var = sum (x - mean)^2 / D;  rstd = (var + eps)^-1/2
//   xh = (x - mean) rstd;  y = xh gamma + beta
//   h = dy gamma;  dx = rstd (h - sum h / D - xh sum(h xh) / D)
//   dgamma = sum over rows of dy xh;  dbeta = sum over rows of dy
//
// Each row is read once: a group of threads (a warp, or a CTA) holds it, in
// registers or in shared memory, forms the sums and writes the result.  The
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
constexpr int kMaxThreads = 512;
// Values of a row that a thread holds: 16, and 32 of rows that would need more
// than kMaxThreads threads so.
constexpr int kFew = 16, kMany = 32;
static_assert(kMaxThreads * kMany == kMaxWidth, "a CTA holds a row");

template <int kBytes> struct UnitOf;
template <> struct UnitOf<16> { using T = uint4; };
template <> struct UnitOf<8> { using T = uint2; };
template <> struct UnitOf<4> { using T = uint32_t; };
template <> struct UnitOf<2> { using T = uint16_t; };

// A thread's part of a row: units of kVals consecutive values, a group's
// threads side by side.
template <int kT, int kVals, int kValues>
struct Part {
  static constexpr int kUnits = kValues / kVals;
  using Unit = typename UnitOf<kVals * elem_bytes<kT>()>::T;
  Unit u[kUnits];

  __device__ __forceinline__ void load(const void* row, int width, int t, int threads) {
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
      const int c = (i * threads + t) * kVals;
      u[i] = c < width ? __ldcs(reinterpret_cast<const Unit*>(static_cast<const char*>(row) + static_cast<int64_t>(c) * elem_bytes<kT>())) : Unit{};
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

// What the kernels for few rows and those for many make of a row's sums, so that
// they make the same of the same sums.
//
// s / width, rounded to nearest, for inv = RN(1 / width): the quotient's
// remainder is exact in one fused multiply-add, and one step with it rounds
// correctly (Markstein 1990) where nothing underflows, for sums above 2^-100.
// (A product with 1 / width alone is a unit, 2^-14, off for a thousand 1000.0,
// and y 0.019, as rstd is 316.)
__device__ __forceinline__ float per_width(float s, float width, float inv) {
  const float q = __fmul_rn(s, inv), r = __fmaf_rn(__fmaf_rn(-width, q, s), inv, q);
  return fabsf(q) <= 3.402823466e38f ? r : q;
}
// (var + eps)^-1/2: rsqrtf is up to two units off, one step of Newton's method
// leaves less than one.  (A correctly rounded root and quotient, 16384 x 4096
// bf16: 51.4 us forward, 47.2 so; 45.7 with rsqrtf alone and the product above.)
__device__ __forceinline__ float rstd_of(float var, float eps) {
  const float x = __fadd_rn(var, eps), y = rsqrtf(x), e = __fmaf_rn(-__fmul_rn(x, y), y, 1.0f);
  return fabsf(e) <= 1.0f ? __fmaf_rn(__fmul_rn(0.5f, y), e, y) : y;
}

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

template <int kT, int kVals, int kValues, bool kWarp>
__global__ void __launch_bounds__(kWarp ? 32 * kWarps : kMaxThreads)
norm_forward_kernel(const ForwardArgs a) {
  constexpr int kUnits = kValues / kVals;
  __shared__ float s_red[2][2][32];
  const int threads = kWarp ? 32 : blockDim.x, t = kWarp ? threadIdx.x % 32 : threadIdx.x;
  const int64_t groups = kWarp ? static_cast<int64_t>(gridDim.x) * kWarps : gridDim.x;
  int64_t row = kWarp ? static_cast<int64_t>(blockIdx.x) * kWarps + threadIdx.x / 32 : blockIdx.x;
  GroupSum<kWarp, 1> sum{s_red};
  const auto x_row = [&](int64_t r) { return static_cast<const char*>(a.x) + r * a.ldx * elem_bytes<kT>(); };
  wait_for_inputs();
  let_next_begin();
  Part<kT, kVals, kValues> next;
  if (row < a.rows) next.load(x_row(row), a.width, t, threads);
  float g[kValues], b[kValues];
#pragma unroll
  for (int i = 0; i < kUnits; ++i)
#pragma unroll
    for (int j = 0; j < kVals; ++j) {
      const int c = (i * threads + t) * kVals;
      g[i * kVals + j] = c < a.width ? vector_at<kT>(a.gamma, c + j, 1.0f) : 0.0f;
      b[i * kVals + j] = c < a.width ? vector_at<kT>(a.beta, c + j, 0.0f) : 0.0f;
    }
  const float width = static_cast<float>(a.width), inv_width = __fdiv_rn(1.0f, width);
  for (; row < a.rows; row += groups) {
    float v[kValues];
    float s[1] = {0.0f};
#pragma unroll
    for (int i = 0; i < kUnits; ++i)
#pragma unroll
      for (int j = 0; j < kVals; ++j) s[0] += v[i * kVals + j] = next.value(i, j);
    if (row + groups < a.rows) next.load(x_row(row + groups), a.width, t, threads);
    sum(s);
    const float mean = per_width(s[0], width, inv_width);
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
    const float rstd = rstd_of(per_width(s[0], width, inv_width), a.eps);
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
        out[j] = __fmaf_rn(__fmul_rn(v[e], rstd), g[e], b[e]);
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

template <int kT, int kVals, int kValues, bool kWarp>
__global__ void __launch_bounds__(kWarp ? 32 * kWarps : kMaxThreads)
norm_backward_kernel(const BackwardArgs a) {
  constexpr int kUnits = kValues / kVals;
  __shared__ float s_sums[kWarp ? 2 * kWarpWidth : 1];  // of a CTA's warps
  __shared__ float s_red[2][2][32];
  const int threads = kWarp ? 32 : blockDim.x, t = kWarp ? threadIdx.x % 32 : threadIdx.x;
  const int64_t groups = kWarp ? static_cast<int64_t>(gridDim.x) * kWarps : gridDim.x;
  int64_t row = kWarp ? static_cast<int64_t>(blockIdx.x) * kWarps + threadIdx.x / 32 : blockIdx.x;
  GroupSum<kWarp, 2> sum{s_red};
  const auto x_row = [&](int64_t r) { return static_cast<const char*>(a.x) + r * a.ldx * elem_bytes<kT>(); };
  const auto dy_row = [&](int64_t r) { return static_cast<const char*>(a.dy) + r * a.lddy * elem_bytes<kT>(); };
  wait_for_inputs();
  let_next_begin();
  Part<kT, kVals, kValues> next_x, next_dy;
  float next_mean = 0.0f, next_rstd = 0.0f;
  const auto fetch = [&](int64_t r) {
    next_x.load(x_row(r), a.width, t, threads);
    next_dy.load(dy_row(r), a.width, t, threads);
    next_mean = a.mean[r];
    next_rstd = a.rstd[r];
  };
  if (row < a.rows) fetch(row);
  float g[kValues], dg[kValues], db[kValues];
#pragma unroll
  for (int i = 0; i < kUnits; ++i)
#pragma unroll
    for (int j = 0; j < kVals; ++j) {
      const int c = (i * threads + t) * kVals, e = i * kVals + j;
      g[e] = c < a.width ? vector_at<kT>(a.gamma, c + j, 1.0f) : 0.0f;
      dg[e] = db[e] = 0.0f;
    }
  const float width = static_cast<float>(a.width), inv_width = __fdiv_rn(1.0f, width);
  for (; row < a.rows; row += groups) {
    const Part<kT, kVals, kValues> x = next_x, dy = next_dy;
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
        dg[e] = __fmaf_rn(d, xh, dg[e]);
        db[e] = __fadd_rn(db[e], d);
        const float h = __fmul_rn(d, g[e]);
        s[0] += h;
        s[1] = __fmaf_rn(h, xh, s[1]);
      }
    }
    if (!a.dx) continue;
    sum(s);
    const float mean_h = per_width(s[0], width, inv_width), mean_hx = per_width(s[1], width, inv_width);
    char* const dx = static_cast<char*>(a.dx) + row * a.width * elem_bytes<kT>();
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
      const int c = (i * threads + t) * kVals;
      if (c >= a.width) continue;
      float out[kVals];
#pragma unroll
      for (int j = 0; j < kVals; ++j) {
        const float h = __fmul_rn(dy.value(i, j), g[i * kVals + j]);
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
              s_sums[c] = w ? __fadd_rn(s_sums[c], dg[e]) : dg[e];
              s_sums[kWarpWidth + c] = w ? __fadd_rn(s_sums[kWarpWidth + c], db[e]) : db[e];
            }
          }
      }
      __syncthreads();
    }
    for (int c = threadIdx.x; c < a.width; c += 32 * kWarps) {
      to_gamma[c] = s_sums[c];
      to_beta[c] = s_sums[kWarpWidth + c];
    }
  } else {
#pragma unroll
    for (int i = 0; i < kUnits; ++i)
#pragma unroll
      for (int j = 0; j < kVals; ++j) {
        const int c = (i * threads + t) * kVals + j;
        if (c >= a.width) continue;
        to_gamma[c] = dg[i * kVals + j];
        to_beta[c] = db[i * kVals + j];
      }
  }
}

// --------------------------------------------------------------------------
// many rows
//
// A CTA takes kR rows at a time: what a row costs beside its bytes is the
// latency of its sums over the CTA, which kR rows share.  Rows come into
// shared memory by bulk copies, up to three sets of kR ahead.  Each pass reads
// them from there, or (forward, up to 8192 columns in whole pieces) the first
// one alone; the registers hold gamma, beta and the columns' sums.
// (16384 x 4096 bf16, forward and backward, with a row at a time in registers:
// 58 and 97 us; from shared memory, a row at a time, 56 and 100, and these sets
// with one operation to an instruction 58 and 89, bound by instructions.)
//
// A copy's pieces have 16 bytes: of rows that start or end inside one, the
// whole pieces that they touch are copied, and the row starts where it does in
// the first.  What that reads beside a row belongs to the rows next to it; the
// first row's start and the last one's end are read by themselves.

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

// A thread's columns, in pairs: of whole pieces neighbours, 16 bytes to a unit;
// of other rows columns that lie a CTA apart, so that each access is a warp's
// worth of neighbours.
template <int kT, bool kPieces, int kValues>
struct Columns {
  static constexpr int kPairs = kValues / 2;
  static constexpr int kUnitPairs = kPieces ? 8 / elem_bytes<kT>() : kPairs;  // of a unit
  static_assert(kPairs % kUnitPairs == 0, "a thread holds whole units");
  int t, threads, width;
  __device__ __forceinline__ int first(int e) const {
    if constexpr (kPieces) return ((e / kUnitPairs * threads + t) * kUnitPairs + e % kUnitPairs) * 2;
    else return 2 * e * threads + t;
  }
  __device__ __forceinline__ int second(int e) const { return first(e) + (kPieces ? 1 : threads); }
  __device__ __forceinline__ float2 vector(const VectorArg& v, int e, float otherwise) const {
    const int c = first(e), d = second(e);
    return make_float2(c < width ? vector_at<kT>(v, c, otherwise) : 0.0f, d < width ? vector_at<kT>(v, d, otherwise) : 0.0f);
  }
  // Calls f(e, there, values of each row) for this thread's pairs of rows in
  // shared memory, and writes what it returns to `out`, where that is wanted.
  // A second value past the row is 0, and not `there`.
  template <bool kOut, int kN, typename F>
  __device__ __forceinline__ void over(char* out, const uint8_t* const (&row)[kN], F f) const {
    if constexpr (kPieces) {
      // all of a thread's loads before the first use, where registers allow it
      constexpr int kUnits = kPairs / kUnitPairs, kAtOnce = kValues == kFew ? kUnits : 1;
#pragma unroll
      for (int i0 = 0; i0 < kUnits; i0 += kAtOnce) {
        uint4 w[kAtOnce][kN];
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) {
          const int c = ((i0 + i) * threads + t) * 2 * kUnitPairs;
#pragma unroll
          for (int n = 0; n < kN; ++n)
            w[i][n] = c < width ? *reinterpret_cast<const uint4*>(row[n] + c * elem_bytes<kT>()) : make_uint4(0u, 0u, 0u, 0u);
        }
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) {
          const int c = ((i0 + i) * threads + t) * 2 * kUnitPairs;
          if (c >= width) continue;
          float o[2 * kUnitPairs];
#pragma unroll
          for (int k = 0; k < kUnitPairs; ++k) {
            float2 v[kN];
#pragma unroll
            for (int n = 0; n < kN; ++n) {
              Part<kT, 2 * kUnitPairs, 2 * kUnitPairs> x;
              x.u[0] = w[i][n];
              v[n] = x.two(0, k);
            }
            const float2 r = f((i0 + i) * kUnitPairs + k, true, v);
            o[2 * k] = r.x;
            o[2 * k + 1] = r.y;
          }
          if constexpr (kOut) store_unit<kT, 2 * kUnitPairs>(out, c, o);
        }
      }
    } else {
#pragma unroll
      for (int e = 0; e < kPairs; ++e) {
        const int c = first(e), d = second(e);
        if (c >= width) continue;
        const bool there = d < width;
        float2 v[kN];
#pragma unroll
        for (int n = 0; n < kN; ++n) v[n] = make_float2(load1<kT>(row[n], c), there ? load1<kT>(row[n], d) : 0.0f);
        const float2 r = f(e, there, v);
        if constexpr (kOut) {
          store1<kT>(out, c, r.x);
          if (there) store1<kT>(out, d, r.y);
        }
      }
    }
  }
};

constexpr int kMaxSets = 4;  // of rows, one of them being read

// One array's rows: where they are, and the whole pieces that they touch.
struct Rows {
  const char* base;
  int64_t ld;       // bytes
  int row_bytes;
  int64_t rows;
};

template <int kT, bool kPieces, int kR, int kArrays>
struct RowRing {
  uint64_t* bars;
  uint8_t* data;  // [sets][kR][kArrays][slot]
  int sets;
  int slot;       // bytes of a row's pieces
  Rows a[kArrays];
  int s = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ uint8_t* place(int set, int r, int array) const { return data + ((set * kR + r) * kArrays + array) * slot; }
  // Row r of the set that is being read, which is row `row` of the array.
  __device__ __forceinline__ const uint8_t* row(int r, int array, int64_t row) const {
    if constexpr (kPieces) return place(s, r, array);
    else return place(s, r, array) + (reinterpret_cast<uintptr_t>(a[array].base + row * a[array].ld) & 15u);
  }
  __device__ __forceinline__ void init() {
    if (threadIdx.x == 0) {
      for (int i = 0; i < sets; ++i) mbar_init(&bars[i], 1);
      asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncthreads();
  }
  // Rows `first` on into a set, by one thread, behind a barrier that all
  // threads passed when they were done with it.
  __device__ __forceinline__ void fill(int set, int64_t first) {
    if (threadIdx.x != 0 || first >= a[0].rows) return;
    const int count = a[0].rows - first < kR ? static_cast<int>(a[0].rows - first) : kR;
    uint32_t bytes = 0;
    for (int r = 0; r < count; ++r)
#pragma unroll
      for (int i = 0; i < kArrays; ++i) {
        const char* const from = a[i].base + (first + r) * a[i].ld;
        uint8_t* const dst = place(set, r, i);
        if constexpr (kPieces) {
          bulk_load(dst, from, a[i].row_bytes, &bars[set]);
          bytes += a[i].row_bytes;
        } else {
          bytes += pieces(dst, reinterpret_cast<uintptr_t>(from), a[i].row_bytes, first + r == 0, first + r + 1 == a[i].rows, &bars[set]);
        }
      }
    mbar_expect_tx(&bars[set], bytes);
  }
  static __device__ __forceinline__ uint32_t pieces(uint8_t* dst, uintptr_t from, int row_bytes, bool first, bool last, uint64_t* bar) {
    const uintptr_t to = from + row_bytes, start = from & ~uintptr_t{15};
    uintptr_t low = start, high = (to + 15) & ~uintptr_t{15};
    if (first || last) {
      // the first row's start and the last one's end, a value at a time
      using Elem = std::conditional_t<kT == kF32, uint32_t, uint16_t>;
      const auto copy = [&](uintptr_t at, uintptr_t end) {
        for (; at < end; at += sizeof(Elem)) *reinterpret_cast<Elem*>(dst + (at - start)) = *reinterpret_cast<const Elem*>(at);
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // a later row's copy writes here too
      };
      if (first && low != from) low += 16;
      if (last && high != to) high -= 16;
      if (low >= high) {
        copy(from, to);
        return 0;
      }
      if (first) copy(from, low);
      if (last) copy(high, to);
    }
    bulk_load(dst + (low - start), reinterpret_cast<const void*>(low), static_cast<uint32_t>(high - low), bar);
    return static_cast<uint32_t>(high - low);
  }
  // Waits for the current set.  Where a wait gives up, the CTA goes on over
  // whatever there is, with no wait any more, so that its barriers still meet.
  __device__ __forceinline__ void wait(volatile int* fail) { mbar_wait(&bars[s], phase, fail); }
  // The first sets, and later what takes the place of the set before this one.
  __device__ __forceinline__ void begin(int64_t row, int64_t step) {
    for (int i = 0; i + 1 < sets; ++i) fill(i, row + i * step);
  }
  __device__ __forceinline__ void refill(int64_t row, int64_t step) { fill(s == 0 ? sets - 1 : s - 1, row + (sets - 1) * step); }
  __device__ __forceinline__ void next() {
    if (++s == sets) { s = 0; phase ^= 1u; }
  }
};

// Sums of kN values over a CTA, the same in each of its threads; two buffers
// in turn, as for GroupSum.  Of several values lanes first divide which ones
// they go on with, so that four take six shuffles and not twenty.  (With those,
// and divisions by the width, a row cost a warp more instructions than its 512
// elements did.)
template <int kN>
__device__ __forceinline__ void cta_sum(float (&s)[kN], float (*red)[32][kN], int& turn) {
  static_assert(kN == 1 || kN == 2 || kN == 4, "values that lanes divide");
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, warps = blockDim.x / 32;
  int mine = 0;  // the value that this lane ends up with
  float a = s[0];
  if constexpr (kN == 4) {
    const bool high = lane & 16, odd = lane & 8;
    float a0 = high ? s[2] : s[0], a1 = high ? s[3] : s[1];
    a0 += __shfl_xor_sync(0xffffffffu, high ? s[0] : s[2], 16);
    a1 += __shfl_xor_sync(0xffffffffu, high ? s[1] : s[3], 16);
    a = (odd ? a1 : a0) + __shfl_xor_sync(0xffffffffu, odd ? a0 : a1, 8);
    mine = lane >> 3;
  } else if constexpr (kN == 2) {
    const bool high = lane & 16;
    a = (high ? s[1] : s[0]) + __shfl_xor_sync(0xffffffffu, high ? s[0] : s[1], 16);
    a += __shfl_xor_sync(0xffffffffu, a, 8);
    mine = lane >> 4;
  } else {
    a += __shfl_xor_sync(0xffffffffu, a, 16);
    a += __shfl_xor_sync(0xffffffffu, a, 8);
  }
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
  if (lane % (32 / kN) == 0) red[turn][warp][mine] = a;
  __syncthreads();
  const float* const from = red[turn][0];
#pragma unroll
  for (int n = 0; n < kN; ++n) s[n] = 0.0f;
#pragma unroll 4
  for (int w = 0; w < warps; ++w) {
    if constexpr (kN == 4) {
      const float4 v = *reinterpret_cast<const float4*>(from + 4 * w);
      s[0] += v.x; s[1] += v.y; s[2] += v.z; s[3] += v.w;
    } else {
#pragma unroll
      for (int n = 0; n < kN; ++n) s[n] += from[kN * w + n];
    }
  }
  turn ^= 1;
}

template <int kT, bool kPieces, int kValues, int kMax, int kR>
__global__ void __launch_bounds__(kMax)
norm_forward_ring_kernel(const ForwardArgs a, int slot, int sets) {
  constexpr int kPairs = kValues / 2;
  constexpr bool kKeep = kPieces && kValues == kFew;
  extern __shared__ __align__(128) uint8_t s_rows[];
  __shared__ __align__(8) uint64_t s_bars[kMaxSets];
  __shared__ __align__(16) float s_red[2][32][kR];
  __shared__ int s_fail;
  const Columns<kT, kPieces, kValues> cols{static_cast<int>(threadIdx.x), static_cast<int>(blockDim.x), a.width};
  const int64_t step = static_cast<int64_t>(gridDim.x) * kR;
  const int row_bytes = a.width * elem_bytes<kT>();
  RowRing<kT, kPieces, kR, 1> ring{s_bars, s_rows, sets, slot, {{static_cast<const char*>(a.x), a.ldx * elem_bytes<kT>(), row_bytes, a.rows}}};
  s_fail = 0;
  ring.init();
  wait_for_inputs();
  let_next_begin();
  int64_t row = static_cast<int64_t>(blockIdx.x) * kR;
  ring.begin(row, step);
  float2 g[kPairs], b[kPairs];
#pragma unroll
  for (int e = 0; e < kPairs; ++e) {
    g[e] = cols.vector(a.gamma, e, 1.0f);
    b[e] = cols.vector(a.beta, e, 0.0f);
  }
  if constexpr (!kPieces) __syncthreads();  // the first row's start, which a thread copied
  const float width = static_cast<float>(a.width), inv_width = __fdiv_rn(1.0f, width);
  int turn = 0;
  for (; row < a.rows; row += step) {
    ring.wait(&s_fail);
    float mean[kR], s[kR];
    if constexpr (kKeep) {
      // A row's values stay in registers, widened once.  (16384 x 4096 bf16 45
      // us, 49.4 with four rows read anew and widened by each pass, 56 with one
      // row in registers; 8192 x 8192 bf16 50.3 and 60.1; 16384 x 768 fp32 15.9
      // and 23.9.  The backward pass, which would hold twice as much, gains
      // nothing: 75.8 and 75.1.)
      constexpr int kUnitPairs = Columns<kT, kPieces, kValues>::kUnitPairs;
      float2 v[kR][kPairs];
#pragma unroll
      for (int r = 0; r < kR; ++r) {
        float2 sum = both(0.0f);
#pragma unroll
        for (int e = 0; e < kPairs; ++e) v[r][e] = both(0.0f);
        cols.template over<false, 1>(nullptr, {ring.row(r, 0, row + r)}, [&](int e, bool, const float2 (&x)[1]) {
          v[r][e] = x[0];
          return sum = add2(sum, x[0]);
        });
        s[r] = __fadd_rn(sum.x, sum.y);
      }
      cta_sum<kR>(s, s_red, turn);
      ring.refill(row, step);
#pragma unroll
      for (int r = 0; r < kR; ++r) {
        mean[r] = per_width(s[r], width, inv_width);
        const float2 less = both(-mean[r]);
        float2 sum = both(0.0f);
#pragma unroll
        for (int e = 0; e < kPairs; ++e) {
          if (cols.first(e) < a.width) {
            v[r][e] = add2(v[r][e], less);
            sum = fma2(v[r][e], v[r][e], sum);
          }
        }
        s[r] = __fadd_rn(sum.x, sum.y);
      }
      cta_sum<kR>(s, s_red, turn);
#pragma unroll
      for (int r = 0; r < kR; ++r) {
        if (row + r >= a.rows) break;
        const float rstd = rstd_of(per_width(s[r], width, inv_width), a.eps);
        if (threadIdx.x == 0) {
          if (a.mean) a.mean[row + r] = mean[r];
          if (a.rstd) a.rstd[row + r] = rstd;
        }
        const float2 scale = both(rstd);
        char* const y = static_cast<char*>(a.y) + (row + r) * row_bytes;
#pragma unroll
        for (int u = 0; u < kPairs; u += kUnitPairs) {
          if (cols.first(u) >= a.width) continue;
          float o[2 * kUnitPairs];
#pragma unroll
          for (int k = 0; k < kUnitPairs; ++k) {
            const float2 z = fma2(mul2(v[r][u + k], scale), g[u + k], b[u + k]);
            o[2 * k] = z.x;
            o[2 * k + 1] = z.y;
          }
          store_unit<kT, 2 * kUnitPairs>(y, cols.first(u), o);
        }
      }
    } else {
#pragma unroll
      for (int r = 0; r < kR; ++r) {
        float2 sum = both(0.0f);
        cols.template over<false, 1>(nullptr, {ring.row(r, 0, row + r)}, [&](int, bool, const float2 (&v)[1]) { return sum = add2(sum, v[0]); });
        s[r] = __fadd_rn(sum.x, sum.y);
      }
      cta_sum<kR>(s, s_red, turn);
      ring.refill(row, step);
#pragma unroll
      for (int r = 0; r < kR; ++r) {
        mean[r] = per_width(s[r], width, inv_width);
        const float2 less = both(-mean[r]);
        float2 sum = both(0.0f);
        cols.template over<false, 1>(nullptr, {ring.row(r, 0, row + r)}, [&](int, bool there, const float2 (&v)[1]) {
          float2 d = add2(v[0], less);
          if (!there) d.y = 0.0f;
          return sum = fma2(d, d, sum);
        });
        s[r] = __fadd_rn(sum.x, sum.y);
      }
      cta_sum<kR>(s, s_red, turn);
#pragma unroll
      for (int r = 0; r < kR; ++r) {
        if (row + r >= a.rows) break;
        const float rstd = rstd_of(per_width(s[r], width, inv_width), a.eps);
        if (threadIdx.x == 0) {
          if (a.mean) a.mean[row + r] = mean[r];
          if (a.rstd) a.rstd[row + r] = rstd;
        }
        const float2 less = both(-mean[r]), scale = both(rstd);
        cols.template over<true, 1>(static_cast<char*>(a.y) + (row + r) * row_bytes, {ring.row(r, 0, row + r)},
                                    [&](int e, bool, const float2 (&v)[1]) { return fma2(mul2(add2(v[0], less), scale), g[e], b[e]); });
      }
    }
    ring.next();
  }
  if (s_fail) let_copies_land();
}

template <int kT, bool kPieces, int kValues, int kMax, int kR>
__global__ void __launch_bounds__(kMax)
norm_backward_ring_kernel(const BackwardArgs a, int slot, int sets) {
  constexpr int kPairs = kValues / 2;
  extern __shared__ __align__(128) uint8_t s_rows[];
  __shared__ __align__(8) uint64_t s_bars[kMaxSets];
  __shared__ __align__(16) float s_red[2][32][2 * kR];
  __shared__ int s_fail;
  const Columns<kT, kPieces, kValues> cols{static_cast<int>(threadIdx.x), static_cast<int>(blockDim.x), a.width};
  const int64_t step = static_cast<int64_t>(gridDim.x) * kR;
  const int row_bytes = a.width * elem_bytes<kT>();
  RowRing<kT, kPieces, kR, 2> ring{s_bars, s_rows, sets, slot,
                          {{static_cast<const char*>(a.x), a.ldx * elem_bytes<kT>(), row_bytes, a.rows},
                           {static_cast<const char*>(a.dy), a.lddy * elem_bytes<kT>(), row_bytes, a.rows}}};
  s_fail = 0;
  ring.init();
  wait_for_inputs();
  let_next_begin();
  int64_t row = static_cast<int64_t>(blockIdx.x) * kR;
  ring.begin(row, step);
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
  float2 g[kPairs], dg[kPairs], db[kPairs];
#pragma unroll
  for (int e = 0; e < kPairs; ++e) {
    g[e] = cols.vector(a.gamma, e, 1.0f);
    dg[e] = db[e] = both(0.0f);
  }
  if constexpr (!kPieces) __syncthreads();  // the first rows' starts, which a thread copied
  const float width = static_cast<float>(a.width), inv_width = __fdiv_rn(1.0f, width);
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
      // (past the row dy is 0, and with it all that is added)
      cols.template over<false, 2>(nullptr, {ring.row(r, 0, row + r), ring.row(r, 1, row + r)}, [&](int e, bool, const float2 (&v)[2]) {
        const float2 xh = mul2(add2(v[0], less), scale), h = mul2(v[1], g[e]);
        dg[e] = fma2(v[1], xh, dg[e]);
        db[e] = add2(db[e], v[1]);
        s0 = add2(s0, h);
        return s1 = fma2(h, xh, s1);
      });
      s[2 * r] = __fadd_rn(s0.x, s0.y);
      s[2 * r + 1] = __fadd_rn(s1.x, s1.y);
    }
    cta_sum<2 * kR>(s, s_red, turn);
    ring.refill(row, step);
#pragma unroll
    for (int r = 0; r < kR; ++r) {
      if (!a.dx || row + r >= a.rows) break;
      const float mean_h = per_width(s[2 * r], width, inv_width), mean_hx = per_width(s[2 * r + 1], width, inv_width);
      const float2 less = both(-mean[r]), scale = both(rstd[r]), less_h = both(-mean_h), less_hx = both(-mean_hx);
      cols.template over<true, 2>(static_cast<char*>(a.dx) + (row + r) * row_bytes, {ring.row(r, 0, row + r), ring.row(r, 1, row + r)},
                                  [&](int e, bool, const float2 (&v)[2]) {
        const float2 xh = mul2(add2(v[0], less), scale);
        return mul2(scale, fma2(xh, less_hx, add2(mul2(v[1], g[e]), less_h)));
      });
    }
    ring.next();
  }
  if (s_fail) let_copies_land();
  if (!a.partial) return;
  float* const to_gamma = a.partial + static_cast<int64_t>(blockIdx.x) * a.width;
  float* const to_beta = to_gamma + static_cast<int64_t>(gridDim.x) * a.width;
#pragma unroll
  for (int e = 0; e < kPairs; ++e) {
    if (cols.first(e) < a.width) {
      to_gamma[cols.first(e)] = dg[e].x;
      to_beta[cols.first(e)] = db[e].x;
    }
    if (cols.second(e) < a.width) {
      to_gamma[cols.second(e)] = dg[e].y;
      to_beta[cols.second(e)] = db[e].y;
    }
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

int values_of(int width) { return width <= kMaxThreads * kFew ? kFew : kMany; }
int threads_of(int width) { return (width + 32 * values_of(width) - 1) / (32 * values_of(width)) * 32; }

// CTAs to an SM, by the registers that a thread takes: in the forward pass some
// 100 for two rows of pieces and 64 for one row without, in the backward pass up
// to 128, and more of rows with many values.
int per_sm(int width, int threads) { return std::max(1, std::min((values_of(width) == kFew ? threads : 384) / threads_of(width), 16)); }
int forward_per_sm(int width, bool pieces) { return per_sm(width, pieces ? 512 : 1024); }
int backward_per_sm(int width) { return per_sm(width, 512); }

// CTAs of the backward pass, and so rows of its workspace, at most: as many as
// are resident, each with two rows or more, since every one adds a row of sums.
int64_t backward_ctas(int64_t rows, int width, int sms) {
  const bool warp = width <= kWarpWidth;
  const int64_t most = static_cast<int64_t>(sms) * (warp ? 2 : backward_per_sm(width));
  const int64_t each = 2 * (warp ? kWarps : 1), need = (rows + each - 1) / each;
  return std::min(need, most);
}

constexpr int64_t kRingBytes = 200 << 10;  // of an SM's shared memory

// Rows that a CTA of the ring kernels takes at a time, whose slots have so many
// bytes, where `ctas` share an SM's shared memory: `most`, or one where that
// does not fit or leaves a CTA less than two sets; 0 where one does not either.
int rows_at_a_time(int64_t slot, int ctas, int64_t rows_each, int most) {
  for (const int r : {most, 1})
    if (2 * r * slot * ctas <= kRingBytes && rows_each >= 2 * r) return r;
  return 0;
}
// Sets of so many bytes that a CTA keeps.
int sets_of(int64_t bytes, int ctas) { return static_cast<int>(std::min<int64_t>(kMaxSets, kRingBytes / ctas / bytes)); }

// Bytes that a row's pieces take.
int64_t slot_of(int64_t row_bytes, bool pieces) { return pieces ? row_bytes : (row_bytes + 15 + 15) / 16 * 16; }

template <typename... Params, typename... Args>
bwd_status launch_ring(void (*kernel)(Params...), int64_t ctas, int threads, int smem, cudaStream_t st, const char* what, const Args&... args) {
  if (smem > 40 * 1024) {  // 48 KB, less the static variables
    const cudaError_t e = opt_in(kernel, static_cast<int>(kRingBytes));
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

// Values of the largest unit that all of a call's rows consist of and start on:
// a piece of 16 bytes, 4 bytes, or one value.
int unit_values(int eb, uintptr_t addresses, int64_t row_bytes) {
  const uintptr_t all = addresses | static_cast<uintptr_t>(row_bytes);
  return all % 16 == 0 ? 16 / eb : all % 4 == 0 ? 4 / eb : 1;
}

// Calls f<type, unit>.
template <typename F>
bwd_status by_type(int type, int values, F f) {
  const auto typed = [&](auto t) {
    constexpr int kT = decltype(t)::value, kEb = elem_bytes<kT>();
    if (values == 16 / kEb) return f(t, std::integral_constant<int, 16 / kEb>{});
    if constexpr (kEb != 4)
      if (values == 2) return f(t, std::integral_constant<int, 2>{});
    return f(t, std::integral_constant<int, 1>{});
  };
  if (type == BWD_F32) return typed(std::integral_constant<int, kF32>{});
  if (type == BWD_BF16) return typed(std::integral_constant<int, kBF16>{});
  return typed(std::integral_constant<int, kF16>{});
}

template <int kT, int kVals>
bwd_status launch_forward(const ForwardArgs& a, int sms, cudaStream_t st) {
  constexpr bool kPieces = kVals * elem_bytes<kT>() == 16;
  const auto plain = [&](auto* kernel, int64_t ctas, int threads) {
    return launch_ex(kernel, dim3(static_cast<unsigned>(ctas)), threads, 0, 0, st, "norm_forward_kernel launch", a);
  };
  if (a.width <= kWarpWidth)
    return plain(norm_forward_kernel<kT, kVals, kFew, true>, std::min<int64_t>((a.rows + kWarps - 1) / kWarps, 3 * sms), 32 * kWarps);
  const int threads = threads_of(a.width), per = forward_per_sm(a.width, kPieces);
  const int64_t ctas = std::min<int64_t>(a.rows, static_cast<int64_t>(sms) * per), slot = slot_of(a.width * elem_bytes<kT>(), kPieces);
  const int r = rows_at_a_time(slot, per, a.rows / ctas, !kPieces ? 1 : 2);
  const auto ring = [&](auto* kernel) {
    const int sets = sets_of(r * slot, per);
    return launch_ring(kernel, ctas, threads, static_cast<int>(sets * r * slot), st, "norm_forward_ring_kernel launch", a, static_cast<int>(slot), sets);
  };
  if (values_of(a.width) == kFew) {
    if constexpr (kPieces)
      if (r == 2) return ring(norm_forward_ring_kernel<kT, kPieces, kFew, kMaxThreads, 2>);
    if (r == 1) return ring(norm_forward_ring_kernel<kT, kPieces, kFew, kMaxThreads, 1>);
    return plain(norm_forward_kernel<kT, kVals, kFew, false>, ctas, threads);
  }
  if constexpr (kPieces)
    if (r == 2) return ring(norm_forward_ring_kernel<kT, kPieces, kMany, kMaxThreads, 2>);
  if (r == 1) return ring(norm_forward_ring_kernel<kT, kPieces, kMany, kMaxThreads, 1>);
  return plain(norm_forward_kernel<kT, kVals, kMany, false>, ctas, threads);
}

template <int kT, int kVals>
bwd_status launch_backward(const BackwardArgs& a, int64_t ctas, cudaStream_t st) {
  constexpr bool kPieces = kVals * elem_bytes<kT>() == 16;
  const auto plain = [&](auto* kernel, int threads) {
    return launch_ex(kernel, dim3(static_cast<unsigned>(ctas)), threads, 0, 0, st, "norm_backward_kernel launch", a);
  };
  if (a.width <= kWarpWidth) return plain(norm_backward_kernel<kT, kVals, kFew, true>, 32 * kWarps);
  const int threads = threads_of(a.width), per = backward_per_sm(a.width);
  const int64_t slot = slot_of(a.width * elem_bytes<kT>(), kPieces);
  const int r = rows_at_a_time(2 * slot, per, a.rows / ctas, kPieces && values_of(a.width) == kFew ? 2 : 1);
  const auto ring = [&](auto* kernel) {
    const int sets = sets_of(2 * r * slot, per);
    return launch_ring(kernel, ctas, threads, static_cast<int>(sets * 2 * r * slot), st, "norm_backward_ring_kernel launch", a, static_cast<int>(slot), sets);
  };
  if (values_of(a.width) == kFew) {
    if constexpr (kPieces)
      if (r == 2) return ring(norm_backward_ring_kernel<kT, kPieces, kFew, kMaxThreads, 2>);
    if (r == 1) return ring(norm_backward_ring_kernel<kT, kPieces, kFew, kMaxThreads, 1>);
    return plain(norm_backward_kernel<kT, kVals, kFew, false>, threads);
  }
  // (a thread's sums and values fit its registers where a CTA has no more than 384)
  if (r == 1 && threads <= 384) return ring(norm_backward_ring_kernel<kT, kPieces, kMany, 384, 1>);
  if (r == 1) return ring(norm_backward_ring_kernel<kT, kPieces, kMany, kMaxThreads, 1>);
  return plain(norm_backward_kernel<kT, kVals, kMany, false>, threads);
}

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
  return by_type(dtype, values, [&](auto t, auto v) {
    return launch_forward<decltype(t)::value, decltype(v)::value>(a, sms, static_cast<cudaStream_t>(stream));
  });
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
    s = by_type(dtype, values, [&](auto t, auto v) { return launch_backward<decltype(t)::value, decltype(v)::value>(a, ctas, st); });
    if (s != BWD_OK) return s;
  }
  if (!sums) return BWD_OK;
  const SumArgs a{static_cast<const float*>(work), rows > 0 ? ctas : 0, static_cast<int>(width), {dgamma, dbeta}, {vector_dtype, vector_dtype}};
  return launch_ex(norm_sums_kernel, dim3(static_cast<unsigned>((width + 31) / 32), 2), 32 * kSumWarps, 0, 0, st, "norm_sums_kernel launch", a);
}

}  // extern "C"
