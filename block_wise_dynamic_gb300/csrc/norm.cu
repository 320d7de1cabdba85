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
  __device__ __forceinline__ float value(int i, int j) const {
    const char* const at = reinterpret_cast<const char*>(&u[i]);
    if constexpr (kT == kF32) {
      return reinterpret_cast<const float*>(at)[j];
    } else {
      const unsigned short h = reinterpret_cast<const unsigned short*>(at)[j];
      if constexpr (kT == kBF16) return __uint_as_float(static_cast<uint32_t>(h) << 16);
      else return __half2float(__ushort_as_half(h));
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
  wait_for_inputs();
  let_next_begin();
  Part<kT, kVals> next;
  if (row < a.rows) next.load(static_cast<const char*>(a.x) + row * a.ldx * elem_bytes<kT>(), a.width, t, threads);
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
    if (row + groups < a.rows)
      next.load(static_cast<const char*>(a.x) + (row + groups) * a.ldx * elem_bytes<kT>(), a.width, t, threads);
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
  extern __shared__ float s_sums[];  // [2][width]: of wide rows, or of a CTA's warps
  __shared__ float s_red[2][2][32];
  const int threads = kWarp ? 32 : blockDim.x, t = kWarp ? threadIdx.x % 32 : threadIdx.x;
  const int64_t groups = kWarp ? static_cast<int64_t>(gridDim.x) * kWarps : gridDim.x;
  int64_t row = kWarp ? static_cast<int64_t>(blockIdx.x) * kWarps + threadIdx.x / 32 : blockIdx.x;
  GroupSum<kWarp, 2> sum{s_red};
  wait_for_inputs();
  let_next_begin();
  Part<kT, kVals> next_x, next_dy;
  float next_mean = 0.0f, next_rstd = 0.0f;
  const auto fetch = [&](int64_t r) {
    next_x.load(static_cast<const char*>(a.x) + r * a.ldx * elem_bytes<kT>(), a.width, t, threads);
    next_dy.load(static_cast<const char*>(a.dy) + r * a.lddy * elem_bytes<kT>(), a.width, t, threads);
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
    float h[kThreadValues], xh[kThreadValues];
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
      const int c = (i * threads + t) * kVals;
      const bool in = c < a.width;
#pragma unroll
      for (int j = 0; j < kVals; ++j) {
        const int e = i * kVals + j;
        const float d = dy.value(i, j);
        xh[e] = in ? __fmul_rn(__fsub_rn(x.value(i, j), mean), rstd) : 0.0f;
        float gamma = 0.0f;
        if constexpr (kKeep) {
          gamma = g[e];
          dg[e] = __fmaf_rn(d, xh[e], dg[e]);
          db[e] = __fadd_rn(db[e], d);
        } else if (in) {
          gamma = vector_at<kT>(a.gamma, c + j, 1.0f);
          if (a.partial) {
            s_sums[c + j] = __fmaf_rn(d, xh[e], s_sums[c + j]);
            s_sums[a.width + c + j] = __fadd_rn(s_sums[a.width + c + j], d);
          }
        }
        h[e] = __fmul_rn(d, gamma);
        s[0] += h[e];
        s[1] = __fmaf_rn(h[e], xh[e], s[1]);
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
        const int e = i * kVals + j;
        out[j] = __fmul_rn(rstd, __fmaf_rn(-xh[e], mean_hx, __fsub_rn(h[e], mean_h)));
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

// Sums of the CTAs' rows: eight warps of a CTA each add every eighth of 32
// columns' rows, in order, and the first then adds the eight.
constexpr int kSumWarps = 8;

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
#pragma unroll 8
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

constexpr int kSms = 160;             // at least as many as the device has
constexpr int kThreadsPerSm = 1024;

// CTAs of the backward pass, and so rows of its workspace, at most.
int64_t backward_ctas(int64_t rows, int width, int sms) {
  const int threads = width <= kWarpWidth ? 32 * kWarps : (width + 32 * kThreadValues - 1) / (32 * kThreadValues) * 32;
  const int64_t most = static_cast<int64_t>(sms) * (threads < kThreadsPerSm ? kThreadsPerSm / threads : 1);
  const int64_t need = width <= kWarpWidth ? (rows + kWarps - 1) / kWarps : rows;
  return need < most ? need : most;
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

int threads_of(int width, int values) {
  const int per = 32 * kThreadValues;
  (void)values;
  return (width + per - 1) / per * 32;
}

template <template <int, int, bool, int> class Launch, typename Args, typename... More>
bwd_status by_type(int type, int values, int width, const Args& a, More... more) {
  const auto sized = [&](auto t, auto v) {
    constexpr int kT = decltype(t)::value, kVals = decltype(v)::value;
    if (width <= kWarpWidth) return Launch<kT, kVals, true, 32 * kWarps>::go(a, more...);
    const int threads = threads_of(width, kVals);
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
    const int threads = kWarp ? 32 * kWarps : threads_of(a.width, kVals);
    const int64_t most = static_cast<int64_t>(sms) * (2 * kThreadsPerSm / threads), need = kWarp ? (a.rows + kWarps - 1) / kWarps : a.rows;
    return launch_ex(norm_forward_kernel<kT, kVals, kWarp, kMax>, dim3(static_cast<unsigned>(need < most ? need : most)), threads, 0, 0, st,
                     "norm_forward_kernel launch", a);
  }
};

template <int kT, int kVals, bool kWarp, int kMax>
struct LaunchBackward {
  static bwd_status go(const BackwardArgs& a, int64_t ctas, cudaStream_t st) {
    const int threads = kWarp ? 32 * kWarps : threads_of(a.width, kVals);
    const int smem = a.partial && (kWarp || kMax == kMaxThreads) ? 8 * a.width : 0;
    if (smem > 48 * 1024) {
      const cudaError_t e = opt_in(norm_backward_kernel<kT, kVals, kWarp, kMax>, 8 * kMaxWidth);
      if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute(MaxDynamicSharedMemorySize)");
    }
    return launch_ex(norm_backward_kernel<kT, kVals, kWarp, kMax>, dim3(static_cast<unsigned>(ctas)), threads, 0, smem, st,
                     "norm_backward_kernel launch", a);
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
